// Decode attention whose contexts are laid end to end and cut into equal parts,
// one per warp: over caches held in 4 bits, and through a window of the newest
// tokens with the first ones (the sinks) kept visible.
//
//   out = sum_i p_i v_i / sum_i p_i,  p_i = 2^(scale log2(e) q . k_i - m)
//
// over the tokens i that the query's token, at position P, sees: i <= P and
// (i < sinks or i > P - window).
//
// Split.  A sequence's tiles (of 16 tokens, of 32 for 8-bit and 4-bit rows) are those
// that hold a token some query of it sees, the sinks' first.  The tiles of all
// sequences make one line, cut into as many equal parts as there are resident warps
// per head, and each head's warp takes its rows of the part, so that a batch of any
// lengths ends everywhere at once without partitions chosen by the caller, and the
// heads of a block, which lie together in the pool, are read at about one time.
// Before each sequence the line has a gap of kFlatGap places, which hold no tile: what
// coming to a sequence and leaving it costs, so that a part of many short ones holds
// fewer tiles.  Every CTA finds its warps' parts from context_lens by one scan.  A
// sequence that lies within a part is written by the part's warps; of one that is cut,
// each warp leaves a piece (o, m, l) in the workspace, at most two per warp, and
// flat_join_kernel joins the pieces by log-sum-exp in the order of the tokens.
// Where there are so few contexts that each has CTAs of its own, a cluster takes each
// (flat_cluster): its warps share the tiles equally, leave their pieces in shared memory
// and join them there, with no second kernel.
//
// A warp works by itself from its part's first tile to the last, without barriers: it
// copies the K and V rows of tiles to come (cp.async, swizzled) into its own ring in
// shared memory, across contexts, and keeps the running maximum and the sums of the
// context it is in (m16n8k16 MMAs, S^T = K Q^T and O^T += V^T P^T, with the query
// columns padded to 8 or 16).  Rows that no query sees are not read, nor is the block
// table where a block has none of the others.
//
// 4-bit rows: value = low + code * scale, codes 0 .. 15, with (scale, low) per
// 64 channels.  Taken from a word by a mask alone, a pair of codes in its place is
// a pair of f16 numbers: in the last bits of a subnormal one a code is code 2^-24, in
// the four bits above them 16 code 2^-24.  So a word of eight codes becomes four MMA
// operands by four masks and one shift, with no conversion; the 16 goes into q (of
// K) and the output's factor (of V).  With A = sum of q code over a group's channels,
// which the MMA gives, and Q = sum of q,
//   q . k = sum over groups of scale A + low Q.
// q is rounded to f16 after the scaling that puts the context's largest |q| in
// [2^14, 2^15): exact but for entries 2^-25 below it.  The second product's
// weights p scale leave f16's range; as for row-scaled caches each query column has
// a running R near the largest product seen, p scale / R is rounded to f16 (half a
// step, 2^-11) and R multiplies the sums at the end.
// All codes being positive, the sums of a long context would grow far above the
// output, which the least values take them back to, and lose bits on the way.  So
// codes of V are counted from the top in rows of odd place, v = (low + 15 scale) -
// scale (15 - code): the sums of the two kinds of rows keep near 0.
// The weights' rounding so meets scale code, some times as large as the value where
// that is near 0.  CENTRED, for f16 outputs, whose own rounding it would pass: the
// codes' middle is left to the exact weights, v = (low + 7.5 scale) + scale (code -
// 7.5), by subtracting 7.5 times the sum of the rounded weights at the end, and what
// remains is the rounding of weights times values (a window of 4 tokens: 2.3e-4 of the
// outputs instead of 3.2e-4, their own rounding being 2.1e-4; eight contexts of up to
// 131072 tokens: 156 us instead of 151, a second MMA on what the rounding leaves 175).
#pragma once

#include <math_constants.h>

#include <type_traits>

#include "pa_decode.cuh"
#include "pa_flat.h"
#include "pa_launch.h"
#include "pa_peer.cuh"

namespace pa {

// The first token in the window of the token at position P.
__device__ __forceinline__ int window_low(int window, int P) { return window > 0 ? max(0, max(P, 0) - window + 1) : 0; }

// Tokens of a tile, and of what a warp attends to at a time: more of the narrower rows,
// so that what a step costs whatever its rows hold is shared by more of them.
template <int KV, int D>
constexpr int flat_rows() { return KV == kInt4 ? (D == 64 ? 64 : 32) : (KV == kE4M3 ? 32 : 16); }
template <int KV>
constexpr int flat_parts() { return KV == kInt4 || KV == kE4M3 ? 2 : 1; }  // of 16 tokens

// A sequence's tiles (T tokens each).
template <int T>
struct FlatSpan {
  int L;           // length, clamped to the table
  int sink_tiles;  // tiles of the sinks, before the window's
  int first;       // the window's first tile
  int tiles;       // at least one, also where nothing is seen
  __device__ __forceinline__ FlatSpan(const FlatParams& p, int len) {
    L = min(max(len, 0), p.maxB << p.bs_log2);
    first = window_low(p.window, L - p.qlen) / T;
    sink_tiles = min((min(p.sinks, L) + T - 1) / T, first);
    tiles = max(1, sink_tiles + (L + T - 1) / T - first);
  }
  __device__ __forceinline__ int token(int t) const { return (t < sink_tiles ? t : first + t - sink_tiles) * T; }
};

// Shared memory of a tile: its rows of K, those of V, and of 4-bit caches their
// parameters.
template <int KV, int D>
struct FlatGeom {
  static constexpr int ROWS = flat_rows<KV, D>();  // a tile
  static constexpr int ROWB = KV == kInt4 ? D / 2 : (KV == kE4M3 ? D : 2 * D);
  static constexpr int PARB = KV == kInt4 ? D / kGroupChannels * 4 : 0;  // of a row
  static constexpr int STAGE = 2 * ROWS * (ROWB + PARB);
  static constexpr int CHUNKS = ROWB / 16;  // 16-byte pieces of a row
  // Address of 16-byte chunk c of row r: chunks are permuted within lines of 128 bytes
  // (within a row's first 128 bytes and its second ones where it has more) so that
  // eight rows' chunks of one index lie in different banks.
  static __device__ __forceinline__ uint32_t chunk(int r, int c) {
    if constexpr (ROWB == 32) return (r >> 2) * 128 + (((r & 3) * 2 + (c ^ ((r >> 2) & 1))) * 16);
    if constexpr (ROWB == 64) return r * 64 + ((c ^ ((r >> 1) & 3)) * 16);
    return r * ROWB + ((c ^ (r & 7)) * 16);
  }
};

template <int KV, int D, int NG>
constexpr int flat_min_ctas() {
  if (KV == kInt4) return NG == 8 ? (D == 64 ? 4 : 3) : (D == 64 ? 3 : 2);
  if (KV == kE4M3) return NG == 8 ? 3 : 2;
  return D == 64 && NG == 8 ? 3 : 2;
}

// Stages of a warp's ring: what the SM's shared memory holds for the variant's CTAs.
constexpr int kFlatMaxStages = 8;
template <int KV, int D, int NG>
__host__ __device__ constexpr int flat_stages() {
  const int n = (228 * 1024 / flat_min_ctas<KV, D, NG>() - 2048) / (kFlatWarps * FlatGeom<KV, D>::STAGE);
  return n < 2 ? 2 : (n > kFlatMaxStages ? kFlatMaxStages : n);
}
template <int KV, int D, int NG>
__host__ __device__ constexpr int flat_smem() {
  return flat_stages<KV, D, NG>() * kFlatWarps * FlatGeom<KV, D>::STAGE;
}

__device__ __forceinline__ uint2 load8_shared(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint32_t load4_shared(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.b32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// mma16816<false> onto sums of 0
__device__ __forceinline__ void mma16816_zero(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
// (w ^ flip) & MASK in one operation: flip in a register, whatever its value
template <uint32_t MASK>
__device__ __forceinline__ uint32_t flip_and(uint32_t w, uint32_t flip) {
  uint32_t d;
  asm("lop3.b32 %0, %1, %2, %3, 0x28;" : "=r"(d) : "r"(w), "r"(flip), "n"(MASK));
  return d;
}
// Nibbles k and k + 4 of a word, k = 0 .. 3, as pairs of subnormal f16 numbers: code
// 2^-24 (k even), 16 code 2^-24 (k odd).
__device__ __forceinline__ void codes_of(uint32_t w, uint32_t (&x)[4]) {
  x[0] = w & 0x000F000Fu;
  x[1] = w & 0x00F000F0u;
  x[2] = w >> 8 & 0x000F000Fu;
  x[3] = w >> 8 & 0x00F000F0u;
}
// The same with the bits of `flip` (0xFFFF0000: 15 - code in the upper half) inverted.
__device__ __forceinline__ void flipped_codes_of(uint32_t w, uint32_t flip, uint32_t (&x)[4]) {
  x[0] = flip_and<0x000F000Fu>(w, flip);
  x[1] = flip_and<0x00F000F0u>(w, flip);
  x[2] = flip_and<0x000F000Fu>(w >> 8, flip);
  x[3] = flip_and<0x00F000F0u>(w >> 8, flip);
}
// base + n * bytes, one instruction
__device__ __forceinline__ const uint8_t* at_octet(const uint8_t* base, uint32_t n, uint32_t bytes) {
  uint64_t d;
  asm("mad.wide.u32 %0, %1, %2, %3;" : "=l"(d) : "r"(n), "r"(bytes), "l"(reinterpret_cast<uint64_t>(base)));
  return reinterpret_cast<const uint8_t*>(d);
}
// sums += the two f16 numbers of w
__device__ __forceinline__ void add_pair(float (&sums)[2], uint32_t w) {
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\tadd.f32.f16 %0, lo, %0;\n\tadd.f32.f16 %1, hi, %1;\n\t}"
      : "+f"(sums[0]), "+f"(sums[1])
      : "r"(w));
}
__device__ __forceinline__ float max3(float a, float b, float c) {
  float d;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(d) : "f"(a), "f"(b), "f"(c));
  return d;
}
constexpr float kLeastMax = -3.40282347e38f;  // a maximum before any score: every weight it gives is 0
constexpr float kCodeUnit = 5.9604644775390625e-8f;  // 2^-24
constexpr float kFlatMostInvR = 1.32922799578491587e36f;  // 2^120: times a weight it is still finite

__device__ __forceinline__ float bf16_low(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float bf16_high(uint32_t w) { return __uint_as_float(w & 0xFFFF0000u); }

__device__ __forceinline__ uint32_t bits_below(int n) {  // of 32
  return n >= 32 ? 0xFFFFFFFFu : (1u << max(n, 0)) - 1u;
}

// Of tokens pos .. pos + 31, those in [low, end) and those in [0, sinks) before end.
__device__ __forceinline__ uint32_t seen_bits(int pos, int end, int low, int sinks) {
  return bits_below(end - pos) & (~bits_below(low - pos) | bits_below(sinks - pos));
}

// Four channels' sums of a query column over pieces (o, m, l), joined by log-sum-exp.
struct FlatSums {
  float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
  float m = kLeastMax, l = 0.f;
  __device__ __forceinline__ void add(float4 v, float2 x) {
    const float M = fmaxf(m, x.x);
    const float a = ex2(m - M), b = ex2(x.x - M);
    o.x = o.x * a + v.x * b;
    o.y = o.y * a + v.y * b;
    o.z = o.z * a + v.z * b;
    o.w = o.w * a + v.w * b;
    l = l * a + x.y * b;
    m = M;
  }
  __device__ __forceinline__ void store(const FlatParams& p, int64_t place, float inv) const {  // times inv, four numbers
    reinterpret_cast<uint2*>(p.out)[place] =
        p.q_bf16 ? make_uint2(pack2<true>(o.x * inv, o.y * inv), pack2<true>(o.z * inv, o.w * inv))
                 : make_uint2(pack2<false>(o.x * inv, o.y * inv), pack2<false>(o.z * inv, o.w * inv));
  }
};

// Tiles of each warp of the cluster that shares a context of `tiles`.
__device__ __forceinline__ int shared_tiles(int tiles, int cluster) {
  const int warps = cluster * kFlatWarps;
  return (tiles + warps - 1) / warps;
}

// SHARED: a cluster of p.cluster CTAs per context.
template <int KV, int D, int NG, bool CENTRED, bool SHARED>
__global__ void __launch_bounds__(kFlatThreads, (flat_min_ctas<KV, D, NG>())) flat_kernel(const FlatParams p) {
  using Gm = FlatGeom<KV, D>;
  constexpr int NST = flat_stages<KV, D, NG>();
  constexpr int SUB = flat_parts<KV>(), ROWS = Gm::ROWS, OCTS = ROWS / 8, ROWB = Gm::ROWB, PARB = Gm::PARB;
  constexpr int NT = NG / 8, KS = D / 16, GRP = D / kGroupChannels;
  constexpr bool I4 = KV == kInt4, BF = KV == kBF16;
  constexpr uint32_t ALL = SUB == 2 ? 0xFFFFFFFFu : 0xFFFFu;  // of a part of the tile
  constexpr float kHeadroom = 5.f;  // a weight grows to 2^5 before its maximum moves
  using Span = FlatSpan<ROWS>;
  static_assert(!CENTRED || I4, "4-bit rows' weights");
  static_assert(ROWS <= kFlatTile && flat_min_ctas<KV, D, NG>() <= kFlatCtasPerSm, "the workspace's and the checks' limits");

  extern __shared__ __align__(128) uint8_t smem[];
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31, qr = lane >> 2, qc = lane & 3;
  __shared__ int64_t warp_tiles[kFlatWarps];
  __shared__ int64_t found_at[kFlatWarps];  // the places before the sequence where a warp's part begins
  __shared__ int found[kFlatWarps][2];      // that sequence, and its length
  // query column n is head n % G of new token n / G: its token, and its row of q and out
  // after the context's first
  __shared__ int col_token[NG], col_row[NG];
  pdl_enter();

  const int ncol = p.G * p.qlen;
  if (tid < NG) {
    const int n = min(tid, ncol - 1), j = n / p.G;
    col_token[tid] = j;
    col_row[tid] = j * p.Hq + n - j * p.G;
  }
  const int id = blockIdx.x * kFlatWarps + warp;
  [[maybe_unused]] const int rank = SHARED ? cluster_rank() : 0;
  int head, at_s, at_t, places, to_come = 0;  // the warp begins at tile at_t of sequence at_s, `places` in all
  [[maybe_unused]] int64_t u0 = 0, part = 0;
  Span c(p, 0);
  if constexpr (SHARED) {
    // ---- the warp's part of the cluster's context ----
    const int context = blockIdx.x / p.cluster;
    at_s = context / p.heads;
    head = context % p.heads;
    const int len = load_written(p.context_lens + at_s);
    c = Span(p, len);
    if (c.L != len && head == 0 && rank == 0 && tid == 0) atomicOr(p.err, kErrContextLen);
    const int share = shared_tiles(c.tiles, p.cluster);
    at_t = min((rank * kFlatWarps + warp) * share, c.tiles);
    places = min(share, c.tiles - at_t);
    __syncthreads();
  } else {
    // ---- the warp's part of the line ----
    const int per = (p.S + kFlatThreads - 1) / kFlatThreads;
    const int s_lo = min(p.S, tid * per), s_hi = min(p.S, s_lo + per);
    int64_t mine = 0;
    for (int s = s_lo; s < s_hi; ++s) {
      const int len = load_written(p.context_lens + s);
      const Span c(p, len);
      if (c.L != len && blockIdx.x == 0) atomicOr(p.err, kErrContextLen);
      mine += c.tiles + p.gap;
    }
    int64_t incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xFFFFFFFFu, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) warp_tiles[warp] = incl;
    __syncthreads();
    int64_t total = 0, before = incl - mine;
#pragma unroll
    for (int w = 0; w < kFlatWarps; ++w) {
      if (w < warp) before += warp_tiles[w];
      total += warp_tiles[w];
    }
    part = max(static_cast<int64_t>(p.least_part), (total + p.nparts - 1) / p.nparts);
#pragma unroll 1
    for (int w = 0; w < kFlatWarps; ++w) {  // where the warps' parts begin: one thread each
      const int64_t u = part * ((blockIdx.x * kFlatWarps + w) / p.heads);
      if (u < before || u >= before + mine) continue;
      int64_t at = before;
      for (int s = s_lo;; ++s) {
        const int len = load_written(p.context_lens + s), n = Span(p, len).tiles + p.gap;
        if (u < at + n) {
          found[w][0] = s;
          found[w][1] = len;
          found_at[w] = at;
          break;
        }
        at += n;
      }
    }
    __syncthreads();
    head = id % p.heads;
    if (id >= p.nparts * p.heads) return;
    u0 = part * (id / p.heads);
    const int64_t u1 = min(u0 + part, total);
    if (p.nparts > 1 && !p.by_context && lane == 0) p.ws_joins[id] = make_int4(0, 0, 0, 0);
    if (u0 >= u1) return;
    // tile at_t's place on the line is `to_come` places after the part's first
    places = static_cast<int>(u1 - u0);
    at_s = found[warp][0];
    c = Span(p, found[warp][1]);
    const int into = static_cast<int>(u0 - found_at[warp]) - p.gap;
    to_come = max(-into, 0);
    at_t = max(into, 0);
    if (to_come >= places) return;  // a gap, and no tile
  }

  // ---- loads ----
  const int log8 = p.bs_log2 - 3, cache_heads = p.heads / p.head_div, kv_head = head / p.head_div;
  const uint32_t ring = smem_u32(smem) + warp * NST * Gm::STAGE;
  // A context's tiles [lo, hi) whose rows every query sees: neither copies nor scores
  // have anything to mask there.
  const auto whole_tiles = [&](const Span& c, int& lo, int& hi) {
    const int to_first = c.first - c.sink_tiles;
    lo = max(c.sink_tiles, (window_low(p.window, c.L - 1) + ROWS - 1) / ROWS - to_first);
    hi = max(c.L - p.qlen + 1, 0) / ROWS - to_first;
  };
  // What is copied next: `run_left` tiles from token ld_pos on, all of them whole or none
  // (then tile ld_t of sequence ld_s), `to_load` places of the part behind them.
  int ld_s = at_s, ld_t = at_t, to_load = places - to_come, ld_L = c.L;
  int run_left = 0, ld_pos = 0;
  bool run_whole = false;
  const auto next_run = [&]() {
    Span d(p, ld_L);
    if (ld_t == d.tiles) {
      to_load -= p.gap;
      if (to_load <= 0) return;
      ++ld_s;
      ld_t = 0;
      d = Span(p, load_written(p.context_lens + ld_s));
      ld_L = d.L;
    }
    if (to_load <= 0) return;
    int lo, hi, end = ld_t < d.sink_tiles ? d.sink_tiles : d.tiles;
    whole_tiles(d, lo, hi);
    run_whole = ld_t >= lo && ld_t < hi;
    if (run_whole) end = min(end, hi);
    if (ld_t < lo) end = min(end, lo);
    run_left = min(end - ld_t, to_load);
    ld_pos = d.token(ld_t);
    to_load -= run_left;
    ld_t += run_left;
  };
  // The next tile to copy: whether a query sees any of it, its first token, and of the
  // eight tokens 8 (lane % OCTS) on which ones are seen (bits) and their table entry.
  bool copying = false;
  uint32_t seen8 = 0;
  int entry = 0, place = 0;
  const int oct = lane % OCTS;
  const auto look_up = [&]() {
    if (run_left == 0) next_run();
    copying = run_left > 0;
    if (!copying) return;
    --run_left;
    place = ld_pos;
    ld_pos += ROWS;
    seen8 = 0xFFu;
    if (!run_whole) {
      seen8 &= seen_bits(place + 8 * oct, ld_L, window_low(p.window, ld_L - p.qlen), p.sinks);
      copying = __any_sync(0xFFFFFFFFu, seen8 != 0);
    }
    entry = 0;
    if (seen8 != 0) entry = load_written(p.block_tables + static_cast<int64_t>(ld_s) * p.maxB + ((place + 8 * oct) >> p.bs_log2));
  };
  // this lane's places in the copies: RPC rows at a time
  constexpr int RPC = 32 / Gm::CHUNKS, COPIES = ROWS / RPC;
  const uint8_t* k_lane = static_cast<const uint8_t*>(p.k_cache) + ((lane / Gm::CHUNKS) & 7) * ROWB + lane % Gm::CHUNKS * 16;
  const uint8_t* v_lane = static_cast<const uint8_t*>(p.v_cache) + ((lane / Gm::CHUNKS) & 7) * ROWB + lane % Gm::CHUNKS * 16;
  const uint32_t dst_lane = Gm::chunk(lane / Gm::CHUNKS, lane % Gm::CHUNKS);
  // of copy i: rows of 128 bytes and more go by their low three bits
  const auto dst_of = [&](int i) { return (ROWB >= 128 ? dst_lane ^ (i * RPC % 8 * 16) : dst_lane) + i * RPC * ROWB; };
  // eight rows of a head are contiguous: their index in the pool (of 256 bytes and more
  // each, so that 32 bits count them), of which these are a block's and the lane's parts
  const uint32_t block_octets = static_cast<uint32_t>(cache_heads) << log8;
  const uint32_t lane_octet = (static_cast<uint32_t>(kv_head) << log8) + (ROWS >= 32 ? oct & ((1 << log8) - 1) : 0);
  // of 4-bit caches also their parameters: PER pieces of 16 bytes of K's, then of V's
  constexpr int PER = ROWS * PARB / 16, PPG = I4 ? 8 * PARB / 16 : 1;  // PPG: of eight tokens
  static_assert(!I4 || PER == 16, "one piece per lane");
  [[maybe_unused]] const uint8_t* par_lane =
      static_cast<const uint8_t*>(I4 && lane >= PER ? p.v_params : p.k_params) + lane % PPG * 16;
  uint32_t load_stage = ring;
  const auto copy_tile = [&]() {  // one group of copies, an empty one past the end
    if (copying) {
      // this lane's octet of the tile, block 0's where there is nothing to read
      if (static_cast<uint32_t>(entry) >= p.blocks32) {
        if (seen8 != 0) atomicOr(p.err, kErrBlockId);
        entry = 0;
        seen8 = 0;  // zeros
      }
      uint32_t octet = static_cast<uint32_t>(entry) * block_octets + lane_octet;
      if constexpr (ROWS < 32) octet += ((place >> 3) + oct) & ((1 << log8) - 1);
      // the octets whose rows copy i takes, and those of the lane's parameters
      const auto octet_of = [&](int i) { return RPC == 16 ? 2 * i + (lane >> 4) : i * RPC / 8; };
      [[maybe_unused]] const int par_octet = lane % (I4 ? PER : 1) / PPG;
      constexpr int BYTES = 8 * ROWB;
      const auto within = [](int i) { return RPC == 16 ? 0 : i * RPC % 8 * ROWB; };
      if (__all_sync(0xFFFFFFFFu, seen8 == 0xFFu)) {
#pragma unroll
        for (int i = 0; i < COPIES; ++i) {
          const uint32_t o = __shfl_sync(0xFFFFFFFFu, octet, octet_of(i));
          copy_async<16>(load_stage + dst_of(i), at_octet(k_lane, o, BYTES) + within(i));
          copy_async<16>(load_stage + ROWS * ROWB + dst_of(i), at_octet(v_lane, o, BYTES) + within(i));
        }
        if constexpr (I4) {
          const uint32_t o = __shfl_sync(0xFFFFFFFFu, octet, par_octet);
          copy_async<16>(load_stage + 2 * ROWS * ROWB + lane * 16, at_octet(par_lane, o, 8 * PARB));
        }
      } else {
#pragma unroll 1
        for (int i = 0; i < COPIES; ++i) {
          const uint32_t o = __shfl_sync(0xFFFFFFFFu, octet, octet_of(i));
          const bool on = (__shfl_sync(0xFFFFFFFFu, seen8, octet_of(i)) >> ((i * RPC + lane / Gm::CHUNKS) % 8)) & 1;
          copy16_async_or_zero(load_stage + dst_of(i), at_octet(k_lane, o, BYTES) + within(i), on);
          copy16_async_or_zero(load_stage + ROWS * ROWB + dst_of(i), at_octet(v_lane, o, BYTES) + within(i), on);
        }
        if constexpr (I4) {
          const uint32_t o = __shfl_sync(0xFFFFFFFFu, octet, par_octet);
          const bool on = __shfl_sync(0xFFFFFFFFu, seen8, par_octet) != 0;
          copy16_async_or_zero(load_stage + 2 * ROWS * ROWB + lane * 16, at_octet(par_lane, o, 8 * PARB), on);
        }
      }
    }
    copies_commit();
    load_stage = load_stage == ring + (NST - 1) * Gm::STAGE ? ring : load_stage + Gm::STAGE;
  };
  look_up();
  for (int i = 0; i < NST - 1; ++i) {
    copy_tile();
    look_up();
  }

  // ---- a context's state ----
  uint32_t qf[KS][NT][2];
  // of each column: the maximum (base 2), the score (before its factor) that moves it, the sums
  float m_run[NT][2], top[NT][2], l_run[NT][2], oacc[KS][NT][4];
  // 4-bit rows: sums of q, of the weights times the values at from_code (0, 15 in odd rows),
  // +-1 / R (- in odd rows), and the scale that moves an R
  [[maybe_unused]] float qsum[GRP][NT][2], mids[GRP][NT][2], rinv[NT][2], vtop;
  [[maybe_unused]] float wsum[GRP][NT][2];  // CENTRED: sums of the second product's weights
  [[maybe_unused]] const float sign = qr & 1 ? -1.f : 1.f, from_code = CENTRED ? 7.5f : (qr & 1 ? 15.f : 0.f);
  float qk_mult = fmaxf(p.scale_log2, kLeastInvR);  // 0 would make NaN of a score of -infinity
  const auto context_row = [&]() { return static_cast<int64_t>(at_s) * p.qlen * p.Hq + head * p.G; };
  const auto start = [&]() {
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      m_run[nt][0] = m_run[nt][1] = kLeastMax;
      top[nt][0] = top[nt][1] = -CUDART_INF_F;
      l_run[nt][0] = l_run[nt][1] = 0.f;
#pragma unroll
      for (int mt = 0; mt < KS; ++mt) oacc[mt][nt][0] = oacc[mt][nt][1] = oacc[mt][nt][2] = oacc[mt][nt][3] = 0.f;
    }
    const int q_type = p.q_bf16 ? kBF16 : kF16;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
      const bool on = nt * 8 + qr < ncol;
      const uint32_t* row = static_cast<const uint32_t*>(p.q) + (context_row() + col_row[nt * 8 + qr]) * (D / 2);
      if constexpr (I4) {
        // the lane's channels of every 32: eight from 8 qc on, in their order
#pragma unroll
        for (int j = 0; j < KS; j += 2) {
          uint4 a = make_uint4(0u, 0u, 0u, 0u);
          if (on) a = load_written(reinterpret_cast<const uint4*>(row) + 2 * j + qc);
          qf[j][nt][0] = a.x, qf[j][nt][1] = a.y, qf[j + 1][nt][0] = a.z, qf[j + 1][nt][1] = a.w;
        }
      } else if constexpr (KV == kE4M3) {
        // k order of the widened fragments: 4 qc .. 4 qc + 3 of each 16
#pragma unroll
        for (int j = 0; j < KS; ++j) {
          const uint2 w = on ? load_written(reinterpret_cast<const uint2*>(row) + 4 * j + qc) : make_uint2(0u, 0u);
          qf[j][nt][0] = w.x, qf[j][nt][1] = w.y;
        }
      } else {
#pragma unroll
        for (int j = 0; j < KS; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i) qf[j][nt][i] = (on ? load_written(row + 8 * j + 4 * i + qc) : 0u) ^ (p.negative ? 0x80008000u : 0u);
      }
    }
    if constexpr (KV == kE4M3 || I4) {
      // scaled by a power of two that puts the context's largest |q| in [2^14, 2^15) and
      // rounded to f16 (f16 queries over E4M3 rows are taken as they are)
      int e = 0;
      if (I4 || p.q_bf16) {
        uint32_t most = 0;  // bits of the largest |q|, of both halves
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < KS; ++j) most = __vmaxu2(most, __vmaxu2(qf[j][nt][0] & 0x7FFF7FFFu, qf[j][nt][1] & 0x7FFF7FFFu));
        const uint32_t inf = p.q_bf16 ? 0x7F80u : 0x7C00u;
        if (max(most & 0xFFFFu, most >> 16) >= inf) {  // the largest finite one: an infinite query is its own row's matter
          most = 0;
#pragma unroll
          for (int nt = 0; nt < NT; ++nt)
#pragma unroll
            for (int j = 0; j < KS; ++j)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                const uint32_t lo = qf[j][nt][i] & 0x7FFFu, hi = qf[j][nt][i] >> 16 & 0x7FFFu;
                most = max(most, max(lo < inf ? lo : 0u, hi < inf ? hi : 0u));
              }
        }
        const float qmax = widen16(__reduce_max_sync(0xFFFFFFFFu, max(most & 0xFFFFu, most >> 16)), q_type);
        if (qmax > 0.f) {
          int ex;
          frexpf(qmax, &ex);
          e = min(15 - ex, 126);
        }
      }
      const float mul = ldexpf(p.negative ? -1.f : 1.f, e);
      qk_mult = fmaxf(ldexpf(p.scale_log2 * p.kv_scale, (I4 ? 24 : 0) - e), kLeastInvR);
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        if (!I4 && !p.q_bf16) {
#pragma unroll
          for (int j = 0; j < KS; ++j)
#pragma unroll
            for (int i = 0; i < 2; ++i) qf[j][nt][i] ^= p.negative ? 0x80008000u : 0u;
          continue;
        }
        [[maybe_unused]] float sum[GRP] = {};
#pragma unroll
        for (int j = 0; j < KS; ++j)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const uint32_t w = qf[j][nt][i];
            const float a = widen16(w & 0xFFFFu, q_type) * mul, b = widen16(w >> 16, q_type) * mul;
            const float part = I4 && i == 1 ? 0.0625f : 1.f;  // codes 16 times as large
            if constexpr (I4) sum[j / 4] += a + b;
            qf[j][nt][i] = pack2<false>(a * part, b * part);
          }
        if constexpr (I4) {
#pragma unroll
          for (int g = 0; g < GRP; ++g) {
            sum[g] += __shfl_xor_sync(0xFFFFFFFFu, sum[g], 1);
            sum[g] += __shfl_xor_sync(0xFFFFFFFFu, sum[g], 2);
            qsum[g][nt][0] = __shfl_sync(0xFFFFFFFFu, sum[g], 8 * qc) * kCodeUnit;
            qsum[g][nt][1] = __shfl_sync(0xFFFFFFFFu, sum[g], 8 * qc + 4) * kCodeUnit;
            mids[g][nt][0] = mids[g][nt][1] = 0.f;
            wsum[g][nt][0] = wsum[g][nt][1] = 0.f;
          }
          rinv[nt][0] = rinv[nt][1] = kFlatMostInvR * sign;
          vtop = kScaleTop / kFlatMostInvR;
        }
      }
    }
  };

  // The warp leaves a context of length L: `whole` if it had all of its tiles.
  const auto leave = [&](int L, bool whole, float* piece_o, float* piece_ml) {
    const auto over_rows = [](float x) {  // sum over the lanes of one column
#pragma unroll
      for (int o = 4; o <= 16; o <<= 1) x += __shfl_xor_sync(0xFFFFFFFFu, x, o);
      return x;
    };
#pragma unroll
    for (int nt = 0; nt < NT; ++nt) {
#pragma unroll
      for (int c2 = 0; c2 < 2; ++c2) {
        const int n = nt * 8 + 2 * qc + c2;
        const bool on = n < ncol;
        const float l = over_rows(l_run[nt][c2]);
        // only a token that sees nothing is 0: a NaN among its scores, or scores that are
        // all -infinity, have made l NaN or 0
        const float inv = L - p.qlen + col_token[nt * 8 + 2 * qc + c2] >= 0 ? 1.f / l : 0.f;
        const int64_t row = context_row() + col_row[nt * 8 + 2 * qc + c2];
        if (!whole && on && qr == 0) {
          *reinterpret_cast<float2*>(piece_ml + 2 * n) = make_float2(m_run[nt][c2], l);
        }
        if constexpr (I4) {
          const float R = rcp(fabsf(rinv[nt][c2]));
#pragma unroll
          for (int g = 0; g < GRP; ++g) {
            float b = over_rows(mids[g][nt][c2]);
            if constexpr (CENTRED) b = fmaf(over_rows(wsum[g][nt][c2]) * -from_code, R, b);
#pragma unroll
            for (int half = 0; half < 2; ++half) {  // 32 channels
              float v[4];  // channels 8 (qr / 2) + qr % 2 + 2 k
#pragma unroll
              for (int k = 0; k < 4; ++k)
                v[k] = fmaf(oacc[4 * g + k][nt][c2 + 2 * half] * ((k & 1 ? 1.f / 16.f : 1.f) / kCodeUnit), R, b);
              // lanes of neighbouring rows exchange two each, so that each has four in a row
              const bool odd = qr & 1;
              const float x = __shfl_xor_sync(0xFFFFFFFFu, odd ? v[0] : v[2], 4);
              const float y = __shfl_xor_sync(0xFFFFFFFFu, odd ? v[1] : v[3], 4);
              const float o[4] = {odd ? x : v[0], odd ? v[2] : x, odd ? y : v[1], odd ? v[3] : y};
              const int d = 64 * g + 32 * half + 4 * qr;
              if (!on) continue;
              if (whole) {
                const uint2 w = p.q_bf16 ? make_uint2(pack2<true>(o[0] * inv, o[1] * inv), pack2<true>(o[2] * inv, o[3] * inv))
                                         : make_uint2(pack2<false>(o[0] * inv, o[1] * inv), pack2<false>(o[2] * inv, o[3] * inv));
                static_cast<uint2*>(p.out)[(row * D + d) / 4] = w;
              } else {
                *reinterpret_cast<float4*>(piece_o + n * D + d) = make_float4(o[0], o[1], o[2], o[3]);
              }
            }
          }
        } else {
          const float mult = (KV == kE4M3 ? p.kv_scale : 1.f) * (whole ? inv : 1.f);
#pragma unroll
          for (int mt = 0; mt < KS; ++mt) {
            // channels qr and qr + 8 of 16: lanes of neighbouring rows exchange one each, so
            // that each has a pair
            const float v0 = oacc[mt][nt][c2] * mult, v1 = oacc[mt][nt][c2 + 2] * mult;
            const bool odd = qr & 1;
            const float got = __shfl_xor_sync(0xFFFFFFFFu, odd ? v0 : v1, 4);
            const float a = odd ? got : v0, b = odd ? v1 : got;
            const int d = 16 * mt + (odd ? 7 + qr : qr);
            if (!on) continue;
            if (whole)
              static_cast<uint32_t*>(p.out)[(row * D + d) / 2] = p.q_bf16 ? pack2<true>(a, b) : pack2<false>(a, b);
            else
              *reinterpret_cast<float2*>(piece_o + n * D + d) = make_float2(a, b);
          }
        }
      }
    }
  };

  // ---- SUB x 16 tokens from token pos on, rows `row` on of the stage.  MASK: some query
  // does not see all of them ----
  const auto attend = [&](auto mask, uint32_t st, int row, [[maybe_unused]] int pos, [[maybe_unused]] int L) {
    constexpr bool MASK = decltype(mask)::value;
    const uint32_t ks = st + row * ROWB, vs = ks + ROWS * ROWB;
    [[maybe_unused]] const uint32_t kp = st + 2 * ROWS * ROWB + row * PARB, vp = kp + ROWS * PARB;
    float sv[SUB][NT][4];
    // ---- scores ----
#pragma unroll
    for (int u = 0; u < SUB; ++u) {
      if constexpr (I4) {
        float acc[GRP][NT][4];
        const int r = 16 * u + (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
        for (int g = 0; g < GRP; ++g) {
          uint32_t R[4];  // rows qr and qr + 8, channels 8 qc on of 32, then of the next 32
          ldsm_x4(ks + Gm::chunk(r, 2 * g + (lane >> 4)), R[0], R[1], R[2], R[3]);
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t xa[4], xb[4];
            codes_of(R[2 * h], xa);
            codes_of(R[2 * h + 1], xb);
#pragma unroll
            for (int k = 0; k < 4; k += 2) {
              const uint32_t f[4] = {xa[k], xb[k], xa[k + 1], xb[k + 1]};
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                const uint32_t(&b)[2] = qf[4 * g + 2 * h + k / 2][nt];
                if (h == 0 && k == 0)
                  mma16816_zero(acc[g][nt], f, b[0], b[1]);
                else
                  mma16816<false>(acc[g][nt], f, b[0], b[1]);
              }
            }
          }
        }
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t par[2];
          if constexpr (GRP == 2) {
            const uint2 w = load8_shared(kp + (16 * u + qr + 8 * i) * PARB);
            par[0] = w.x, par[1] = w.y;
          } else {
            par[0] = load4_shared(kp + (16 * u + qr + 8 * i) * PARB);
          }
#pragma unroll
          for (int g = 0; g < GRP; ++g) {
            const uint32_t w = par[g];
            const float scale = bf16_low(w), low = bf16_high(w);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt)
#pragma unroll
              for (int c2 = 0; c2 < 2; ++c2) {
                const float t = g == 0 ? low * qsum[g][nt][c2] : fmaf(low, qsum[g][nt][c2], sv[u][nt][2 * i + c2]);
                sv[u][nt][2 * i + c2] = fmaf(acc[g][nt][2 * i + c2], scale, t);
              }
          }
        }
      } else {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) sv[u][nt][0] = sv[u][nt][1] = sv[u][nt][2] = sv[u][nt][3] = 0.f;
        if constexpr (KV == kE4M3) {
          const int r = 16 * u + tok_perm((lane & 7) + ((lane >> 3) & 1) * 8);
#pragma unroll
          for (int j = 0; j < KS; j += 2) {
            uint32_t R[4];
            ldsm_x4(ks + Gm::chunk(r, j + (lane >> 4)), R[0], R[1], R[2], R[3]);
#pragma unroll
            for (int kk = 0; kk < 2; ++kk) {
              uint32_t a[4];
              e4m3x4_to_f16x2x2(R[2 * kk], a[0], a[2]);
              e4m3x4_to_f16x2x2(R[2 * kk + 1], a[1], a[3]);
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma16816<false>(sv[u][nt], a, qf[j + kk][nt][0], qf[j + kk][nt][1]);
            }
          }
        } else {
          const int r = 16 * u + (lane & 7) + ((lane >> 3) & 1) * 8;
#pragma unroll
          for (int j = 0; j < KS; ++j) {
            uint32_t a[4];
            ldsm_x4(ks + Gm::chunk(r, 2 * j + (lane >> 4)), a[0], a[1], a[2], a[3]);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816<BF>(sv[u][nt], a, qf[j][nt][0], qf[j][nt][1]);
          }
        }
      }
    }
    // 4-bit rows: the parameters of token tok's row at par
    [[maybe_unused]] const auto params_of = [](uint32_t par, int tok, uint32_t (&w)[2]) {
      if constexpr (GRP == 2) {
        const uint2 v = load8_shared(par + tok * PARB);
        w[0] = v.x, w[1] = v.y;
      } else {
        w[0] = load4_shared(par + tok * PARB);
      }
    };
    // hidden: bit 2 u + i, token tok(i) of part u is not seen by the column
    [[maybe_unused]] uint32_t hidden[NT][2];
    if constexpr (MASK) {
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int c2 = 0; c2 < 2; ++c2) {
          const int P = L - p.qlen + col_token[nt * 8 + 2 * qc + c2];
          const uint32_t bits = seen_bits(pos, P + 1, window_low(p.window, P), p.sinks);
          hidden[nt][c2] = 0;
#pragma unroll
          for (int u = 0; u < SUB; ++u)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
              // the token (of 16) of accumulator row qr + 8 i
              const int tok = 16 * u + (KV == kE4M3 ? tok_perm(qr + 8 * i) : qr + 8 * i);
              if (!((bits >> tok) & 1)) {
                hidden[nt][c2] |= 1u << (2 * u + i);
                sv[u][nt][2 * i + c2] = -CUDART_INF_F;
              }
            }
        }
    }
    // ---- online softmax: the maximum moves when a score passes it by kHeadroom ----
    bool lift = false;
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c2 = 0; c2 < 2; ++c2) {
        float most = fmaxf(sv[0][nt][c2], sv[0][nt][c2 + 2]);
        if constexpr (SUB == 2) most = max3(most, sv[SUB - 1][nt][c2], sv[SUB - 1][nt][c2 + 2]);
        lift |= most > top[nt][c2];
      }
    // 4-bit rows: the largest scale of V's tokens qr + 8 i of part u, seen or not (their
    // parameters are read again where they are used: held until then they would take eight
    // registers)
    [[maybe_unused]] float largest = 0.f;
    if constexpr (I4) {
#pragma unroll
      for (int u = 0; u < SUB; ++u)
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          uint32_t w[2];
          params_of(vp, 16 * u + qr + 8 * i, w);
          if constexpr (GRP == 2)
            largest = max3(largest, fabsf(bf16_low(w[0])), fabsf(bf16_low(w[1])));
          else
            largest = fmaxf(largest, fabsf(bf16_low(w[0])));
        }
      lift |= largest > vtop;
    }
    if (__any_sync(0xFFFFFFFFu, lift)) {
      // each column by its own scores and the scales that it sees: the bits of a query's
      // output do not depend on the columns beside it (but through the power of two that
      // start() gives them all) nor on rows that it does not see, where anything may lie
      if constexpr (I4 && !MASK) {
#pragma unroll
        for (int o = 4; o <= 16; o <<= 1) largest = fmaxf(largest, __shfl_xor_sync(0xFFFFFFFFu, largest, o));
      }
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float alpha[2];
#pragma unroll
        for (int c2 = 0; c2 < 2; ++c2) {
          float mx = -CUDART_INF_F;
#pragma unroll
          for (int u = 0; u < SUB; ++u) mx = fmaxf(mx, fmaxf(sv[u][nt][c2], sv[u][nt][c2 + 2]));
#pragma unroll
          for (int o = 4; o <= 16; o <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xFFFFFFFFu, mx, o));
          const bool moves = mx > top[nt][c2];
          mx = moves ? fmaxf(mx * qk_mult, kLeastMax) : m_run[nt][c2];
          if (moves) top[nt][c2] = (mx + kHeadroom) / qk_mult;
          alpha[c2] = ex2(m_run[nt][c2] - mx);
          l_run[nt][c2] *= alpha[c2];
          if constexpr (I4) {
#pragma unroll
            for (int g = 0; g < GRP; ++g) mids[g][nt][c2] *= alpha[c2];
            float most = -CUDART_INF_F;  // of log2(p scale) + maximum
            float widest = MASK ? 0.f : largest;  // scale that the column sees
#pragma unroll
            for (int u = 0; u < SUB; ++u)
#pragma unroll
              for (int i = 0; i < 2; ++i) {
                uint32_t w[2];
                params_of(vp, 16 * u + qr + 8 * i, w);
#pragma unroll
                for (int g = 0; g < GRP; ++g) {
                  const float scale = fabsf(bf16_low(w[g]));
                  most = fmaxf(most, sv[u][nt][2 * i + c2] * qk_mult + lg2(scale));
                  if constexpr (MASK) widest = (hidden[nt][c2] >> (2 * u + i)) & 1 ? widest : fmaxf(widest, scale);
                }
              }
#pragma unroll
            for (int o = 4; o <= 16; o <<= 1) {
              most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, o));
              if constexpr (MASK) widest = fmaxf(widest, __shfl_xor_sync(0xFFFFFFFFu, widest, o));
            }
            // as the maximum rises the sums can stay what they are: R falls instead
            const float old = fabsf(rinv[nt][c2]), keep = old * ex2(mx - m_run[nt][c2]);
            const float now = fminf(fmaxf(fminf(keep, ex2(mx - most + kProductStart)), kLeastInvR), kFlatMostInvR);
            if (moves || widest * old > kScaleTop) {
              rinv[nt][c2] = now * sign;
              alpha[c2] = now == keep ? 1.f : now * alpha[c2] * rcp(old);
            } else {
              alpha[c2] = 1.f;
            }
          }
          m_run[nt][c2] = mx;
          if constexpr (CENTRED) {
#pragma unroll
            for (int g = 0; g < GRP; ++g) wsum[g][nt][c2] *= alpha[c2];
          }
        }
#pragma unroll
        for (int mt = 0; mt < KS; ++mt) {
          oacc[mt][nt][0] *= alpha[0];
          oacc[mt][nt][1] *= alpha[1];
          oacc[mt][nt][2] *= alpha[0];
          oacc[mt][nt][3] *= alpha[1];
        }
      }
      if constexpr (I4) {
        float most = 0.f;
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) most = fmaxf(most, fmaxf(fabsf(rinv[nt][0]), fabsf(rinv[nt][1])));
        vtop = kScaleTop * rcp(most);
      }
    }
#pragma unroll
    for (int nt = 0; nt < NT; ++nt)
#pragma unroll
      for (int c2 = 0; c2 < 2; ++c2) {
        const float m = m_run[nt][c2];
#pragma unroll
        for (int u = 0; u < SUB; ++u) {
          sv[u][nt][c2] = ex2(fmaf(sv[u][nt][c2], qk_mult, -m));
          sv[u][nt][c2 + 2] = ex2(fmaf(sv[u][nt][c2 + 2], qk_mult, -m));
          l_run[nt][c2] += sv[u][nt][c2] + sv[u][nt][c2 + 2];
        }
      }
    // ---- O^T += V^T P^T ----
#pragma unroll
    for (int u = 0; u < SUB; ++u) {
      if constexpr (I4) {
        uint32_t par[2][2];
        params_of(vp, 16 * u + qr, par[0]);
        params_of(vp, 16 * u + qr + 8, par[1]);
#pragma unroll
        for (int g = 0; g < GRP; ++g) {
          uint32_t pb[NT][2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float scale = bf16_low(par[i][g]), mid = fmaf(from_code, scale, bf16_high(par[i][g]));
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) {
              float w[2];
#pragma unroll
              for (int c2 = 0; c2 < 2; ++c2) {
                // a token that is not seen adds nothing, whatever its parameters
                bool off = false;
                if constexpr (MASK) off = (hidden[nt][c2] >> (2 * u + i)) & 1;
                w[c2] = off ? 0.f : sv[u][nt][2 * i + c2] * rinv[nt][c2] * scale;
                mids[g][nt][c2] = off ? mids[g][nt][c2] : fmaf(sv[u][nt][2 * i + c2], mid, mids[g][nt][c2]);
              }
              const uint32_t pair = pack2<false>(w[0], w[1]);
              if constexpr (CENTRED) add_pair(wsum[g][nt], pair);
              pb[nt][i] = movm_t(pair);
            }
          }
          // four codes of tokens 2 qc (low half) and 2 qc + 1, then of 8 on: of the group's
          // first 32 channels 8 (qr / 2) + qr % 2 + 2 k, and of its last
          uint32_t R[4], xa[4], xb[4], ya[4], yb[4];
          ldsm_x4_t(vs + Gm::chunk(16 * u + (lane & 7) + (lane >> 4) * 8, 2 * g + ((lane >> 3) & 1)), R[0], R[1], R[2], R[3]);
          flipped_codes_of(R[0], p.flip, xa);
          flipped_codes_of(R[1], p.flip, ya);
          flipped_codes_of(R[2], p.flip, xb);
          flipped_codes_of(R[3], p.flip, yb);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t f[4] = {xa[k], ya[k], xb[k], yb[k]};
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma16816<false>(oacc[4 * g + k][nt], f, pb[nt][0], pb[nt][1]);
          }
        }
      } else {
        uint32_t pb[NT][2];
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          pb[nt][0] = movm_t(pack2<BF>(sv[u][nt][0], sv[u][nt][1]));
          pb[nt][1] = movm_t(pack2<BF>(sv[u][nt][2], sv[u][nt][3]));
        }
        // adds the part's V rows of `keep` (bits) times their weights: mma(sums, V, column tile)
        const auto add_pv = [&](uint32_t keep, auto mma) {
          if constexpr (KV == kE4M3) {
            uint32_t bytes = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) bytes |= (keep >> (4 * qc + i)) & 1 ? 0xFFu << (8 * i) : 0u;
#pragma unroll
            for (int j = 0; j < KS; j += 2) {
              uint32_t R[4];
              ldsm_b8_x2_t(vs + Gm::chunk(16 * u + (lane & 15), j + (lane >> 4)), R[0], R[1], R[2], R[3]);
#pragma unroll
              for (int kk = 0; kk < 2; ++kk) {
                uint32_t a[4];
                e4m3x4_to_f16x2x2(R[2 * kk] & bytes, a[0], a[2]);
                e4m3x4_to_f16x2x2(R[2 * kk + 1] & bytes, a[1], a[3]);
#pragma unroll
                for (int nt = 0; nt < NT; ++nt) mma(oacc[j + kk][nt], a, nt);
              }
            }
          } else {
            const int r = 16 * u + (lane & 7) + (lane >> 4) * 8;
            const uint32_t two = keep >> (2 * qc);
            const uint32_t lo = (two & 1 ? 0xFFFFu : 0u) | (two & 2 ? 0xFFFF0000u : 0u);
            const uint32_t hi = (two & 256 ? 0xFFFFu : 0u) | (two & 512 ? 0xFFFF0000u : 0u);
#pragma unroll
            for (int mt = 0; mt < KS; ++mt) {
              uint32_t a[4];
              ldsm_x4_t(vs + Gm::chunk(r, 2 * mt + ((lane >> 3) & 1)), a[0], a[1], a[2], a[3]);
              a[0] &= lo;
              a[1] &= lo;
              a[2] &= hi;
              a[3] &= hi;
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) mma(oacc[mt][nt], a, nt);
            }
          }
        };
        const auto all_columns = [&](float (&o)[4], const uint32_t (&a)[4], int nt) { mma16816<BF>(o, a, pb[nt][0], pb[nt][1]); };
        // rows that only some of the new tokens see: a NaN or an infinity there
        // would reach the others through their weights of 0
        bool apart = false;
        if constexpr (MASK) {
          const uint32_t some = (seen_bits(pos, L, window_low(p.window, L - p.qlen), p.sinks) &
                                 ~seen_bits(pos, L - p.qlen + 1, window_low(p.window, L - 1), p.sinks)) >> (16 * u);
          if (p.qlen > 1 && (some & 0xFFFFu)) {
            for (int i = lane; i < 16 * Gm::CHUNKS; i += 32) {
              const int r = i / Gm::CHUNKS;
              if (!((some >> r) & 1)) continue;
              uint32_t w[4];
              load16_shared(vs + Gm::chunk(16 * u + r, i % Gm::CHUNKS), w);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                // a field of ones in the exponent (in all seven bits of an E4M3 code)
                // plus one carries into the bit above it
                if constexpr (KV == kE4M3) apart |= (((w[k] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0;
                if constexpr (KV == kBF16) apart |= (((w[k] & 0x7F807F80u) + 0x00800080u) & 0x80008000u) != 0;
                if constexpr (KV == kF16) apart |= (((w[k] & 0x7C007C00u) + 0x04000400u) & 0x80008000u) != 0;
              }
            }
          }
          apart = __any_sync(0xFFFFFFFFu, apart);
        }
        if (!apart) {
          add_pv(0xFFFFu, all_columns);
        } else {
          for (int j = 0; j < p.qlen; ++j) {  // one new token at a time: the rows it sees, to its own columns
            const int P = L - p.qlen + j;
            const uint32_t keep = seen_bits(pos, P + 1, window_low(p.window, P), p.sinks) >> (16 * u) & 0xFFFFu;
            if (keep == 0) continue;
            add_pv(keep, [&](float (&o)[4], const uint32_t (&a)[4], int nt) {
              float t[4] = {o[0], o[1], o[2], o[3]};
              mma16816<BF>(t, a, pb[nt][0], pb[nt][1]);
#pragma unroll
              for (int e = 0; e < 4; ++e) o[e] = col_token[nt * 8 + 2 * qc + (e & 1)] == j ? t[e] : o[e];
            });
          }
        }
      }
    }
  };

  // ---- the contexts of the part ----
  [[maybe_unused]] constexpr int PIECE_STRIDE = NST * Gm::STAGE;  // a warp's piece takes the place of its ring
  static_assert(PIECE_STRIDE >= NG * (D + 2) * 4);
  uint32_t stage = ring;
  bool first = true;
#pragma unroll 1
  for (int n = to_come; n < places; n += p.gap) {  // n: the place of the tile
    int whole_lo, whole_hi;
    whole_tiles(c, whole_lo, whole_hi);
    const int from = at_t, to = min(c.tiles, from + places - n);
    start();
#pragma unroll 1
    for (int t = from; t < to; ++t) {
      copies_wait<NST - 2>();
      __syncwarp();  // the other lanes' copies too; and every lane has read the tile before, whose stage is filled next
      copy_tile();
      look_up();
      const bool whole_tile = t >= whole_lo && t < whole_hi;
#pragma unroll 1
      for (int row = 0; row < ROWS; row += 16 * SUB) {
        const int pos = c.token(t) + row;
        if (whole_tile)
          attend(std::false_type{}, stage, row, pos, c.L);
        else if (seen_bits(pos, c.L, window_low(p.window, c.L - p.qlen), p.sinks) & ALL)
          attend(std::true_type{}, stage, row, pos, c.L);
      }
      stage = stage == ring + (NST - 1) * Gm::STAGE ? ring : stage + Gm::STAGE;
    }
    // pieces lie at slot 2 i of warp i where the context came first, else at 2 i + 1
    const int slot = 2 * id + (first ? 0 : 1);
    n += to - from;
    if (!SHARED && from == 0 && lane == 0 && (p.by_context || to < c.tiles)) {
      const int64_t last = u0 + n - 1 + (c.tiles - to);  // the place of the context's last tile
      const int pieces = to == c.tiles ? 0 : static_cast<int>(last / part) - id / p.heads + 1, context = at_s * p.heads + head;
      p.ws_joins[p.by_context ? context : id] = make_int4(context, pieces, slot, 0);
    }
    const bool whole = from == 0 && to == c.tiles;
    if constexpr (!SHARED) {
      leave(c.L, whole, p.ws_o + static_cast<int64_t>(slot) * kFlatColumns * D, p.ws_ml + static_cast<int64_t>(slot) * kFlatColumns * 2);
    } else {
      copies_wait<0>();
      __syncwarp();
      float* piece = reinterpret_cast<float*>(smem + warp * PIECE_STRIDE);
      leave(c.L, whole, piece, piece + NG * D);
      break;
    }
    first = false;
    at_t = 0;
    if (++at_s < p.S) c = Span(p, load_written(p.context_lens + at_s));
  }
  copies_wait<0>();
  if constexpr (SHARED) {
    // ---- the cluster's pieces: first each CTA's own, into its warp 0's, then the CTAs' ----
    const int share = shared_tiles(c.tiles, p.cluster);
    const int pieces = (c.tiles + share - 1) / share, own = min(pieces - rank * kFlatWarps, kFlatWarps);
    if (pieces == 1) return;
    __syncthreads();
    constexpr int LANES = D / 4;
    const int count = (pieces + kFlatWarps - 1) / kFlatWarps;  // of CTAs
    const uint32_t area = smem_u32(smem);
    const auto join = [&](int idx, int num, auto at) {  // elements 4 idx .. 4 idx + 3 of the pieces at(0) .. at(num - 1)
      const int n = idx / LANES, col = idx % LANES;
      FlatSums sums;
#pragma unroll 4
      for (int i = 0; i < num; ++i) {
        const uint32_t from = at(i);
        sums.add(load_peer4(from + (n * D + 4 * col) * 4), load_peer2(from + (NG * D + 2 * n) * 4));
      }
      return sums;
    };
    constexpr int EACH = (NG * LANES + kFlatThreads - 1) / kFlatThreads;
    FlatSums mine[EACH];
    if (own > 1) {
#pragma unroll
      for (int e = 0; e < EACH; ++e)
        if (tid + e * kFlatThreads < ncol * LANES)
          mine[e] = join(tid + e * kFlatThreads, own, [&](int i) { return area + i * PIECE_STRIDE; });
      __syncthreads();
#pragma unroll
      for (int e = 0; e < EACH; ++e) {
        const int idx = tid + e * kFlatThreads, n = idx / LANES;
        if (idx >= ncol * LANES) break;
        float* piece = reinterpret_cast<float*>(smem);
        reinterpret_cast<float4*>(piece)[idx] = mine[e].o;
        if (idx % LANES == 0) reinterpret_cast<float2*>(piece + NG * D)[n] = make_float2(mine[e].m, mine[e].l);
      }
    }
    cluster_sync();
    for (int idx = rank * kFlatThreads + tid; idx < ncol * LANES; idx += p.cluster * kFlatThreads) {
      const FlatSums sums = join(idx, count, [&](int i) { return peer_shared(area, i); });
      const int n = idx / LANES;
      const float inv = c.L - p.qlen + col_token[n] >= 0 ? 1.f / sums.l : 0.f;
      sums.store(p, (static_cast<int64_t>(at_s) * p.qlen * p.Hq + head * p.G + col_row[n]) * LANES + idx % LANES, inv);
    }
    cluster_sync();  // no CTA leaves while its piece is read
  }
}

// Joins the pieces of one context: M = max m_i, and for every query column
// out = sum_i o_i 2^(m_i - M) / sum_i l_i 2^(m_i - M), in the order of the context.
// D / 4 lanes read a piece's column, four channels each.  The CTA's groups of so many
// lanes take the columns, several groups a column where there are more of them
// (every so-manieth piece each, added in their order); with APART, for few
// contexts of many pieces, a CTA takes one column alone.
constexpr int kJoinThreads = 256;

template <int D, bool APART>
__global__ void __launch_bounds__(kJoinThreads) flat_join_kernel(const FlatParams p) {
  constexpr int LANES = D / 4, GROUPS = kJoinThreads / LANES;
  pdl_enter();
  const int ncol = p.G * p.qlen;
  const int4 join = load_written(p.ws_joins + (APART ? blockIdx.x / ncol : blockIdx.x));
  if (join.y == 0) return;
  const int grp = threadIdx.x / LANES, q = threadIdx.x % LANES;
  __shared__ float4 sums[GROUPS][LANES];
  __shared__ float2 ml[GROUPS];
  const int s = join.x / p.heads, h = join.x % p.heads;
  const int L = min(max(load_written(p.context_lens + s), 0), p.maxB << p.bs_log2);
  int share = 1;  // groups of a column
  if (APART) share = GROUPS;
  else while (2 * share * ncol <= GROUPS) share *= 2;
  const int sub = grp % share;
#pragma unroll 1
  for (int n0 = APART ? blockIdx.x % ncol : 0; n0 < ncol; n0 += APART ? ncol : GROUPS / share) {
    const int n = n0 + grp / share;
    FlatSums own;
    if (n < ncol) {
#pragma unroll 4
      for (int i = sub; i < join.y; i += share) {
        const int64_t piece = static_cast<int64_t>(i == 0 ? join.z : 2 * ((join.z >> 1) + i * p.heads)) * kFlatColumns + n;
        own.add(load_written(reinterpret_cast<const float4*>(p.ws_o + piece * D) + q),
                load_written(reinterpret_cast<const float2*>(p.ws_ml) + piece));
      }
    }
    if (share > 1) {
      __syncthreads();
      sums[grp][q] = own.o;
      if (q == 0) ml[grp] = make_float2(own.m, own.l);
      __syncthreads();
      if (sub == 0)
        for (int g = 1; g < min(share, join.y); ++g) own.add(sums[grp + g][q], ml[grp + g]);
    }
    if (n >= ncol || sub != 0) continue;
    const int j = n / p.G;
    const float inv = L - p.qlen + j >= 0 ? 1.f / own.l : 0.f;
    own.store(p, ((static_cast<int64_t>(s) * p.qlen + j) * p.Hq + h * p.G + n - j * p.G) * LANES + q, inv);
  }
}


constexpr int kFlatGap = 2;
constexpr int kFlatLeastPart = 3;

// CTAs of the clusters that share a context each, or 0: the line.  As many as have their
// places at once (clusters of four and eight need places near one another: an eighth is
// left free) and a tile each.  A warp's share of a context's tiles, of the longest one
// there may be, is then weighed against its part of the line, where what joining pieces
// costs is worth kLineTokens, and without a window contexts count as half as long as the
// table: the lengths are the device's.  A table far wider than its contexts so goes by the
// line (one context of 2000 4-bit tokens in one of 131072: 12.9 us, 9.2 where it is cut to
// the context; of 40000 and 131000 tokens 26.7 and 51).  (One context of 2000, 8000, 16000 4-bit tokens, 32/8 heads: 9.3, 14.1, 20.3 us
// by clusters of eight, 12.7, 15.9, 22.1 by the line; 16 of 16 to 4000 tokens by clusters
// of two 26.2, by the line 22.0.  A bf16 window of 1024 of 1, 16, 32 streams: 9.5, 14.3,
// 25.7 with eight, two, one CTA each, 12.2, 18.9, 31.6.  A window of 4096 of 20, 37, 75
// streams of two new tokens, 4-bit, 64 channels: 27.4, 28.5, 44.8 with two, two, one, by
// the line 25.0, 34.6, 49.2.)
// More contexts than places, through a window and so of much the same length: those of
// 16-bit caches, which memory bounds, go by a CTA each from half as many more on, as CTAs
// that end early make room for others (256 streams x 8 heads through 4096 tokens 521 us,
// by the line 545, through 1024 tokens 173 both, through 512 tokens 104 and 94; 40 x 8,
// little more than there are places, 131 and 108).  Narrower rows and more than eight
// columns stay on the line: 4-bit rows and twelve columns, bound by instructions (200 x 8,
// two tokens, 4-bit, window of 2048: 75 us by CTAs, 66 by the line; 100 x 8 of 12 columns,
// bf16, 64 channels, window of 1024: 55 and 50), and E4M3 rows, whose line is at the
// memory's rate too (256 x 8 through 4096 tokens 318 by CTAs and 321 by the line, through
// 1024 99 and 95; 128 x 8 through 4096 178 and 169; 200 x 8, two tokens, 2048, 139 and 140).
constexpr int kFlatMostCluster = 8;
constexpr int kLineTokens = 256;

template <int KV, int D, int NG>
int flat_cluster(const FlatParams& p) {
  constexpr int ROWS = flat_rows<KV, D>();
  const int64_t contexts = static_cast<int64_t>(p.S) * p.heads, places = static_cast<int64_t>(flat_min_ctas<KV, D, NG>()) * p.sms;
  int64_t tiles = ((static_cast<int64_t>(p.maxB) << p.bs_log2) + ROWS - 1) / ROWS;  // of a context at most
  if (p.window > 0)
    tiles = std::min(tiles, (static_cast<int64_t>(p.window) + p.qlen - 2) / ROWS + 2 + (static_cast<int64_t>(p.sinks) + ROWS - 1) / ROWS);
  if (contexts > places)
    return KV != kInt4 && KV != kE4M3 && NG == 8 && p.window >= 1024 && 2 * contexts >= 3 * places ? 1 : 0;
  int c = kFlatMostCluster;
  while (c > 1 && (contexts * c > (c > 2 ? places * 7 / 8 : places) || tiles <= c / 2 * kFlatWarps)) c /= 2;
  const int64_t share = (tiles + c * kFlatWarps - 1) / (c * kFlatWarps);
  const int64_t part = contexts * (tiles + kFlatGap) / (places * kFlatWarps) / (p.window > 0 ? 1 : 2);
  return share <= part + kLineTokens / ROWS ? c : 0;
}

template <int KV, int D, int NG, bool CENTRED>
cudaError_t launch_flat_one(FlatParams p, cudaStream_t st) {
  constexpr int smem = flat_smem<KV, D, NG>();
  const int64_t contexts = static_cast<int64_t>(p.S) * p.heads;
  cudaError_t e;
  p.cluster = flat_cluster<KV, D, NG>(p);
  if (p.cluster > 0) {
    auto kern = flat_kernel<KV, D, NG, CENTRED, true>;
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (e != cudaSuccess) return e;
    return launch_in_clusters(kern, static_cast<unsigned>(contexts * p.cluster), p.cluster, kFlatThreads, smem, st, p);
  }
  auto kern = flat_kernel<KV, D, NG, CENTRED, false>;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
  if (e != cudaSuccess) return e;
  // at least a part, with more CTAs than there are places if it has so many heads
  const int warps = flat_min_ctas<KV, D, NG>() * p.sms * kFlatWarps;
  p.nparts = std::max(1, warps / p.heads);
  const int ncta = (p.nparts * p.heads + kFlatWarps - 1) / kFlatWarps;
  // one part: nothing is cut, and there may be more heads than the workspace has joins
  p.by_context = p.nparts > 1 && contexts <= static_cast<int64_t>(p.nparts) * p.heads;
  p.gap = kFlatGap;
  p.least_part = kFlatLeastPart;
  e = launch_in_order(kern, static_cast<unsigned>(ncta), kFlatThreads, smem, st, p);
  return e == cudaSuccess ? launch_flat_join(p, D, st) : e;
}

// More than eight query columns are one context of 16, so that its rows are read and
// unpacked once; but where contexts of at most eight are no more than the SMs and would
// be shared by clusters, they are taken: the chains of a tile's instructions are
// shorter.  (Four drafts through a window of 2000, E4M3, 16/4 heads, of 1, 4, 19 streams:
// 11.7, 12.4, 19.2 us with 16 columns, 9.2, 10.8, 18.4 with twice eight; of 33, 264
// contexts of eight, 22.7 and 26.6.  One 4-bit context of 2000 tokens, 128/8 heads, 12.7
// and 9.6; four of 40000, on the line, 62 and 75.)
template <int KV, int D, bool CENTRED>
cudaError_t launch_flat_columns(const FlatParams& p, cudaStream_t st) {
  if (p.G * p.qlen <= 8) return launch_flat_one<KV, D, 8, CENTRED>(p, st);
  if (p.qlen <= 8) {
    int n = 8 / p.qlen;  // query heads of each
    while (p.G % n) --n;
    FlatParams few = p;
    few.head_div *= p.G / n;
    few.heads *= p.G / n;
    few.G = n;
    if (static_cast<int64_t>(p.S) * few.heads <= p.sms && flat_cluster<KV, D, 8>(few) > 0)
      return launch_flat_one<KV, D, 8, CENTRED>(few, st);
  }
  return launch_flat_one<KV, D, 16, CENTRED>(p, st);
}

template <int KV, bool CENTRED = false>
cudaError_t launch_flat_kv(const FlatParams& p, int D, cudaStream_t st) {
  return D == 64 ? launch_flat_columns<KV, 64, CENTRED>(p, st) : launch_flat_columns<KV, 128, CENTRED>(p, st);
}

}  // namespace pa
