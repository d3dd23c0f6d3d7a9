// norm_rope_cache: RMS norm of each query and key head, rotation by the
// token's position, K and V rows into the paged cache, in one pass.  32768
// tokens of 32 query and 8 K/V heads of 128 bf16 channels (805 MB): 126 us,
// 0.96 of the rate of a plain copy; 64 tokens: 3.4 us, launch and latency.
//
// Bound by memory: a token's heads are read once and written once, with some
// ten operations per element, so instructions have to be spared.  TPT threads
// take a token; groups of D / 8 lanes take a head each, eight channels per
// lane, so the head's mean square is a shuffle reduction over the group.  With
// pairs (i, i + rot / 2) a lane's eight channels are four neighbours of the
// first half and their four partners (two 8-byte accesses; rot / 2 is a
// multiple of 4), with pairs (2 i, 2 i + 1) eight neighbours (one 16-byte
// access): either way the rotation stays inside the lane, without the eight
// shuffles per head that partners in another lane would take.
//
// The rotation of a normed pair is linear in the raw pair (a, b):
//   y = inv (a (wa cos) - b (wb sin)),   z = inv (b (wb cos) + a (wa sin)),
// inv = rsqrt(mean x^2 + eps), so the weights and the token's cosines make
// four factors per pair that all the token's query heads share (and four that
// its key heads share): two products, two fused multiply-adds and two products
// with inv per pair and head.  (Partners in other lanes and factors made per
// head: 273 us; factors shared, heads loaded as they are used: 167; heads copied
// eight steps ahead: 134 with the 64 threads per token that took.)
#include "pa_launch.h"
#include "pa_pdl.cuh"
#include "pa_ptx.cuh"
#include "pa_row_quant.cuh"
#include "pagedattn.h"

namespace pa {

namespace {

constexpr int kNrThreads = 256;
constexpr int kAhead = 8;  // steps of a group's heads in flight

// Factors of the lane's four pairs.
struct PairFactors {
  float ac[4], as[4], bc[4], bs[4];  // wa cos, wa sin, wb cos, wb sin
};

template <int D, int KIND, bool BF16, bool INTER, int TPT>
__global__ void __launch_bounds__(kNrThreads) norm_rope_kernel(const NormRopeParams p) {
  constexpr int LPR = D / 8;         // lanes per head
  constexpr int GROUPS = TPT / LPR;  // heads at a time
  pdl_enter();
  const unsigned token = blockIdx.x * (kNrThreads / TPT) + threadIdx.x / TPT;
  if (token >= static_cast<unsigned>(p.T)) return;
  const int t = static_cast<int>(token);
  const int c = threadIdx.x % LPR, g = threadIdx.x % TPT / LPR;
  // this lane's pieces of four channels
  const int half = p.rot / 2;
  const bool paired = !INTER && c < p.rot / 8;
  const int pa = paired ? c : 2 * c, pb = paired ? c + half / 4 : 2 * c + 1;

  // The group's heads in order: nq steps of queries, nkv of keys, nkv of
  // values, copied ahead into a ring of kAhead steps in shared memory; a lane
  // reads back only its own copies, so no barrier is needed.
  const int nq = (p.Hq + GROUPS - 1) / GROUPS, nkv = (p.sink.Hkv + GROUPS - 1) / GROUPS;
  __shared__ __align__(16) uint8_t ring[kAhead * kNrThreads * 16];
  const uint32_t ring0 = smem_u32(ring) + threadIdx.x * 16;
  auto fetch = [&](int n) {  // one group of copies per step, empty ones too
    const uint16_t* row = nullptr;
    if (n < nq) {
      const int h = n * GROUPS + g;
      if (h < p.Hq) row = static_cast<const uint16_t*>(p.q) + t * p.q_stride + h * D;
    } else if (n < nq + nkv) {
      const int h = (n - nq) * GROUPS + g;
      if (h < p.sink.Hkv) row = static_cast<const uint16_t*>(p.key) + t * p.key_stride + h * D;
    } else {
      const int h = (n - nq - nkv) * GROUPS + g;
      if (h < p.sink.Hkv) row = static_cast<const uint16_t*>(p.value) + t * p.value_stride + h * D;
    }
    const uint32_t dst = ring0 + (n % kAhead) * kNrThreads * 16;
    if (row != nullptr) {
      if constexpr (INTER) {
        copy_async<16>(dst, row + 4 * pa);
      } else {
        copy_async<8>(dst, row + 4 * pa);
        copy_async<8>(dst + 8, row + 4 * pb);
      }
    }
    copies_commit();
  };
#pragma unroll
  for (int n = 0; n < kAhead; ++n) fetch(n);

  const int64_t slot = load_written(p.sink.slot_mapping + t);
  if (slot < 0) {  // padding token
    copies_wait<0>();
    return;
  }
  const bool in_pool = slot < p.sink.num_slots;
  const bool lead = threadIdx.x % TPT == 0;
  if (!in_pool && lead) atomicOr(p.sink.err, PA_DEVERR_SLOT);
  const int64_t row0 = in_pool ? row_index(p.sink, slot, 0) : 0;  // head h: row0 + (h << bs_log2)

  // cosine and sine of the lane's four pairs
  float cs[4], sn[4];
  bool turn[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    turn[i] = 4 * c + i < half;
    cs[i] = 1.f;
    sn[i] = 0.f;
  }
  if (p.rot > 0) {
    int64_t pos = load_written(p.positions + t);
    if (pos < 0 || pos >= p.num_positions) {
      if (lead) atomicOr(p.sink.err, PA_DEVERR_POSITION);
      pos = pos < 0 ? 0 : p.num_positions - 1;
    }
    const float* tab = p.cos_sin + pos * p.rot;
    if (p.rot == D && p.tab16) {  // whole rows, 16-byte aligned
      const float4 u = load_written(reinterpret_cast<const float4*>(tab) + c);
      const float4 v = load_written(reinterpret_cast<const float4*>(tab + D / 2) + c);
      cs[0] = u.x, cs[1] = u.y, cs[2] = u.z, cs[3] = u.w;
      sn[0] = v.x, sn[1] = v.y, sn[2] = v.z, sn[3] = v.w;
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (turn[i]) {
          cs[i] = load_written(tab + 4 * c + i);
          sn[i] = load_written(tab + half + 4 * c + i);
        }
    }
  }
  const bool norm = p.q_weight != nullptr;
  auto factors = [&](const void* weight) {
    float w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = 1.f;
    if (norm) widen8<BF16>(load_pieces<INTER>(static_cast<const uint16_t*>(weight), pa, pb), w);
    PairFactors f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float wa = w[INTER ? 2 * i : i], wb = w[INTER ? 2 * i + 1 : i + 4];
      f.ac[i] = wa * cs[i];
      f.as[i] = wa * sn[i];
      f.bc[i] = wb * cs[i];
      f.bs[i] = wb * sn[i];
    }
    return f;
  };
  // one head: norm and rotation in place
  auto turned = [&](float (&x)[8], const PairFactors& f) {
    float inv = 1.f;
    if (norm) {
      float ss = 0.f;
#pragma unroll
      for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
      for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
      inv = rsqrtf(ss * (1.f / D) + p.eps);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float& a = x[INTER ? 2 * i : i];
      float& b = x[INTER ? 2 * i + 1 : i + 4];
      const float y = fmaf(a, f.ac[i], -(b * f.bs[i])), z = fmaf(b, f.bc[i], a * f.as[i]);
      // channels that are not rotated take only their own value, which may be
      // infinite; their factors ac and bc are the weights
      a = (turn[i] ? y : a * f.ac[i]) * inv;
      b = (turn[i] ? z : b * f.bc[i]) * inv;
    }
  };
  const int Hkv = p.sink.Hkv;
  uint16_t* q_out = static_cast<uint16_t*>(p.q_out) + static_cast<int64_t>(t) * p.Hq * D;
  int n = 0;
  // the next `count` steps of the ring: work(head, values)
  auto steps = [&](int count, auto work) {
    for (int i = 0; i < count; ++i, ++n) {
      copies_wait<kAhead - 1>();  // all but the latest kAhead - 1 steps have landed
      uint32_t w[4];
      load16_shared(ring0 + (n % kAhead) * kNrThreads * 16, w);
      float x[8];
      widen8<BF16>(make_uint4(w[0], w[1], w[2], w[3]), x);
      fetch(n + kAhead);
      work(i * GROUPS + g, x);
    }
  };
  {
    const PairFactors f = factors(p.q_weight);
    steps(nq, [&](int h, float (&x)[8]) {
      turned(x, f);
      if (h < p.Hq) store_pieces<INTER>(q_out + h * D, pa, pb, narrow8<BF16>(x));
    });
  }
  {
    const PairFactors f = factors(p.k_weight);
    steps(nkv, [&](int h, float (&x)[8]) {
      turned(x, f);
      store_row<D, KIND, BF16, INTER>(p.sink, false, row0 + (static_cast<int64_t>(h) << p.sink.bs_log2), pa, pb, c == 0,
                                      x, h < Hkv && in_pool);
    });
  }
  steps(nkv, [&](int h, float (&x)[8]) {
    store_row<D, KIND, BF16, INTER>(p.sink, true, row0 + (static_cast<int64_t>(h) << p.sink.bs_log2), pa, pb, c == 0, x,
                                    h < Hkv && in_pool);
  });
}

// Threads per token: with few tokens a token's heads run side by side, with
// many the factors are shared by more heads of a group.  Measured (152 SMs, 32 query
// and 8 K/V heads of 128 channels; 256, 128, 64, 32 threads): 64 tokens 3.4, 4.1,
// 5.8, 9.1 us; 608: 5.1, 4.8, 5.8, 9.2; 1216: 9.0, 6.9, 7.0, 9.2; 2432: 16.9,
// 12.2, 10.9, 11.5; 32768: 257, 181, 134, 126.  No more groups than query heads:
// 1216 tokens of 2 query heads 4.2 -> 3.4 us (64 tokens 3.1 -> 3.2).
template <int D, int KIND, bool BF16, bool INTER, int TPT>
cudaError_t launch_threads(const NormRopeParams& p, cudaStream_t st) {
  constexpr unsigned per_cta = kNrThreads / TPT;
  const unsigned T = static_cast<unsigned>(p.T);
  return launch_in_order(norm_rope_kernel<D, KIND, BF16, INTER, TPT>, (T + per_cta - 1) / per_cta, kNrThreads, 0, st, p);
}

template <int D, int KIND, bool BF16, bool INTER>
cudaError_t launch_tokens(const NormRopeParams& p, cudaStream_t st) {
  int threads = p.T <= p.sms * 2 ? 256 : (p.T <= p.sms * 8 ? 128 : (p.T <= p.sms * 16 ? 64 : 32));
  while (threads > 32 && threads / 2 >= p.Hq * (D / 8)) threads /= 2;
  if (threads == 256) return launch_threads<D, KIND, BF16, INTER, 256>(p, st);
  if (threads == 128) return launch_threads<D, KIND, BF16, INTER, 128>(p, st);
  if (threads == 64) return launch_threads<D, KIND, BF16, INTER, 64>(p, st);
  return launch_threads<D, KIND, BF16, INTER, 32>(p, st);
}

template <int D, int KIND>
cudaError_t launch_type(const NormRopeParams& p, cudaStream_t st) {
  if (p.interleaved)
    return p.bf16 ? launch_tokens<D, KIND, true, true>(p, st) : launch_tokens<D, KIND, false, true>(p, st);
  return p.bf16 ? launch_tokens<D, KIND, true, false>(p, st) : launch_tokens<D, KIND, false, false>(p, st);
}

template <int D>
cudaError_t launch_kind(const NormRopeParams& p, int kind, cudaStream_t st) {
  if (kind == kSink16) return launch_type<D, kSink16>(p, st);
  return kind == kSinkTensor ? launch_type<D, kSinkTensor>(p, st) : launch_type<D, kSinkRows>(p, st);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& p0, int sink_kind, cudaStream_t st) {
  NormRopeParams p = p0;
  p.tab16 = (reinterpret_cast<uintptr_t>(p.cos_sin) & 15) == 0;
  return p.sink.D == 64 ? launch_kind<64>(p, sink_kind, st) : launch_kind<128>(p, sink_kind, st);
}

}  // namespace pa
