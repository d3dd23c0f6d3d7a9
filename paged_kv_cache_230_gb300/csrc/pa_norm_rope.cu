// norm_rope_cache: RMS norm of each query and key head, rotation by the
// token's position, K and V rows into the paged cache, in one pass.
//
// Bound by memory: a token's heads are read once and written once, with a few
// operations per element.  One CTA per token: groups of D / 8 lanes take a head
// each, eight channels (one 16-byte load) per lane, so the head's mean square
// is a shuffle reduction.  The token's cosines and sines are the same for all
// its heads: each lane loads those of its own channels once.  With pairs
// (i, i + rot / 2) a lane's partners are the eight channels of the lane
// rot / 16 further on, exchanged by shuffles (hence rot_dim % 16 == 0); with
// pairs (2 i, 2 i + 1) both are its own.
#include "pa_row_quant.cuh"
#include "pagedattn.h"

namespace pa {

namespace {

constexpr int kNrThreads = 256;

template <int D, int KIND, bool BF16, bool INTER>
__global__ void __launch_bounds__(kNrThreads) norm_rope_kernel(const NormRopeParams p) {
  constexpr int LPR = D / 8;                // lanes per head
  constexpr int GROUPS = kNrThreads / LPR;  // heads at a time
  const int t = blockIdx.x;
  const int c = threadIdx.x % LPR, g0 = threadIdx.x / LPR;
  const int64_t slot = p.sink.slot_mapping[t];
  if (slot < 0) return;  // padding token
  const bool in_pool = slot < p.sink.num_slots;
  if (!in_pool && threadIdx.x == 0) atomicOr(p.sink.err, PA_DEVERR_SLOT);

  // cosines and sines of this lane's eight channels; (1, 0) where not rotated
  float cs[8], sn[8];
  const int half = p.rot / 2;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    cs[i] = 1.f;
    sn[i] = 0.f;
  }
  if (p.rot > 0) {
    int64_t pos = p.positions[t];
    if (pos < 0 || pos >= p.num_positions) {
      if (threadIdx.x == 0) atomicOr(p.sink.err, PA_DEVERR_POSITION);
      pos = pos < 0 ? 0 : p.num_positions - 1;
    }
    const float* row = p.cos_sin + pos * p.rot;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const int d = 8 * c + i;
      if (d < p.rot) {
        const int pair = INTER ? d / 2 : (d < half ? d : d - half);
        cs[i] = __ldg(row + pair);
        const float s = __ldg(row + half + pair);
        // the first of a pair subtracts, the second adds
        sn[i] = (INTER ? (d & 1) == 0 : d < half) ? -s : s;
      }
    }
  }
  // the lane that holds the partners (pairs a half apart), within the head
  int partner = c;
  if (!INTER && 8 * c < p.rot) partner = 8 * c < half ? c + half / 8 : c - half / 8;
  const int src = (threadIdx.x & 31) - c + partner;

  const int rows = p.Hq + 2 * p.sink.Hkv;
  for (int r0 = 0; r0 < rows; r0 += GROUPS) {
    const int r = r0 + g0;
    const bool on = r < rows;
    const bool is_q = r < p.Hq, is_v = r >= p.Hq + p.sink.Hkv;
    const int h = is_q ? r : (is_v ? r - p.Hq - p.sink.Hkv : r - p.Hq);
    float x[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = 0.f;
    if (on) {
      const uint16_t* in = static_cast<const uint16_t*>(is_q ? p.q : (is_v ? p.value : p.key)) +
                           t * (is_q ? p.q_stride : (is_v ? p.value_stride : p.key_stride));
      widen8<BF16>(*reinterpret_cast<const uint4*>(in + h * D + c * 8), x);
    }
    // mean square (all lanes take part in the shuffles; V rows ignore it)
    float ss = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) ss = fmaf(x[i], x[i], ss);
#pragma unroll
    for (int o = LPR / 2; o > 0; o >>= 1) ss += __shfl_xor_sync(0xFFFFFFFFu, ss, o);
    if (on && !is_v && p.q_weight != nullptr) {
      const float inv = 1.f / sqrtf(ss * (1.f / D) + p.eps);
      float w[8];
      widen8<BF16>(__ldg(reinterpret_cast<const uint4*>(static_cast<const uint16_t*>(is_q ? p.q_weight : p.k_weight) +
                                                        c * 8)),
                   w);
#pragma unroll
      for (int i = 0; i < 8; ++i) x[i] = x[i] * inv * w[i];
    }
    float y[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float other = INTER ? x[i ^ 1] : __shfl_sync(0xFFFFFFFFu, x[i], src);
      // unrotated channels keep their value whatever their "partner" holds
      y[i] = !is_v && 8 * c + i < p.rot ? fmaf(x[i], cs[i], other * sn[i]) : x[i];
    }
    if (on && is_q)
      *reinterpret_cast<uint4*>(static_cast<uint16_t*>(p.q_out) + (static_cast<int64_t>(t) * p.Hq + h) * D + c * 8) =
          narrow8<BF16>(y);
    store_row<D, KIND, BF16>(p.sink, is_v, slot, h, c, y, on && !is_q && in_pool);
  }
}

template <int D, int KIND, bool BF16>
void launch_pairs(const NormRopeParams& p, cudaStream_t st) {
  if (p.interleaved)
    norm_rope_kernel<D, KIND, BF16, true><<<p.T, kNrThreads, 0, st>>>(p);
  else
    norm_rope_kernel<D, KIND, BF16, false><<<p.T, kNrThreads, 0, st>>>(p);
}

template <int D, int KIND>
void launch_type(const NormRopeParams& p, cudaStream_t st) {
  if (p.bf16)
    launch_pairs<D, KIND, true>(p, st);
  else
    launch_pairs<D, KIND, false>(p, st);
}

template <int D>
void launch_kind(const NormRopeParams& p, int kind, cudaStream_t st) {
  if (kind == kSink16)
    launch_type<D, kSink16>(p, st);
  else if (kind == kSinkTensor)
    launch_type<D, kSinkTensor>(p, st);
  else
    launch_type<D, kSinkRows>(p, st);
}

}  // namespace

cudaError_t launch_norm_rope(const NormRopeParams& p, int sink_kind, cudaStream_t st) {
  if (p.sink.D == 64)
    launch_kind<64>(p, sink_kind, st);
  else
    launch_kind<128>(p, sink_kind, st);
  return cudaGetLastError();
}

}  // namespace pa
