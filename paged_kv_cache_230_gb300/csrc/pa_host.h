// Host helpers of the C-ABI front end (pa_api.cu) shared with its other
// translation units: the device error word, argument checks, tensor maps.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "pa_internal.h"
#include "pagedattn.h"

namespace pa {
namespace host {

int sms();                                          // multiprocessors of the current device
int* error_word();                                  // nullptr if CUDA fails
int finish(cudaError_t launch, cudaStream_t st);    // a launch's status; in check mode after waiting for it
bool aligned16(const void* p);
int check_cache(const pa_cache_desc* c, const void* k, const void* v);
int check_kv_scale(int kv_dtype, float kv_scale);
int make_cache_tensor_map(CUtensorMap* m, const void* base, const pa_cache_desc* c);
int64_t split_partitions(int32_t max_context_len, int32_t partition_size);
// Splitting of p's contexts into partitions (p.S, p.Hkv set; Pmax from the
// caller's bound), with the workspace's layout; runs of partitions such that
// there are about `ctas_per_sm` CTAs per SM, and a context's last `fringe` by
// themselves.
void set_split(DecodeParams& p, int64_t Pmax, int32_t partition_size, int head_dim, void* workspace, int ctas_per_sm,
               int fringe);
// Device address through which kernels may touch a buffer; false if none.
bool device_view(const void* p, void** dev);

}  // namespace host
}  // namespace pa
