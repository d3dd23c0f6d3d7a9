// Programmatic dependent launch between kernels of one stream: a kernel
// launched with the programmatic-serialization attribute may start while the
// kernel before it runs, once every CTA of that kernel has signalled
// (pdl_trigger) or exited; its threads that read what the earlier kernel
// writes wait for that kernel's completion and memory first (pdl_wait).
// Launched without the attribute, the wait returns at once.
#pragma once

namespace pa {

__device__ __forceinline__ void pdl_trigger() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

// At the start of every thread of a kernel launched by launch_in_order, before
// it can return.
__device__ __forceinline__ void pdl_enter() {
  pdl_wait();
  pdl_trigger();
}

// A load of what an earlier kernel of the stream may have written, in a kernel
// that may have started before that kernel ended.  __ldg would promise that the
// memory is read-only for this kernel's whole lifetime, which lets a load move
// ahead of the wait.
template <class T>
__device__ __forceinline__ T load_written(const T* p) {
  return *p;
}

}  // namespace pa
