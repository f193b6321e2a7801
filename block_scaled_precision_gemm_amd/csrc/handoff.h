// Handing results from the workgroups of one launch to the last of them to finish.
//
// A release / acquire fence at device scope writes back and invalidates an XCD's whole L2; with one
// per workgroup these serialise (measured 0.6-1 us per workgroup and XCD: an attention call of 512
// workgroups took 298 us, 100 us without them).  Here only the handed data pays: it is stored and loaded with
// device scope (through the L2s, which are not coherent with each other), each thread waits for its
// own stores, and a relaxed counter is raised after the workgroup's barrier.
#pragma once

#include "common.h"

namespace bsg {

typedef uint32_t v4u_t __attribute__((ext_vector_type(4)));
constexpr int kDeviceScope = 16;  // cache-policy bit sc1 of a buffer access

// A buffer descriptor over `bytes` bytes at `p` (uniform; at most 2^31 - 1).
__device__ __forceinline__ __amdgpu_buffer_rsrc_t handoff_buffer(const void* p, uint32_t bytes) {
  return __builtin_amdgcn_make_buffer_rsrc((void*)p, (short)0, (int)bytes, (int)0x00020000);
}
__device__ __forceinline__ void handoff_store4(__amdgpu_buffer_rsrc_t b, uint32_t float_at, v4f v) {
  __builtin_amdgcn_raw_buffer_store_b128(__builtin_bit_cast(v4u_t, v), b, (int)(float_at * 4u), 0, kDeviceScope);
}
__device__ __forceinline__ v4f handoff_load4(__amdgpu_buffer_rsrc_t b, uint32_t float_at) {
  return __builtin_bit_cast(v4f, __builtin_amdgcn_raw_buffer_load_b128(b, (int)(float_at * 4u), 0, kDeviceScope));
}
__device__ __forceinline__ void handoff_store(float* p, float v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float handoff_load(const float* p) {
  return __hip_atomic_load(const_cast<float*>(p), __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Called by all threads of a workgroup after their handoff stores: whether this workgroup is the last
// of `expected` at `counter`, which is then zero again.  `shared`: an int in LDS.
__device__ __forceinline__ bool last_arrival(int* counter, int expected, int* shared) {
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  __syncthreads();
  if (threadIdx.x == 0) {
    const int before = __hip_atomic_fetch_add(counter, 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    *shared = before == expected - 1;
    if (before == expected - 1) __hip_atomic_store(counter, 0, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
  }
  __syncthreads();
  return *shared;
}

}  // namespace bsg
