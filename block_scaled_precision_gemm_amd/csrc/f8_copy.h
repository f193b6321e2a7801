// Memory to LDS and registers through buffer descriptors, for the products in E4M3.
#pragma once

#include "common.h"

namespace bsg {

constexpr int kOut = (int)0x80000000u;  // an offset past any buffer: zeros, no traffic
constexpr int kRaw = 0x00020000;
typedef __attribute__((address_space(3))) void lds_void;

// 16 or 4 bytes per lane from memory to LDS at dst (uniform), lane after lane.
__device__ __forceinline__ void copy16(__amdgpu_buffer_rsrc_t b, uint8_t* dst, int voff, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (lds_void*)dst, 16, voff, soff, 0, 0);
}
__device__ __forceinline__ void copy4(__amdgpu_buffer_rsrc_t b, uint8_t* dst, int voff, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (lds_void*)dst, 4, voff, soff, 0, 0);
}

}  // namespace bsg
