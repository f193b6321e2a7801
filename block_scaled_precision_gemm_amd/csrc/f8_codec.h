// Values to E4M3 codes with a power-of-two scale for each block of 128 (include/bsg_f8.h), on the device.
//
// v_cvt_scalef32_pk_fp8_{bf16,f16,f32} divides by the power of two that its scale operand's exponent holds and rounds
// the exact quotient to nearest even, so 16-bit values become codes without being widened.
#pragma once

#include "codec.h"
#include "f8.h"

namespace bsg {

typedef __bf16 v2bf __attribute__((ext_vector_type(2)));
typedef short v2s __attribute__((ext_vector_type(2)));
typedef uint16_t v2us __attribute__((ext_vector_type(2)));

constexpr int f8_src_bytes(Src s) { return s == Src::CODES ? 1 : s == Src::F32 ? 4 : 2; }

// 16 consecutive values of a row, in NV vectors of 16 bytes.
template <Src S>
struct Values16 {
  static constexpr int NV = f8_src_bytes(S);
  v4i v[NV];

  // Bits, in fp32, of their largest magnitude; those of an infinity or a NaN are at least 0x7F800000.
  __device__ __forceinline__ uint32_t amax() const {
    if constexpr (S == Src::F32) {
      uint32_t m = 0;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) m = max(m, (uint32_t)v[i][j] & 0x7FFFFFFFu);
      return m;
    } else {
      v2us m = {0, 0};
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j)
          m = __builtin_elementwise_max(m, __builtin_bit_cast(v2us, (uint32_t)v[i][j] & 0x7FFF7FFFu));
      const uint16_t t = m[0] > m[1] ? m[0] : m[1];
      if constexpr (S == Src::BF16) return (uint32_t)t << 16;
      else return __builtin_bit_cast(uint32_t, (float)__builtin_bit_cast(_Float16, t));
    }
  }

  __device__ __forceinline__ v4i codes(float scale) const {
    v4i q;
#pragma unroll
    for (int d = 0; d < 4; ++d) {  // four codes
      v2s w = {0, 0};
      if constexpr (S == Src::F32) {
        w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, at(4 * d), at(4 * d + 1), scale, false);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, at(4 * d + 2), at(4 * d + 3), scale, true);
      } else {
        const uint32_t a = (uint32_t)v[d / 2][d % 2 * 2], b = (uint32_t)v[d / 2][d % 2 * 2 + 1];
        if constexpr (S == Src::BF16) {
          w = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(w, __builtin_bit_cast(v2bf, a), scale, false);
          w = __builtin_amdgcn_cvt_scalef32_pk_fp8_bf16(w, __builtin_bit_cast(v2bf, b), scale, true);
        } else {
          w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(w, __builtin_bit_cast(v2h, a), scale, false);
          w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f16(w, __builtin_bit_cast(v2h, b), scale, true);
        }
      }
      q[d] = __builtin_bit_cast(int, w);
    }
    return q;
  }

 private:
  __device__ __forceinline__ float at(int i) const {
    const int bits = v[i / 4][i % 4];  // (a copy: taken from the vector itself, every element is read as the first)
    return __builtin_bit_cast(float, bits);
  }
};

// 32 codes as fp16.
__device__ __forceinline__ void f8_widen(v4i a, v4i b, v8h out[4]) {
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    v2h h[4];
#pragma unroll
    for (int d = 0; d < 2; ++d) {
      const int w = j < 2 ? a[2 * j + d] : b[2 * (j - 2) + d];
      h[2 * d] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, false);
      h[2 * d + 1] = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w, 1.0f, true);
    }
    out[j] = v8h{h[0][0], h[0][1], h[1][0], h[1][1], h[2][0], h[2][1], h[3][0], h[3][1]};
  }
}

// Four values as codes.
__device__ __forceinline__ int f8_codes4(v4f v, float scale) {
  v2s w = {0, 0};
  w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, v[0], v[1], scale, false);
  w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, v[2], v[3], scale, true);
  return __builtin_bit_cast(int, w);
}

// SiLU(gate) up, with the hardware's exponential and reciprocal (1 ulp each).
__device__ __forceinline__ float f8_gated(float gate, float up) {
  return gate * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-gate * 1.44269504088896341f)) * up;
}

// The largest of a value over the 8 lanes that hold a block.
__device__ __forceinline__ uint32_t f8_max8(uint32_t x) {
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0xB1, 0xF, 0xF, true));   // lanes 1, 0, 3, 2 of each four
  x = max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x4E, 0xF, 0xF, true));   // lanes 2, 3, 0, 1
  return max(x, (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, 0x141, 0xF, 0xF, true));  // of each eight, back to front
}

constexpr int kF8Nan = 0x7F7F7F7F;  // four codes of a block that holds an infinity or a NaN
__device__ __forceinline__ bool f8_not_finite(uint32_t amax) { return amax >= 0x7F800000u; }

}  // namespace bsg
