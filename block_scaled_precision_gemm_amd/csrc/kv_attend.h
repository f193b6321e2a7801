// What the attention kernels share: layouts of fragments, decoding, query rows.
#pragma once

#include "kv.h"
#include "kv_split.h"

namespace bsg {

typedef float v2f __attribute__((ext_vector_type(2)));

// x, but not known to be the same in every iteration: for paths that few of them take, so that nothing formed
// from it is kept in registers throughout a loop.
__device__ __forceinline__ int rare(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

constexpr int kJoin = 16;       // parts joined at a time
constexpr float kNegInf = -__builtin_inff();
constexpr float kLog2e = 1.44269504088896341f, kLn2 = 0.693147180559945309f;

// Combine the four lanes of one row (lane % 16): each swap gives every lane its own value and its partner's.
__device__ __forceinline__ void swap32(float x, float& a, float& b) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane32_swap(u, u, false, false);
  const uint32_t r0 = r[0], r1 = r[1];
  a = __builtin_bit_cast(float, r0);
  b = __builtin_bit_cast(float, r1);
}
__device__ __forceinline__ void swap16(float x, float& a, float& b) {
  const uint32_t u = __builtin_bit_cast(uint32_t, x);
  const auto r = __builtin_amdgcn_permlane16_swap(u, u, false, false);
  const uint32_t r0 = r[0], r1 = r[1];
  a = __builtin_bit_cast(float, r0);
  b = __builtin_bit_cast(float, r1);
}
__device__ __forceinline__ float max_over_g(float x) {
  float a, b;
  swap32(x, a, b);
  swap16(__builtin_fmaxf(a, b), a, b);
  return __builtin_fmaxf(a, b);
}
__device__ __forceinline__ float sum_over_g(float x) {
  float a, b;
  swap32(x, a, b);
  swap16(a + b, a, b);
  return a + b;
}

// Two non-negative E4M3 codes (bytes SEL picks) -> fp16 pair, times 2^-8; 0x7F -> NaN (0x3F80 + 0x80
// carries into the bit that makes it one).
template <uint32_t SEL>
__device__ __forceinline__ uint32_t scale_pair(uint32_t w) {
  const uint32_t t = __builtin_amdgcn_perm(0u, w, SEL) >> 1;
  return t | ((t + 0x00800080u) & 0x40004000u);
}
constexpr uint32_t kLow = 0x010C000Cu, kHigh = 0x030C020Cu;  // bytes 0, 1 and bytes 2, 3

__device__ __forceinline__ v2h fp4_pair(uint32_t w, int b) {
  // the byte is an immediate of the instruction
  switch (b) {
    case 0: return __builtin_bit_cast(v2h, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 0));
    case 1: return __builtin_bit_cast(v2h, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 1));
    case 2: return __builtin_bit_cast(v2h, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 2));
    default: return __builtin_bit_cast(v2h, __builtin_amdgcn_cvt_scalef32_pk_f16_fp4(w, 1.0f, 3));
  }
}

template <Out O>
__device__ __forceinline__ uint16_t out_bits(float y) {
  if constexpr (O == Out::BF16) return __builtin_bit_cast(uint16_t, (__bf16)y);
  else return __builtin_bit_cast(uint16_t, (_Float16)y);
}

// Query row `row` (token first_token + row / group, head h * group + row % group) in the lanes of its
// column: lane / 16 = g holds dims g D/4 .. (g+1) D/4 - 1.
template <int D>
__device__ __forceinline__ void load_query(const KvArgs& p, int first_token, int h, int row, int g, v4i w[D / 32]) {
  const int i = row / p.group, hq = row - i * p.group;
  const uint16_t* src = (const uint16_t*)p.q.ptr + (int64_t)(first_token + i) * p.q.token_stride +
                        (int64_t)(h * p.group + hq) * p.q.head_stride + g * (D / 4);
#pragma unroll
  for (int j = 0; j < D / 32; ++j) w[j] = *(const v4i*)(src + 8 * j);
}

// The row as fp16, and the base-2 score of one unit of q . k as the products give it, made positive (q
// takes the sign), so that maxima can be taken over the products themselves.  Keys decode times 2^-8;
// bf16 rows are scaled so that their largest magnitude lies in [2^14, 2^15): fp16's steps are then 2^-38 of it and
// less, so that all 8 bits of an element are kept down to 2^-31 of it.  (A row with an infinity or a NaN is scaled as
// if its largest were 2^127, so that its finite elements stay finite.)
template <Out O, int D>
__device__ __forceinline__ void convert_query(const KvArgs& p, const v4i w[D / 32], v8h q[D / 32], float& mul) {
  constexpr int NJ = D / 32;
  mul = p.score_mul * (kLog2e * 256.0f);
  if constexpr (O == Out::F16) {
#pragma unroll
    for (int j = 0; j < NJ; ++j) q[j] = __builtin_bit_cast(v8h, w[j]);
  } else {
    float f[NJ][8], most = 0.0f;
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        f[j][2 * k] = __builtin_bit_cast(float, (uint32_t)w[j][k] << 16);
        f[j][2 * k + 1] = __builtin_bit_cast(float, (uint32_t)w[j][k] & 0xFFFF0000u);
        most = __builtin_fmaxf(most, __builtin_fmaxf(__builtin_fabsf(f[j][2 * k]), __builtin_fabsf(f[j][2 * k + 1])));
      }
    most = max_over_g(most);
    const int e = (int)(__builtin_bit_cast(uint32_t, most) >> 23) - 127;  // -127 for zero and subnormals
    const int up = 14 - min(e, 127);
#pragma unroll
    for (int j = 0; j < NJ; ++j)
#pragma unroll
      for (int k = 0; k < 8; ++k) q[j][k] = (_Float16)__builtin_amdgcn_ldexpf(f[j][k], up);
    mul = __builtin_amdgcn_ldexpf(mul, -up);
  }
  if (p.score_mul < 0.0f)
#pragma unroll
    for (int j = 0; j < NJ; ++j) q[j] = -q[j];
  mul = __builtin_amdgcn_fmed3f(__builtin_fabsf(mul), 1.17549435e-38f, 3.402823466e38f);
}

// The soft cap c of a row's scores, c tanh(score / c), on the products s whose score is s mul (all in base 2; the results are
// products too).  With y = s mul / c:
// * up to y = 1/4: y - y^3/3 + 2 y^5/15 - 17 y^7/315, the next term being 2^-21 of y there;
// * beyond: 1 - 2 / (e^2y + 1), within 2^-20 from there on.  For small y it would lose the digits that y shares with 1, an
//   error of 2^-22 c: a score of 4 under a cap of 1e5 would be off by 0.02, but by no more than 2^-16 under one of 64.
// Caps are mostly far above the scores, so a wave looks first whether any of its scores is beyond.  If so, all of them take
// the second form under caps up to 64, and each its own under others.  64 tokens over up to 16384 positions, 64 heads on 8,
// and 2 x 2048 tokens against 8192 and 3351 positions, 32 heads on 8: 141 and 404 us with no score beyond, 143 and 441 us
// with some and the second form for all, 153 and 554 us with some and both forms.
constexpr float kLowCap = 64.0f * kLog2e;
template <int N>
__device__ __forceinline__ void soft_cap(const KvArgs& p, float mul, v4f s[N]) {
  const float to_y = __builtin_fminf(mul * p.cap_inv, 3e38f);
  float most = 0.0f;
#pragma unroll
  for (int k = 0; k < N; ++k)
#pragma unroll
    for (int i = 0; i < 4; ++i) most = __builtin_fmaxf(most, __builtin_fabsf(s[k][i]));
  auto small = [&](float x, float z) {
    return x * __builtin_fmaf(z, __builtin_fmaf(z, __builtin_fmaf(z, -17.0f / 315, 2.0f / 15), -1.0f / 3), 1.0f);
  };
  if (!__any(most * to_y >= 0.25f)) {
#pragma unroll
    for (int k = 0; k < N; ++k)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float y = s[k][i] * to_y;
        s[k][i] = small(s[k][i], y * y);
      }
  } else {
    const float to_exp = to_y * (2.0f * kLog2e), cap = p.cap * __builtin_amdgcn_rcpf(mul);
    auto large = [&](float x) {
      return cap * __builtin_fmaf(-2.0f, __builtin_amdgcn_rcpf(__builtin_amdgcn_exp2f(x * to_exp) + 1.0f), 1.0f);
    };
    if (p.cap <= kLowCap) {
#pragma unroll
      for (int k = 0; k < N; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) s[k][i] = large(s[k][i]);
    } else {
#pragma unroll
      for (int k = 0; k < N; ++k)
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const float x = s[k][i], y = x * to_y, z = y * y;
          s[k][i] = z >= 0.0625f ? large(x) : small(x, z);
        }
    }
  }
}

hipError_t kv_attend_rows_launch(const KvArgs& a, int dtype, int head_dim, int cus, hipStream_t stream);
// All rows of the batch over the first a->shared positions; fills in where the parts are.  What that costs, in
// microseconds, or a negative number where the parts do not fit the workspace.
double kv_shared_cost(const KvArgs& a, int head_dim, int cus);
hipError_t kv_attend_shared_launch(KvArgs* a, int dtype, int head_dim, int cus, hipStream_t stream);
// 2^kRowsBias P is what the many-row kernels' parts hold, relative to their maxima.
constexpr float kRowsBias = 10.0f;
// Floats of parts that kv_attend_rows_launch may use.
size_t kv_rows_part_floats(const bsg_kv_problem& p, int cus);

}  // namespace bsg
