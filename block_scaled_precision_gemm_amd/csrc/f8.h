// Shared definitions of the products in E4M3 with a scale for each block of 128 (include/bsg_f8.h).
#pragma once

#include "bsg_f8.h"
#include "common.h"

namespace bsg {

// One product's arguments.  w13 products ("gated"): w holds 2 n rows, gate's and then up's, each with its own grid of
// scales, and the result is SiLU(gate) up, n values of a token.
struct F8Args {
  int tokens, n, k, kb;  // kb = ceil(k / 128)
  const uint8_t* x;      // token rows: codes, or 16- or 32-bit values that a kernel quantises as it reads them
  const float* sx;       // [kb][sx_stride], with codes
  int64_t x_stride, sx_stride;  // bytes, floats
  const uint8_t* w;
  const float* sw;
  const float* bias;
  uint8_t* out;          // 16-bit values, codes, or fp32 values
  int64_t out_stride;    // elements
  float* so;             // scales of codes, [ceil(n / 128)][so_stride]
  int64_t so_stride;
  // workspace, and parts of K (the tiled kernel's)
  float* part;
  int* arrived;          // one for each tile, zero between calls
  int splits;
  int exact;             // (host) products of widened codes, however many tokens
};

// How token rows come: codes with scales, or values of 16 or 32 bits.
enum class Src : int { CODES, BF16, F16, F32 };

__host__ __device__ constexpr int f8_blocks(int64_t n) { return (int)((n + 127) / 128); }

// The scale of a block whose largest magnitude has the bits `b` in fp32: the least power of two s >= 2^-126 with
// that magnitude <= 448 s = 1.75 * 2^8 s, so its exponent less 8, and one more where the significand passes 1.75.
__device__ __forceinline__ float f8_scale(uint32_t b) {
  const int e = (int)((b + 0x1FFFFFu) >> 23) - 8;
  return __builtin_bit_cast(float, (uint32_t)max(e, 1) << 23);
}

hipError_t f8_quantize_launch(Src src, int64_t rows, int64_t cols, const void* x, int64_t x_stride, void* codes,
                              int64_t codes_stride, float* scales, int64_t scale_stride, hipStream_t stream);

// dtype: 0 bf16, 1 f16.
// Up to kF8OneTile tokens.  Gated results are fp32 values [tokens][out_stride].
constexpr int kF8OneTile = 16;
hipError_t f8_few_launch(const F8Args& a, Src src, bool gated, int dtype, hipStream_t stream);

// Any number of tokens, as codes.  Gated results are codes with scales, of up to kF8WideTokens tokens (f8_cut.h) by products of
// widened codes.
hipError_t f8_tiled_launch(const F8Args& a, bool gated, int dtype, int cus, hipStream_t stream);

// The same, in tiles of 256 x 256 (gated: 128 outputs).
hipError_t f8_pp_launch(const F8Args& a, bool gated, int dtype, int cus, hipStream_t stream);

}  // namespace bsg
