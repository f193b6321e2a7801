// Rows of 16-bit values to E4M3 codes with a power-of-two scale for each block of 128 (include/bsg_f8.h).
//
// A lane holds 16 consecutive values, so 8 lanes hold a block.  A workgroup takes 16 rows of 8 blocks, two blocks of all
// rows at a time: a row's part is at least 512 bytes in a row, and the 16 scales of a block are neighbours in memory.  All of a
// lane's loads (four blocks) are on their way before the first is used.
//
// Bound: memory, three bytes and a little for each value: 8191 rows of 8192 in 39 to 47 us (4.3 to 5.2 TB/s; a copy of as many
// bytes takes 40 us).  One row of 4096: 2.5 us, a launch.
#include "f8_codec.h"

namespace bsg {
namespace {

constexpr int kThreads = 256, kRows = 16, kStep = 2, kSteps = 4;

template <Src S>
__global__ __launch_bounds__(kThreads) void quant_kernel(const uint8_t* x, int64_t x_stride, uint8_t* codes,
                                                        int64_t codes_stride, float* scales, int64_t scale_stride,
                                                        int64_t rows, int cols) {
  constexpr int NV = Values16<S>::NV;
  const int in_block = threadIdx.x & 7, slot = threadIdx.x >> 3;
  const int64_t row = (int64_t)blockIdx.x * kRows + slot % kRows;
  const int b0 = blockIdx.y * (kStep * kSteps) + slot / kRows;
  const uint8_t* src = x + row * x_stride;
  Values16<S> v[kSteps];
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int col = (b0 + kStep * i) * 128 + 16 * in_block;
#pragma unroll
    for (int j = 0; j < NV; ++j)
      v[i].v[j] = row < rows && col < cols ? *(const v4i*)(src + (int64_t)col * NV + 16 * j) : v4i{0, 0, 0, 0};
  }
#pragma unroll
  for (int i = 0; i < kSteps; ++i) {
    const int b = b0 + kStep * i, col = b * 128 + 16 * in_block;
    const uint32_t most = f8_max8(v[i].amax());
    const float s = f8_scale(most);
    v4i q = v[i].codes(s);
    if (f8_not_finite(most)) q = v4i{kF8Nan, kF8Nan, kF8Nan, kF8Nan};
    if (row < rows && col < cols) {
      *(v4i*)(codes + row * codes_stride + col) = q;
      if (in_block == 0) scales[b * scale_stride + row] = s;
    }
  }
}

}  // namespace

hipError_t f8_quantize_launch(Src src, int64_t rows, int64_t cols, const void* x, int64_t x_stride, void* codes,
                              int64_t codes_stride, float* scales, int64_t scale_stride, hipStream_t stream) {
  const void* fn = src == Src::BF16 ? (const void*)&quant_kernel<Src::BF16> : (const void*)&quant_kernel<Src::F16>;
  const int64_t bytes = x_stride * f8_src_bytes(src);
  int n = (int)cols;
  void* argv[] = {&x, (void*)&bytes, &codes, &codes_stride, &scales, &scale_stride, &rows, &n};
  const dim3 grid((unsigned)((rows + kRows - 1) / kRows), (unsigned)((f8_blocks(cols) + kStep * kSteps - 1) / (kStep * kSteps)));
  return hipLaunchKernel(fn, grid, dim3(kThreads), argv, 0, stream);
}

}  // namespace bsg
