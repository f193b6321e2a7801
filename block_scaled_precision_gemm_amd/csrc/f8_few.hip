// Products in E4M3 with a scale for each block of 128, for up to 16 tokens: the weights stream through.
//
// A workgroup takes 16 RT weight rows; its eight waves take every eighth block of 128 along k and are joined through
// LDS, in the order of the waves.  Weights go from memory to registers in the layout of a matrix product's operand: lane l
// holds row l % 16, and of each block bytes 16 g .. 16 g + 15 and 64 + 16 g .. (g = l / 16).  The order of k inside a block
// is free as long as both operands have it.  The tokens are the columns, so a lane's four sums are four consecutive outputs
// of one token, and the product of a block is scaled by one factor per lane, sx sw, as it is added.
//
// The codes are widened to fp16, which holds every E4M3 value, and multiplied by v_mfma_f32_16x16x32_f16: its products are
// exact and its sums fp32.  The matrix instructions that take E4M3 itself align the products of a group to the largest and
// keep 14 bits (1.4e-5 of the result, measured), which is more than what the weights' bytes leave idle here would save, and
// would turn one in 400 of the block's inner values to a neighbouring code.
#include "epilogue.h"
#include "f8_codec.h"

namespace bsg {
namespace {

constexpr int kWaves = 8, kThreads = 64 * kWaves;
constexpr int kOut = (int)0x80000000u;  // an offset past any buffer: zeros, no traffic
constexpr int kRaw = 0x00020000;

__device__ __forceinline__ v4i load16(__amdgpu_buffer_rsrc_t b, int voff, int soff) {
  return __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(b, voff, soff, 0));
}

// The largest of a value over the four lanes of a column.
__device__ __forceinline__ uint32_t umax_over_g(uint32_t x) {
  const auto a = __builtin_amdgcn_permlane32_swap(x, x, false, false);
  const uint32_t y = max((uint32_t)a[0], (uint32_t)a[1]);
  const auto b = __builtin_amdgcn_permlane16_swap(y, y, false, false);
  return max((uint32_t)b[0], (uint32_t)b[1]);
}

// S: how tokens come.  TT: tiles of 16 tokens.  RT: tiles of 16 weight rows; gated, alternately gate's and up's.
// D: blocks in flight per wave.
template <Src S, int TT, int RT, bool GATED, Out O, int D>
__global__ __launch_bounds__(kThreads) void few_kernel(F8Args p) {
  constexpr int NS = GATED ? 2 : 1, XB = f8_src_bytes(S);
  __shared__ v4f red[kWaves][RT * TT][64];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int c = lane & 15, g = lane >> 4;
  const int n0 = blockIdx.x * (16 * RT / NS), k = p.k;

  __amdgpu_buffer_rsrc_t wb[NS];
  const float* sw[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    wb[s] = __builtin_amdgcn_make_buffer_rsrc((void*)(p.w + ((int64_t)s * p.n + n0) * k), (short)0,
                                              min(16 * RT / NS, p.n - n0) * k, kRaw);
    sw[s] = p.sw + ((int64_t)s * f8_blocks(p.n) + n0 / 128) * p.kb;
  }
  const int xs = (int)p.x_stride;
  const __amdgpu_buffer_rsrc_t xb =
      __builtin_amdgcn_make_buffer_rsrc((void*)p.x, (short)0, (p.tokens - 1) * xs + k * XB, kRaw);
  const int w_lane = c * k + 16 * g, x_lane = c * xs + 16 * XB * g;
  int w_row[RT / NS];
#pragma unroll
  for (int r = 0; r < RT / NS; ++r) w_row[r] = w_lane + 16 * r * k;
  int sx_at[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) sx_at[t] = min(16 * t + c, p.tokens - 1);

  struct Step {
    v4i w[RT][2];
    Values16<S> x[TT][2];
    float sx[TT], sw[NS];
  } step[D];
  auto load = [&](Step& q, int b) __attribute__((always_inline)) {
    const bool in0 = 128 * b + 16 * g < k, in1 = 128 * b + 64 + 16 * g < k;  // (k is a multiple of 16)
    const int col = b < p.kb ? 128 * b : 0;  // scalar offsets stay inside the buffers, lane offsets tell what is outside
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      q.w[r][0] = load16(wb[r % NS], in0 ? w_row[r / NS] : kOut, col);
      q.w[r][1] = load16(wb[r % NS], in1 ? w_row[r / NS] + 64 : kOut, col);
    }
    const int x0 = in0 ? x_lane : kOut, x1 = in1 ? x_lane + 64 * XB : kOut;
#pragma unroll
    for (int t = 0; t < TT; ++t)
#pragma unroll
      for (int j = 0; j < XB; ++j) {
        q.x[t][0].v[j] = load16(xb, x0 + 16 * j, XB * col + 16 * t * xs);
        q.x[t][1].v[j] = load16(xb, x1 + 16 * j, XB * col + 16 * t * xs);
      }
    const int at = min(b, p.kb - 1);
#pragma unroll
    for (int s = 0; s < NS; ++s) q.sw[s] = sw[s][at];
    if constexpr (S == Src::CODES)
#pragma unroll
      for (int t = 0; t < TT; ++t) q.sx[t] = p.sx[at * p.sx_stride + sx_at[t]];
  };

  v4f acc[RT][TT];
#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[r][t] = v4f{0, 0, 0, 0};
  auto compute = [&](const Step& q) __attribute__((always_inline)) {
    v8h x[TT][4];
    float sx[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      if constexpr (S == Src::CODES) {
        f8_widen(q.x[t][0].v[0], q.x[t][1].v[0], x[t]);
        sx[t] = q.sx[t];
      } else {
        const uint32_t most = umax_over_g(max(q.x[t][0].amax(), q.x[t][1].amax()));
        sx[t] = f8_scale(most);
        f8_widen(q.x[t][0].codes(sx[t]), q.x[t][1].codes(sx[t]), x[t]);
        if (f8_not_finite(most)) sx[t] = __builtin_nanf("");
      }
    }
    float f[NS][TT];
#pragma unroll
    for (int s = 0; s < NS; ++s)
#pragma unroll
      for (int t = 0; t < TT; ++t) f[s][t] = sx[t] * q.sw[s];
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      v8h w[4];
      f8_widen(q.w[r][0], q.w[r][1], w);
      v4f y[TT];
#pragma unroll
      for (int j = 0; j < 4; ++j)
#pragma unroll
        for (int t = 0; t < TT; ++t)
          y[t] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[j], x[t][j], j ? y[t] : v4f{0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
      for (int t = 0; t < TT; ++t)
#pragma unroll
        for (int i = 0; i < 4; ++i) acc[r][t][i] = __builtin_fmaf(f[r % NS][t], y[t][i], acc[r][t][i]);
    }
  };
#pragma unroll
  for (int d = 0; d < D; ++d) load(step[d], wave + kWaves * d);
  for (int b = wave; b < p.kb; b += kWaves * D) {
#pragma unroll
    for (int d = 0; d < D; ++d) {
      if (b + kWaves * d < p.kb) compute(step[d]);
      load(step[d], b + kWaves * (d + D));
    }
  }

#pragma unroll
  for (int r = 0; r < RT; ++r)
#pragma unroll
    for (int t = 0; t < TT; ++t) red[wave][r * TT + t][lane] = acc[r][t];
  __syncthreads();
  auto sum_of = [&](int tile, int l) {
    v4f y = red[0][tile][l];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) y += red[w][tile][l];
    return y;
  };
  for (int i = tid; i < RT / NS * TT * 64; i += kThreads) {
    const int l = i & 63, t = i / 64 % TT, r = i / 64 / TT;
    const int n = n0 + 16 * r + 4 * (l >> 4), token = 16 * t + (l & 15);
    if (token >= p.tokens || n >= p.n) continue;
    if constexpr (GATED) {
      const v4f gate = sum_of((2 * r) * TT + t, l), up = sum_of((2 * r + 1) * TT + t, l);
      v4f h;
#pragma unroll
      for (int j = 0; j < 4; ++j)
        h[j] = f8_gated(gate[j], up[j]);
      *(v4f*)((float*)p.out + token * p.out_stride + n) = h;
    } else {
      v4f y = sum_of(r * TT + t, l);
      if (p.bias) y += v4f{p.bias[n], p.bias[n + 1], p.bias[n + 2], p.bias[n + 3]};
      *(uint2*)((uint16_t*)p.out + token * p.out_stride + n) = make_uint2(pack2_out<O>(y[0], y[1]), pack2_out<O>(y[2], y[3]));
    }
  }
}

template <Src S, int TT, int RT, bool GATED, Out O, int D>
hipError_t launch(F8Args a, hipStream_t stream) {
  constexpr int rows = 16 * RT / (GATED ? 2 : 1);
  void* argv[] = {&a};
  return hipLaunchKernel((const void*)&few_kernel<S, TT, RT, GATED, O, D>, dim3((unsigned)((a.n + rows - 1) / rows)),
                         dim3(kThreads), argv, 0, stream);
}

}  // namespace

hipError_t f8_few_launch(const F8Args& a, Src src, bool gated, int dtype, hipStream_t stream) {
  if (src == Src::CODES)
    return dtype ? launch<Src::CODES, 1, 1, false, Out::F16, 4>(a, stream) : launch<Src::CODES, 1, 1, false, Out::BF16, 4>(a, stream);
  if (gated)
    return src == Src::F16 ? launch<Src::F16, 1, 2, true, Out::F16, 2>(a, stream)
                           : launch<Src::BF16, 1, 2, true, Out::BF16, 2>(a, stream);
  return dtype ? launch<Src::F32, 1, 1, false, Out::F16, 2>(a, stream) : launch<Src::F32, 1, 1, false, Out::BF16, 2>(a, stream);
}

}  // namespace bsg
