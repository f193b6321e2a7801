// Products in E4M3 with a scale for each block of 128, for up to 16 tokens: the weights stream through.
//
// A workgroup takes 16 RT weight rows; its eight waves take every eighth block of 128 along k and are joined through
// LDS, in the order of the waves.  Weights go from memory to registers in the layout of a matrix product's operand: lane l
// holds row l % 16, and of each block bytes 16 g .. 16 g + 15 and 64 + 16 g .. (g = l / 16).  The order of k inside a block
// is free as long as both operands have it.  The tokens are the columns, so a lane's four sums are four consecutive outputs
// of one token, and the product of a block is scaled by one factor per lane, sx sw, as it is added.
//
// Tokens that come as 16- or 32-bit values are quantised on the way (the feed-forward block of few tokens has no launch of its
// own for that): the workgroup puts their codes into LDS while its first weights are on their way.  Read by every wave for
// its own blocks, the values would be most of the load instructions, as one token fills one column of 16 (block of one
// token, hidden 2048, inter 4096: 12.7 us so, 11.6 us from LDS; hidden 4096, inter 8192: 28.1 and 25.2 us).  16 tokens,
// also quantised by every workgroup: hidden 4096, inter 8192 36 to 39 us.  Codes are read by the waves: one token
// x 4096 x 4096 takes 5.2 to 5.6 us, 16 tokens 6.3, 16 x 8192 x 8192 18.9 (by way of LDS, with two blocks in flight, one token
// took 6.1 us for 5.5 and 16 tokens 8.3 for 6.4).
//
// The next block is asked for when the last is computed, and the machine's other waves (two workgroups a CU, and all CUs) fill
// the rest: with two blocks in flight 5.6 us for 5.2, with four 5.9 (one token x 8192 x 8192: 13.4 and 14.3 for 12.5 us).
//
// The codes are widened to fp16, which holds every E4M3 value, and multiplied by v_mfma_f32_16x16x32_f16: its products are
// exact and its sums fp32.  The matrix instructions that take E4M3 itself align the products of 8 elements to the largest and
// drop what lies 2^-13 below (2e-6 of the sum of magnitudes for Gaussian elements), which turns one in 400 of the feed-forward
// block's inner values to a neighbouring code; their rate is of no use here, where the matrix units wait for the weights' bytes.
#include "epilogue.h"
#include "f8_codec.h"
#include "f8_copy.h"

namespace bsg {
namespace {

constexpr int kWaves = 8, kThreads = 64 * kWaves;
constexpr int kHeld = 512;              // blocks of tokens held in LDS at a time

__device__ __forceinline__ v4i load16(__amdgpu_buffer_rsrc_t b, int voff, int soff) {
  return __builtin_bit_cast(v4i, __builtin_amdgcn_raw_buffer_load_b128(b, voff, soff, 0));
}

// S: how tokens come.  RT: tiles of 16 weight rows; gated, alternately gate's and up's.
template <Src S, int RT, bool GATED, Out O>
__global__ __launch_bounds__(kThreads, 2) void few_kernel(F8Args p) {
  constexpr int NS = GATED ? 2 : 1, XB = f8_src_bytes(S);
  constexpr bool HELD = S != Src::CODES;  // tokens in LDS
  constexpr int kCodes = HELD ? kHeld * 128 : 16;
  __shared__ union {
    struct {
      uint8_t codes[kCodes];  // [block][token], chunk q of 16 at q ^ (token / 2 % 8)
      float scales[HELD ? kHeld : 1];
    } x;
    v4f red[kWaves][RT][64];
  } sh;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int c = lane & 15, g = lane >> 4, T = p.tokens, k = p.k;
  const int n0 = blockIdx.x * (16 * RT / NS);

  __amdgpu_buffer_rsrc_t wb[NS];
  const float* sw[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) {
    wb[s] = __builtin_amdgcn_make_buffer_rsrc((void*)(p.w + ((int64_t)s * p.n + n0) * k), (short)0,
                                              min(16 * RT / NS, p.n - n0) * k, kRaw);
    sw[s] = p.sw + ((int64_t)s * f8_blocks(p.n) + n0 / 128) * p.kb;
  }
  int w_row[RT / NS];
#pragma unroll
  for (int r = 0; r < RT / NS; ++r) w_row[r] = (16 * r + c) * k + 16 * g;
  const int xs = (int)p.x_stride, col = min(c, T - 1), x_lane = c * xs + 16 * g;
  const __amdgpu_buffer_rsrc_t xb = __builtin_amdgcn_make_buffer_rsrc((void*)p.x, (short)0, (T - 1) * xs + k, kRaw);
  struct Step {
    v4i w[RT][2];
    float sw[NS];
    v4i x[HELD ? 1 : 2];
    float sx;
  } step;
  auto load = [&](Step& q, int b) __attribute__((always_inline)) {
    const bool in0 = 128 * b + 16 * g < k, in1 = 128 * b + 64 + 16 * g < k;  // (k is a multiple of 16)
    const int col128 = b < p.kb ? 128 * b : 0;  // scalar offsets stay inside the buffers, lane offsets tell what is outside
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      q.w[r][0] = load16(wb[r % NS], in0 ? w_row[r / NS] : kOut, col128);
      q.w[r][1] = load16(wb[r % NS], in1 ? w_row[r / NS] + 64 : kOut, col128);
    }
#pragma unroll
    for (int s = 0; s < NS; ++s) q.sw[s] = sw[s][min(b, p.kb - 1)];
    if constexpr (!HELD) {
      q.x[0] = load16(xb, in0 ? x_lane : kOut, col128);
      q.x[1] = load16(xb, in1 ? x_lane + 64 : kOut, col128);
      q.sx = p.sx[min(b, p.kb - 1) * p.sx_stride + col];
    }
  };

  // Tokens' blocks b0 .. b1 - 1 to LDS: 16 values per thread and time, 8 neighbours a block.  The first AT_ONCE loads are
  // issued before `then` is called.
  constexpr int AT_ONCE = 2;
  auto hold = [&](int b0, int b1, auto then) __attribute__((always_inline)) {
    const int blocks = b1 - b0, units = T * blocks * 8;
    Values16<S> v[AT_ONCE];
    auto fetch = [&](Values16<S>& x, int u) __attribute__((always_inline)) {
      const int i = u & 7, t = u / 8 / blocks, b = u / 8 - t * blocks, col = 128 * (b0 + b) + 16 * i;
#pragma unroll
      for (int j = 0; j < XB; ++j)
        x.v[j] = u < units && col < k ? *(const v4i*)(p.x + t * p.x_stride + (int64_t)col * XB + 16 * j) : v4i{0, 0, 0, 0};
    };
    auto keep = [&](const Values16<S>& x, int u) __attribute__((always_inline)) {
      const int i = u & 7, t = u / 8 / blocks, b = u / 8 - t * blocks, at = b * T + t;
      const uint32_t most = f8_max8(x.amax());
      if (u >= units) return;
      *(v4i*)(sh.x.codes + at * 128 + 16 * (i ^ (t >> 1 & 7))) = x.codes(f8_scale(most));
      if (i == 0) sh.x.scales[at] = f8_not_finite(most) ? __builtin_nanf("") : f8_scale(most);
    };
    auto all = [&](int u0, auto first) __attribute__((always_inline)) {
#pragma unroll
      for (int d = 0; d < AT_ONCE; ++d) fetch(v[d], u0 + kThreads * d);
      first();
#pragma unroll
      for (int d = 0; d < AT_ONCE; ++d) keep(v[d], u0 + kThreads * d);
    };
    all(tid, then);
    for (int u0 = tid + kThreads * AT_ONCE; u0 - tid < units; u0 += kThreads * AT_ONCE) all(u0, [] {});
    __syncthreads();
  };

  v4f acc[RT];
#pragma unroll
  for (int r = 0; r < RT; ++r) acc[r] = v4f{0, 0, 0, 0};
  const int f = col >> 1 & 7;
  auto compute = [&](const Step& q, int at) __attribute__((always_inline)) {  // at: the block's place among those held
    v8h x[4];
    float sx;
    if constexpr (HELD) {
      const uint8_t* row = sh.x.codes + (at * T + col) * 128;
      f8_widen(*(const v4i*)(row + 16 * (g ^ f)), *(const v4i*)(row + 16 * ((g + 4) ^ f)), x);
      sx = sh.x.scales[at * T + col];
    } else {
      f8_widen(q.x[0], q.x[1], x);
      sx = q.sx;
    }
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      v8h w[4];
      f8_widen(q.w[r][0], q.w[r][1], w);
      v4f y = {0, 0, 0, 0};
#pragma unroll
      for (int j = 0; j < 4; ++j) y = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[j], x[j], y, 0, 0, 0);
      const float fct = sx * q.sw[r % NS];
#pragma unroll
      for (int i = 0; i < 4; ++i) acc[r][i] = __builtin_fmaf(fct, y[i], acc[r][i]);
    }
  };
  const int chunk = HELD ? kHeld / T : p.kb;  // blocks of tokens held at a time
  for (int b0 = 0; b0 < p.kb; b0 += chunk) {
    const int b1 = min(b0 + chunk, p.kb);
    auto first = [&] {
      if (b0 + wave < b1) load(step, b0 + wave);
    };
    if constexpr (HELD) hold(b0, b1, first);
    else first();
    for (int b = b0 + wave; b < b1; b += kWaves) {
      compute(step, b - b0);
      if (b + kWaves < b1) load(step, b + kWaves);
    }
    if constexpr (HELD) __syncthreads();
  }

#pragma unroll
  for (int r = 0; r < RT; ++r) sh.red[wave][r][lane] = acc[r];
  __syncthreads();
  auto sum_of = [&](int r, int l) {
    v4f y = sh.red[0][r][l];
#pragma unroll
    for (int w = 1; w < kWaves; ++w) y += sh.red[w][r][l];
    return y;
  };
  for (int i = tid; i < RT / NS * 64; i += kThreads) {
    const int l = i & 63, r = i / 64;
    const int n = n0 + 16 * r + 4 * (l >> 4), token = l & 15;
    if (token >= T || n >= p.n) continue;
    if constexpr (GATED) {
      const v4f gate = sum_of(2 * r, l), up = sum_of(2 * r + 1, l);
      v4f h;
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = f8_gated(gate[j], up[j]);
      *(v4f*)((float*)p.out + token * p.out_stride + n) = h;
    } else {
      v4f y = sum_of(r, l);
      if (p.bias) y += v4f{p.bias[n], p.bias[n + 1], p.bias[n + 2], p.bias[n + 3]};
      *(uint2*)((uint16_t*)p.out + token * p.out_stride + n) = make_uint2(pack2_out<O>(y[0], y[1]), pack2_out<O>(y[2], y[3]));
    }
  }
}

template <Src S, int RT, bool GATED, Out O>
hipError_t launch(F8Args a, hipStream_t stream) {
  constexpr int rows = 16 * RT / (GATED ? 2 : 1);
  void* argv[] = {&a};
  return hipLaunchKernel((const void*)&few_kernel<S, RT, GATED, O>, dim3((unsigned)((a.n + rows - 1) / rows)),
                         dim3(kThreads), argv, 0, stream);
}

}  // namespace

hipError_t f8_few_launch(const F8Args& a, Src src, bool gated, int dtype, hipStream_t stream) {
  if (src == Src::CODES)
    return dtype ? launch<Src::CODES, 1, false, Out::F16>(a, stream) : launch<Src::CODES, 1, false, Out::BF16>(a, stream);
  if (gated)
    return src == Src::F16 ? launch<Src::F16, 2, true, Out::F16>(a, stream) : launch<Src::BF16, 2, true, Out::BF16>(a, stream);
  return dtype ? launch<Src::F32, 1, false, Out::F16>(a, stream) : launch<Src::F32, 1, false, Out::BF16>(a, stream);
}

}  // namespace bsg
