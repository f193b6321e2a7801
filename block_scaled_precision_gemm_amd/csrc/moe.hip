// Mixture-of-experts layer for few tokens: router, gate/up with SiLU, down with the weighted sum.
//
// Few tokens read many weights, so the layer is bound by the bytes of the chosen experts' weights,
// and every kernel streams weight rows through registers into v_mfma_f32_16x16x32: rows of weights are
// the product's first operand (16 rows), tokens the second (16 columns, unused ones repeat the first
// token).  A lane loads the codes of 32 consecutive k of one row (16 bytes of E2M1, 32 of E4M3) and
// uses them in four products; the k order of a product is free, so the tokens' operand is read in the
// same order, 64 contiguous bytes per lane.  A workgroup's waves take alternate slabs of 128 k and are
// summed through LDS.
//
// Operands are bf16: E2M1 * E4M3 has at most 6 significant bits and E4M3 * 2^e has 4, so decoded
// weights are exact and keep fp32's range.  16-bit activations are exact as bf16 x, or as the sum of
// two bf16 parts for fp16 x; SiLU(gate) up is held as two bf16 parts (16 significant bits, so its
// rounding is far below the output's).  Each part is one more product per weight fragment.
//
// Three launches: the router must know every token's choice before weights can be read, and the second
// product needs all of an expert's SiLU(gate) up.
#include "handoff.h"
#include "moe.h"

namespace bsg {
namespace {

typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef _Float16 v8h __attribute__((ext_vector_type(8)));
typedef _Float16 v2h __attribute__((ext_vector_type(2)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));

constexpr int kSlab = 128;

__device__ __forceinline__ v4f mfma(v4i a, v4i b, v4f c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8b, a), __builtin_bit_cast(v8b, b), c, 0, 0, 0);
}

__device__ __forceinline__ uint16_t bf16_bits(float x) { return __builtin_bit_cast(uint16_t, (__bf16)x); }
__device__ __forceinline__ float bf16_value(uint16_t b) { return __builtin_bit_cast(float, (uint32_t)b << 16); }

// ------------------------------------------------------------------------------------------- router
constexpr int kRouterThreads = 512;
constexpr int kKeys = 8192;  // logits held in LDS at a time while they are ranked

// Order of floats as unsigned: larger float, larger key; NaN above all; -0 as 0.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = __builtin_bit_cast(uint32_t, x + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Top k of every token and the tokens of every expert; one workgroup.
__device__ void choose(const MoeArgs& p, uint32_t* keys, int* chosen, int* sums) {
  const int tid = threadIdx.x, E = p.experts, K = p.top_k, T = p.tokens;
  const int step = kKeys / E;  // tokens at a time
  for (int t0 = 0; t0 < T; t0 += step) {
    const int n = min(step, T - t0) * E;
    __syncthreads();
    for (int i = tid; i < n; i += kRouterThreads) keys[i] = order_key(handoff_load(p.logits + (size_t)t0 * E + i));
    __syncthreads();
    for (int i = tid; i < n; i += kRouterThreads) {
      const int t = i / E, e = i - t * E;
      const uint32_t mine = keys[i];
      int rank = 0;
      for (int j = 0; j < E; ++j) {
        const uint32_t other = keys[t * E + j];
        rank += other > mine || (other == mine && j < e);
      }
      if (rank < K) chosen[(t0 + t) * K + rank] = e;  // ranks are a permutation: each place is filled once
    }
  }
  __syncthreads();
  // rows of each expert: thread e counts its tokens, places by a scan
  int count = 0;
  if (tid < E)
    for (int i = 0; i < T * K; ++i) count += chosen[i] == tid;
  int rows = count, slots = count > 0;
  const int lane = tid & 63, wave = tid >> 6;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int a = __shfl_up(rows, o), b = __shfl_up(slots, o);
    if (lane >= o) rows += a, slots += b;
  }
  if (lane == 63) sums[wave] = rows, sums[8 + wave] = slots;
  __syncthreads();
  for (int w = 0; w < wave; ++w) rows += sums[w], slots += sums[8 + w];
  if (tid < E && count) {
    int row = rows - count;
    p.slot_expert[slots - 1] = tid;
    p.slot_start[slots - 1] = row;
    for (int i = 0; i < T * K; ++i)
      if (chosen[i] == tid) {
        p.row_token[row] = i / K;
        p.row_of[i] = row++;
      }
  }
  if (tid == kRouterThreads - 1) {
    *p.active = slots;
    p.slot_start[slots] = rows;
  }
  __threadfence_block();
  __syncthreads();
  for (int t = tid; t < T; t += kRouterThreads) {
    const float* l = p.logits + (size_t)t * E;
    const float top = handoff_load(l + chosen[t * K]);
    float sum = 0.0f;
    if (p.keep)
      for (int e = 0; e < E; ++e) sum += __builtin_amdgcn_exp2f((handoff_load(l + e) - top) * 1.44269504088896341f);
    else
      for (int j = 0; j < K; ++j) sum += __builtin_amdgcn_exp2f((handoff_load(l + chosen[t * K + j]) - top) * 1.44269504088896341f);
    for (int j = 0; j < K; ++j) {
      const int i = t * K + j;
      const float w = __builtin_amdgcn_exp2f((handoff_load(l + chosen[i]) - top) * 1.44269504088896341f) / sum;
      p.row_weight[p.row_of[i]] = w;
      if (p.ids) p.ids[i] = chosen[i];
      if (p.weights) p.weights[i] = w;
    }
  }
}

// Workgroup (x, y): logits of experts 16x .. 16x+15 for tokens 16y .. 16y+15, its 8 waves taking
// alternate steps of 32 k; the last workgroup to finish chooses.
template <bool F16>
__global__ __launch_bounds__(kRouterThreads) void router_kernel(MoeArgs p) {
  __shared__ union {
    float part[8][64][4];
    uint32_t keys[kKeys];
  } sh;
  __shared__ int chosen[BSG_MOE_MAX_TOKENS * BSG_MOE_MAX_TOP_K];
  __shared__ int sums[16], last;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, c = lane & 15, g = lane >> 4;
  const int e0 = blockIdx.x * 16, t0 = blockIdx.y * 16;
  const uint16_t* a = p.router + (size_t)min(e0 + c, p.experts - 1) * p.hidden + 8 * g;
  const uint16_t* b = p.x + (int64_t)min(t0 + c, p.tokens - 1) * p.x_stride + 8 * g;
  v4f acc = {0, 0, 0, 0};
  const int steps = p.hidden / 32;
  for (int s = wave; s < steps; s += 8) {
    const v4i aw = *(const v4i*)(a + 32 * s), bw = *(const v4i*)(b + 32 * s);
    if constexpr (F16)
      acc = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, aw), __builtin_bit_cast(v8h, bw), acc, 0, 0, 0);
    else
      acc = mfma(aw, bw, acc);
  }
  *(v4f*)sh.part[wave][lane] = acc;
  if constexpr (F16) {
    // x as two bf16 parts: each workgroup of the row of tokens writes its share of the columns
    const int share = (p.hidden / 8 + gridDim.x - 1) / gridDim.x;
    const int first = blockIdx.x * share, n = min(share, p.hidden / 8 - first);
    const int rows = min(16, p.tokens - t0);
    for (int i = tid; i < rows * n; i += kRouterThreads) {
      const int r = t0 + i / n, col = 8 * (first + i % n);
      const v8h v = *(const v8h*)(p.x + (int64_t)r * p.x_stride + col);
      v4i hi, lo;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const float f0 = (float)v[2 * k], f1 = (float)v[2 * k + 1];
        const uint16_t h0 = bf16_bits(f0), h1 = bf16_bits(f1);
        const bool fin0 = __builtin_fabsf(f0) < 65536.0f, fin1 = __builtin_fabsf(f1) < 65536.0f;  // else no low part
        hi[k] = h0 | h1 << 16;
        lo[k] = (fin0 ? bf16_bits(f0 - bf16_value(h0)) : 0) | (fin1 ? bf16_bits(f1 - bf16_value(h1)) : 0) << 16;
      }
      *(v4i*)(p.xs + (size_t)r * p.hidden + col) = hi;
      *(v4i*)(p.xs + (size_t)(p.tokens + r) * p.hidden + col) = lo;
    }
  }
  __syncthreads();
  if (wave == 0) {
    v4f s = *(v4f*)sh.part[0][lane];
#pragma unroll
    for (int w = 1; w < 8; ++w) s += *(v4f*)sh.part[w][lane];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (t0 + c < p.tokens && e0 + 4 * g + i < p.experts) 
        handoff_store(p.logits + (size_t)(t0 + c) * p.experts + e0 + 4 * g + i, s[i]);
  }
  if (last_arrival(p.arrived, gridDim.x * gridDim.y, &last)) choose(p, sh.keys, chosen, sums);
}

// ------------------------------------------------------------------------------------------- weights
// One row's 32 codes from k0 on, and their scales, decoded to four bf16 fragments.
template <bool NV>
struct Row;

template <>
struct Row<true> {  // NVFP4: two scales
  v4i q;
  uint32_t s;
  __device__ __forceinline__ void load(const uint8_t* w, const uint8_t* sc, int64_t row, int K, int k0) {
    q = *(const v4i*)(w + row * (K / 2) + k0 / 2);
    s = *(const uint16_t*)(sc + row * (K / 16) + k0 / 16);
  }
  __device__ __forceinline__ void clear() {
    q = v4i{0, 0, 0, 0};
    s = 0;
  }
  __device__ __forceinline__ v4i fragment(int j) const {
    const float f = j < 2 ? __builtin_amdgcn_cvt_f32_fp8((int)s, 0) : __builtin_amdgcn_cvt_f32_fp8((int)s, 1);
    const uint32_t w = (uint32_t)q[j];
    const v2f a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 1);
    const v2f c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(w, 1.0f, 3);
    // products of at most 6 significant bits: their upper halves are the bf16 values
    auto pair = [&](float x, float y) {
      return (int)__builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, y * f), __builtin_bit_cast(uint32_t, x * f), 0x07060302u);
    };
    const float a0 = a[0], a1 = a[1], b0 = b[0], b1 = b[1], c0 = c[0], c1 = c[1], d0 = d[0], d1 = d[1];
    return v4i{pair(a0, a1), pair(b0, b1), pair(c0, c1), pair(d0, d1)};
  }
};

template <>
struct Row<false> {  // MXFP8: one scale
  v4i q0, q1;
  uint32_t s;
  __device__ __forceinline__ void load(const uint8_t* w, const uint8_t* sc, int64_t row, int K, int k0) {
    q0 = *(const v4i*)(w + row * K + k0);
    q1 = *(const v4i*)(w + row * K + k0 + 16);
    s = sc[row * (K / 32) + k0 / 32];
  }
  __device__ __forceinline__ void clear() {
    q0 = q1 = v4i{0, 0, 0, 0};
    s = 0;
  }
  __device__ __forceinline__ v4i fragment(int j) const {
    const float f = __builtin_bit_cast(float, s << 23);
    const v4i q = j < 2 ? q0 : q1;
    const int lo = q[2 * (j & 1)], hi = q[2 * (j & 1) + 1];
    return v4i{__builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, f, false)),
               __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, f, true)),
               __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, f, false)),
               __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, f, true))};
  }
};

// acc[tile][nt] += rows x columns over the slabs wave, wave + 4, ...: rows of tile m are w's rows
// row[m] + lane % 16, columns the activations at b + column[nt] (element offsets), PARTS parts `part`
// elements apart.
template <bool NV, int TILES, int NT, int PARTS>
__device__ __forceinline__ void products(const uint8_t* w, const uint8_t* sc, const int64_t row[TILES], int K, int wave,
                                         int g, const uint16_t* b, const int64_t column[NT], int64_t part, int nts,
                                         v4f acc[TILES][NT]) {
  const int slabs = (K + kSlab - 1) / kSlab;
  Row<NV> cur[TILES], next[TILES];
  auto fetch = [&](Row<NV>* r, int s) {
    const int k0 = s * kSlab + 32 * g;
    if (k0 < K) {
#pragma unroll
      for (int m = 0; m < TILES; ++m) r[m].load(w, sc, row[m], K, k0);
    } else {
#pragma unroll
      for (int m = 0; m < TILES; ++m) r[m].clear();
    }
  };
  if (wave < slabs) fetch(cur, wave);
  for (int s = wave; s < slabs; s += 4) {
    if (s + 4 < slabs) fetch(next, s + 4);
    const int k0 = s * kSlab + 32 * g;
    v4i x[PARTS][NT][4];
#pragma unroll
    for (int q = 0; q < PARTS; ++q)
#pragma unroll
      for (int n = 0; n < NT; ++n)
        if (n < nts) {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            x[q][n][j] = k0 < K ? *(const v4i*)(b + q * part + column[n] + k0 + 8 * j) : v4i{0, 0, 0, 0};
        }
#pragma unroll
    for (int m = 0; m < TILES; ++m)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const v4i a = cur[m].fragment(j);
#pragma unroll
        for (int n = 0; n < NT; ++n)
          if (n < nts) {
#pragma unroll
            for (int q = 0; q < PARTS; ++q) acc[m][n] = mfma(a, x[q][n][j], acc[m][n]);
          }
      }
#pragma unroll
    for (int m = 0; m < TILES; ++m) cur[m] = next[m];
  }
}

constexpr int kThreads = 256;

// Workgroup (x, slot): SiLU(gate) up of dims 32x .. 32x+31 for the tokens of the slot's expert.
template <bool NV, int NT, int PARTS>
__global__ __launch_bounds__(kThreads) void gate_up_kernel(MoeArgs p) {
  constexpr int TILES = 4;  // gate rows 0..15, 16..31, up rows 0..15, 16..31
  __shared__ v4f sh[4][TILES][NT][64];
  if ((int)blockIdx.y >= *p.active) return;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, c = lane & 15, g = lane >> 4;
  const int e = p.slot_expert[blockIdx.y], start = p.slot_start[blockIdx.y], count = p.slot_start[blockIdx.y + 1] - start;
  const int nts = (count + 15) / 16, i0 = blockIdx.x * 32;
  int64_t row[TILES], column[NT];
#pragma unroll
  for (int m = 0; m < TILES; ++m) {
    const int i = min(i0 + (m & 1) * 16 + c, p.inter - 1);
    row[m] = (int64_t)e * 2 * p.inter + (m < 2 ? 0 : p.inter) + i;
  }
  const uint16_t* b = PARTS == 1 ? p.x : p.xs;
  const int64_t stride = PARTS == 1 ? p.x_stride : p.hidden;
#pragma unroll
  for (int n = 0; n < NT; ++n) column[n] = p.row_token[start + min(16 * n + c, count - 1)] * stride;
  v4f acc[TILES][NT] = {};
  products<NV, TILES, NT, PARTS>(p.w13, p.s13, row, p.hidden, wave, g, b, column, (int64_t)p.tokens * p.hidden, nts, acc);
#pragma unroll
  for (int m = 0; m < TILES; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) sh[wave][m][n][lane] = acc[m][n];
  __syncthreads();
  const float alpha = p.alpha13 ? p.alpha13[e] : 1.0f;
  const int64_t rows = (int64_t)p.tokens * p.top_k;
  for (int k = tid; k < 2 * nts * 64; k += kThreads) {
    const int l = k & 63, m = (k >> 6) & 1, n = k >> 7, col = 16 * n + (l & 15), i = i0 + 16 * m + 4 * (l >> 4);
    v4f gate = sh[0][m][n][l], up = sh[0][m + 2][n][l];
#pragma unroll
    for (int w = 1; w < 4; ++w) gate += sh[w][m][n][l], up += sh[w][m + 2][n][l];
    if (col >= count || i >= p.inter) continue;
    uint16_t hi[4], lo[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float x = alpha * gate[r], u = alpha * up[r];
      const float v = x / (1.0f + __builtin_amdgcn_exp2f(x * -1.44269504088896341f)) * u;
      hi[r] = bf16_bits(v);
      const float rest = v - bf16_value(hi[r]);
      lo[r] = rest - rest == 0.0f ? bf16_bits(rest) : 0;  // an infinite high part has no low part
    }
    uint16_t* dst = p.h + (start + col) * (int64_t)p.inter + i;
    *(uint2*)dst = make_uint2(hi[0] | hi[1] << 16, hi[2] | hi[3] << 16);
    *(uint2*)(dst + rows * p.inter) = make_uint2(lo[0] | lo[1] << 16, lo[2] | lo[3] << 16);
  }
}

// Workgroup (x, slot): output dims 64x .. 64x+63 of the slot's tokens, times their weights; the last
// slot of a row of workgroups to finish adds each token's choices in the order of their rank.
template <bool NV, bool F16, int NT>
__global__ __launch_bounds__(kThreads) void down_kernel(MoeArgs p) {
  constexpr int TILES = 4;
  __shared__ v4f sh[4][TILES][NT][64];
  __shared__ int last;
  const int active = *p.active;
  if ((int)blockIdx.y >= active) return;
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, c = lane & 15, g = lane >> 4;
  const int e = p.slot_expert[blockIdx.y], start = p.slot_start[blockIdx.y], count = p.slot_start[blockIdx.y + 1] - start;
  const int nts = (count + 15) / 16, d0 = blockIdx.x * 64;
  int64_t row[TILES], column[NT];
#pragma unroll
  for (int m = 0; m < TILES; ++m) row[m] = (int64_t)e * p.hidden + min(d0 + 16 * m + c, p.hidden - 1);
#pragma unroll
  for (int n = 0; n < NT; ++n) column[n] = (int64_t)(start + min(16 * n + c, count - 1)) * p.inter;
  v4f acc[TILES][NT] = {};
  products<NV, TILES, NT, 2>(p.w2, p.s2, row, p.inter, wave, g, p.h, column, (int64_t)p.tokens * p.top_k * p.inter, nts, acc);
#pragma unroll
  for (int m = 0; m < TILES; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) sh[wave][m][n][lane] = acc[m][n];
  __syncthreads();
  const float alpha = p.alpha2 ? p.alpha2[e] : 1.0f;
  // (a few tokens' rows: far below 2^31 bytes)
  const __amdgpu_buffer_rsrc_t ybuf = handoff_buffer(p.y, (uint32_t)(p.tokens * p.top_k) * (uint32_t)p.hidden * 4u);
  for (int k = tid; k < TILES * nts * 64; k += kThreads) {
    const int l = k & 63, m = (k >> 6) % TILES, n = (k >> 6) / TILES, col = 16 * n + (l & 15), d = d0 + 16 * m + 4 * (l >> 4);
    v4f y = sh[0][m][n][l];
#pragma unroll
    for (int w = 1; w < 4; ++w) y += sh[w][m][n][l];
    if (col >= count || d >= p.hidden) continue;
    handoff_store4(ybuf, (uint32_t)(start + col) * p.hidden + d, y * (alpha * p.row_weight[start + col]));
  }
  if (!last_arrival(p.arrived + 1 + blockIdx.x, active, &last)) return;
  for (int k = tid; k < p.tokens * 16; k += kThreads) {
    const int t = k >> 4, d = d0 + 4 * (k & 15);
    if (d >= p.hidden) continue;
    v4f y = {0, 0, 0, 0};
    for (int j = 0; j < p.top_k; ++j) y += handoff_load4(ybuf, (uint32_t)p.row_of[t * p.top_k + j] * p.hidden + d);
    uint32_t b[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) b[r] = F16 ? __builtin_bit_cast(uint16_t, (_Float16)y[r]) : bf16_bits(y[r]);
    *(uint2*)(p.out + t * p.out_stride + d) = make_uint2(b[0] | b[1] << 16, b[2] | b[3] << 16);
  }
}

template <bool NV, bool F16, int NT>
hipError_t launch(const MoeArgs& a, hipStream_t stream) {
  MoeArgs args = a;
  void* argv[] = {&args};
  hipError_t e = hipLaunchKernel((const void*)&router_kernel<F16>, dim3((a.experts + 15) / 16, (a.tokens + 15) / 16),
                                 dim3(kRouterThreads), argv, 0, stream);
  if (e != hipSuccess) return e;
  const unsigned slots = a.tokens * a.top_k < a.experts ? a.tokens * a.top_k : a.experts;
  e = hipLaunchKernel((const void*)&gate_up_kernel<NV, NT, F16 ? 2 : 1>, dim3((a.inter + 31) / 32, slots), dim3(kThreads),
                      argv, 0, stream);
  if (e != hipSuccess) return e;
  return hipLaunchKernel((const void*)&down_kernel<NV, F16, NT>, dim3((a.hidden + 63) / 64, slots), dim3(kThreads), argv, 0,
                         stream);
}

template <bool NV, bool F16>
hipError_t launch_nt(const MoeArgs& a, hipStream_t stream) {
  // an expert may get every token
  if (a.tokens <= 16) return launch<NV, F16, 1>(a, stream);
  if (a.tokens <= 32) return launch<NV, F16, 2>(a, stream);
  return launch<NV, F16, 4>(a, stream);
}

}  // namespace

hipError_t moe_launch(const MoeArgs& a, int format, int dtype, hipStream_t stream) {
  if (format) return dtype ? launch_nt<true, true>(a, stream) : launch_nt<true, false>(a, stream);
  return dtype ? launch_nt<false, true>(a, stream) : launch_nt<false, false>(a, stream);
}

size_t moe_workspace(const bsg_moe_problem& p, uint8_t* base, MoeArgs* a, size_t* counters_at, size_t* counters_bytes) {
  const size_t T = (size_t)p.max_tokens, rows = T * p.top_k;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) & ~(size_t)255;
    return base ? base + here : nullptr;
  };
  a->logits = (float*)take(T * p.experts * 4);
  a->xs = (uint16_t*)take(p.dtype == BSG_OUT_F16 ? 2 * T * p.hidden * 2 : 0);
  a->h = (uint16_t*)take(2 * rows * p.inter * 2);
  a->y = (float*)take(rows * p.hidden * 4);
  a->active = (int*)take(4);
  a->slot_expert = (int*)take((size_t)p.experts * 4);
  a->slot_start = (int*)take(((size_t)p.experts + 1) * 4);
  a->row_token = (int*)take(rows * 4);
  a->row_weight = (float*)take(rows * 4);
  a->row_of = (int*)take(rows * 4);
  *counters_at = at;
  *counters_bytes = (1 + ((size_t)p.hidden + 63) / 64) * 4;
  a->arrived = (int*)take(*counters_bytes);
  return at;
}

}  // namespace bsg
