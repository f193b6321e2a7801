// Products in E4M3 with a scale for each block of 128, for many tokens: tiles of BN weight rows and BT tokens.
//
// * K in steps of one block (128 bytes of a row).  Both operands go from memory to LDS with buffer_load_dwordx4 ... lds,
//   two stages, one barrier per step.  A row is 128 bytes = 8 chunks of 16; chunk q of row R is stored at q ^ ((R >> 1) & 7),
//   so that the fragments' reads hit distinct banks.
// * v_mfma_f32_16x16x128_f8f6f4 with weights as rows and tokens as columns, each product of a block by itself (its
//   third operand is zero), added by vector operations with the factor sx sw, of which a lane has one per 16 tokens: two
//   instructions of a wave's matrix unit leave room for the eight that add their results.
// * LDS rows are ordered so that a lane's results are neighbours in memory: tokens TT c + j (c = lane % 16, tile j), whose
//   scales are one load, and 8 consecutive outputs (16 bytes of 16-bit values, 64 bytes of a row per 4 lanes) or, gated,
//   all of a lane's codes of a token.
#include "epilogue.h"
#include "f8_codec.h"
#include "kv_attend.h"

namespace bsg {
namespace {

constexpr int kOut = (int)0x80000000u;  // an offset past any buffer: zeros, no traffic
constexpr int kRaw = 0x00020000;
typedef __attribute__((address_space(3))) void lds_void;

// 16 bytes per lane from memory to 1 KiB of LDS at dst (uniform).
__device__ __forceinline__ void copy16(__amdgpu_buffer_rsrc_t b, uint8_t* dst, int voff, int soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(b, (lds_void*)dst, 16, voff, soff, 0, 0);
}

template <int BN_, int BT_, int WN_, int WT_, int WG_>
struct Cfg {
  static constexpr int BN = BN_, BT = BT_, WN = WN_, WT = WT_;
  static constexpr int WAVES = WN * WT, THREADS = 64 * WAVES, PER_CU = WG_;
  static constexpr int NT = BN / WN / 16, TT = BT / WT / 16;  // a wave's tiles of 16 rows and 16 tokens
  static constexpr int STAGE = (BN + BT) * 128, COPIES = (BN + BT) / 8 / WAVES;
  static_assert(COPIES * 8 * WAVES == BN + BT && BN % (8 * WAVES) == 0, "copies: whole instructions of one operand");
  static_assert(NT % 2 == 0 && 128 % (16 * NT) == 0, "a wave's rows share a block of scales");
};

__device__ __forceinline__ int2 tile_of(int bid, int tiles_m, int tiles_n) {
  const int T = tiles_m * tiles_n;
  int id = bid;
  if ((T & 7) == 0) id = (bid & 7) * (T >> 3) + (bid >> 3);  // contiguous range per XCD
  constexpr int GM = 8;
  const int per_group = GM * tiles_n;
  const int group = id / per_group;
  const int first_m = group * GM;
  const int gsize = min(tiles_m - first_m, GM);
  const int in_group = id - group * per_group;
  return make_int2(first_m + in_group % gsize, in_group / gsize);
}

template <int BN, int BT, int WN, int WT, int WG, bool GATED, Out O>
__global__ __launch_bounds__(64 * WN * WT, WN* WT* WG / 4) void tiled_kernel(F8Args p) {
  using C = Cfg<BN, BT, WN, WT, WG>;
  constexpr int NT = C::NT, TT = C::TT, NS = GATED ? 2 : 1, BH = C::BN / NS;  // BH: outputs of a tile
  __shared__ __attribute__((aligned(1024))) uint8_t lds[2 * C::STAGE];
  __shared__ uint32_t sh_most[GATED ? C::BT : 1];
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int c = lane & 15, g = lane >> 4;
  const int wn = wave / C::WT, wt = wave % C::WT;
  const int2 at = tile_of(blockIdx.x, (p.tokens + C::BT - 1) / C::BT, (p.n + BH - 1) / BH);
  const int t0 = at.x * C::BT, n0 = at.y * BH, k = p.k;
  const int tokens = min(C::BT, p.tokens - t0), outs = min(BH, p.n - n0);

  // ---- copies: instruction i of the tile fills LDS rows 8 i .. 8 i + 7, eight lanes a row
  const __amdgpu_buffer_rsrc_t xb =
      __builtin_amdgcn_make_buffer_rsrc((void*)(p.x + t0 * p.x_stride), (short)0, (tokens - 1) * (int)p.x_stride + k, kRaw);
  __amdgpu_buffer_rsrc_t wb[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s)
    wb[s] = __builtin_amdgcn_make_buffer_rsrc((void*)(p.w + ((int64_t)s * p.n + n0) * k), (short)0, outs * k, kRaw);
  int voff[C::COPIES], kpos[C::COPIES];
#pragma unroll
  for (int i = 0; i < C::COPIES; ++i) {
    const int ins = wave + C::WAVES * i, R = 8 * ins + (lane >> 3);
    kpos[i] = 16 * ((lane & 7) ^ ((R >> 1) & 7));
    if (8 * ins < C::BN) {
      const int r = R & 15, i16 = R / 16 % NT, w = R / (16 * NT);  // tile i16 of wave row w
      const int row = GATED ? 8 * NT * w + 2 * NT * (r >> 2) + 4 * (i16 % (NT / 2)) + (r & 3)
                            : 16 * NT * w + 32 * (i16 >> 1) + 8 * (r >> 2) + 4 * (i16 & 1) + (r & 3);
      voff[i] = row * k + kpos[i];
    } else {
      const int Q = R - C::BN;
      voff[i] = (Q / (16 * TT) * 16 * TT + TT * (Q & 15) + Q / 16 % TT) * (int)p.x_stride + kpos[i];
    }
  }
  auto copy = [&](int b, int stage) __attribute__((always_inline)) {
    const int left = k - 128 * b;
#pragma unroll
    for (int i = 0; i < C::COPIES; ++i) {
      const int ins = wave + C::WAVES * i;
      // (instructions of one i are all of one operand: BN is a multiple of 8 WAVES)
      const bool weights = 8 * C::WAVES * i < C::BN;
      const bool up = GATED && weights && 8 * ins / 16 % NT >= NT / 2;
      copy16(weights ? (up ? wb[NS - 1] : wb[0]) : xb, lds + stage * C::STAGE + ins * 1024, kpos[i] < left ? voff[i] : kOut,
             128 * b);
    }
  };

  // ---- scales
  const float* sw[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) sw[s] = p.sw + ((int64_t)s * f8_blocks(p.n) + min(n0 + BH / C::WN * wn, p.n - 1) / 128) * p.kb;
  const int first = t0 + 16 * TT * wt + TT * c;
  const float* sx = p.sx + min((int64_t)first, p.sx_stride - TT);
  float x_s[TT], w_s[NS];
  auto scales = [&](int b) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < TT; ++j) x_s[j] = sx[b * p.sx_stride + j];
#pragma unroll
    for (int s = 0; s < NS; ++s) w_s[s] = sw[s][b];
  };

  v4f acc[NT][TT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < TT; ++j) acc[i][j] = v4f{0, 0, 0, 0};

  copy(0, 0);
  scales(0);
  const int f = (c >> 1) & 7, ch0 = 16 * (g ^ f), ch1 = 16 * ((g + 4) ^ f);
  for (int b = 0; b < p.kb; ++b) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
    __syncthreads();
    float s[NS][TT];
#pragma unroll
    for (int a = 0; a < NS; ++a)
#pragma unroll
      for (int j = 0; j < TT; ++j) s[a][j] = x_s[j] * w_s[a];
    if (b + 1 < p.kb) {
      copy(b + 1, (b + 1) & 1);
      scales(b + 1);
    }
    const uint8_t* stage = lds + (b & 1) * C::STAGE;
    auto frag = [&](int row) {
      const v4i lo = *(const v4i*)(stage + row * 128 + ch0), hi = *(const v4i*)(stage + row * 128 + ch1);
      return v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    };
    v8i x[TT];
#pragma unroll
    for (int j = 0; j < TT; ++j) x[j] = frag(C::BN + 16 * (TT * wt + j) + c);
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const v8i w = frag(16 * (NT * wn + i) + c);
#pragma unroll
      for (int j = 0; j < TT; ++j) {
        const v4f y = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, x[j], v4f{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
#pragma unroll
        for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(s[GATED && i >= NT / 2][j], y[e], acc[i][j][e]);
      }
    }
  }

  // ---- results
  if constexpr (GATED) {
    constexpr int H = NT / 2;
    for (int i = tid; i < C::BT; i += C::THREADS) sh_most[i] = 0;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < TT; ++j) {
      uint32_t most = 0;
#pragma unroll
      for (int i = 0; i < H; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float gate = acc[i][j][e];
          const float h = gate * __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-gate * kLog2e)) * acc[H + i][j][e];
          acc[i][j][e] = h;
          most = max(most, __builtin_bit_cast(uint32_t, h) & 0x7FFFFFFFu);
        }
      atomicMax(&sh_most[16 * TT * wt + TT * c + j], most);
    }
    __syncthreads();
    const int n = n0 + 8 * NT * wn + 2 * NT * g;
#pragma unroll
    for (int j = 0; j < TT; ++j) {
      const int t = 16 * TT * wt + TT * c + j;
      const uint32_t most = sh_most[t];
      const float s = f8_scale(most);
      int q[H];
#pragma unroll
      for (int i = 0; i < H; ++i) {
        v2s w = {0, 0};
        w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, acc[i][j][0], acc[i][j][1], s, false);
        w = __builtin_amdgcn_cvt_scalef32_pk_fp8_f32(w, acc[i][j][2], acc[i][j][3], s, true);
        q[i] = f8_not_finite(most) ? kF8Nan : __builtin_bit_cast(int, w);
      }
      if (t < tokens) {
        uint8_t* dst = p.out + (int64_t)(t0 + t) * p.out_stride + n;
        if (n < p.n) {
          if constexpr (H == 4) *(v4i*)dst = v4i{q[0], q[1], q[2], q[3]};
          else *(int2*)dst = make_int2(q[0], q[1]);
        }
        if (wn == 0 && g == 0) p.so[(int64_t)(n0 / 128) * p.so_stride + t0 + t] = s;
      }
    }
  } else {
#pragma unroll
    for (int i = 0; i < NT; i += 2) {
      const int n = n0 + 16 * NT * wn + 16 * i + 8 * g;
      if (n >= p.n) continue;
      float bias[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) bias[e] = p.bias ? p.bias[n + e] : 0.0f;
#pragma unroll
      for (int j = 0; j < TT; ++j) {
        const int t = 16 * TT * wt + TT * c + j;
        if (t >= tokens) continue;
        v4i w;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const v4f y = acc[i + e / 2][j];
          w[e] = (int)pack2_out<O>(y[e % 2 * 2] + bias[2 * e], y[e % 2 * 2 + 1] + bias[2 * e + 1]);
        }
        *(v4i*)((uint16_t*)p.out + (int64_t)(t0 + t) * p.out_stride + n) = w;
      }
    }
  }
}

template <int BN, int BT, int WN, int WT, int WG, bool GATED, Out O>
hipError_t launch(F8Args a, hipStream_t stream) {
  constexpr int BH = BN / (GATED ? 2 : 1);
  void* argv[] = {&a};
  const int64_t tiles = (int64_t)((a.tokens + BT - 1) / BT) * ((a.n + BH - 1) / BH);
  return hipLaunchKernel((const void*)&tiled_kernel<BN, BT, WN, WT, WG, GATED, O>, dim3((unsigned)tiles), dim3(64 * WN * WT),
                         argv, 0, stream);
}

template <Out O>
hipError_t plain(const F8Args& a, int cus, hipStream_t stream) {
  const int64_t large = (int64_t)((a.tokens + 255) / 256) * ((a.n + 255) / 256);
  return large >= cus ? f8_pp_launch(a, false, O == Out::F16, cus, stream) : launch<128, 128, 2, 2, 2, false, O>(a, stream);
}

}  // namespace

hipError_t f8_tiled_launch(const F8Args& a, bool gated, int dtype, int cus, hipStream_t stream) {
  if (!gated) return dtype ? plain<Out::F16>(a, cus, stream) : plain<Out::BF16>(a, cus, stream);
  const int64_t large = (int64_t)((a.tokens + 255) / 256) * ((a.n + 127) / 128);
  return large >= cus ? f8_pp_launch(a, true, dtype, cus, stream)
                      : launch<256, 64, 4, 2, 1, true, Out::BF16>(a, stream);
}

}  // namespace bsg
