// Products in E4M3 with a scale for each block of 128, in tiles of BN weight rows and BT tokens, K split over workgroups
// where there are few tiles.
//
// * K in steps of one block (128 bytes of a row).  Both operands go from memory to LDS with buffer_load_dwordx4 ... lds, in
//   STAGES stages, as many steps ahead, and fragments from LDS to registers one step ahead; one barrier per step.  A row is
//   128 bytes = 8 chunks of 16; chunk q of row R is stored at q ^ ((R >> 1) & 7), so that the fragments' reads hit distinct
//   banks.
// * Weights are the rows and tokens the columns of the matrix products; each block's product is by itself and is added by
//   vector operations with the factor sx sw, of which a lane has one per 16 tokens.  A wave's tokens' scales come with the
//   copies, the weights' are kept 64 blocks at a time, one per lane.
// * LDS rows are ordered so that a lane's results are neighbours in memory: tokens TT c + j (c = lane % 16, tile j), whose
//   scales are one read, and 8 consecutive outputs (16 bytes of 16-bit values, 64 bytes of a row per 4 lanes) or, gated,
//   all of a lane's codes of a token.
// * WIDE: codes are widened to fp16, which holds every E4M3 value, and multiplied by v_mfma_f32_16x16x32_f16: exact products,
//   sums in fp32.  Otherwise v_mfma_f32_16x16x128_f8f6f4, which aligns the products of 8 elements to the largest and drops what
//   lies 2^-13 below: 2e-6 of the sum of magnitudes for Gaussian elements, well below a rounding of bf16 or fp16, at twice the
//   rate and without the widening.  But where the results become codes, one in 400 then gets a neighbouring code; over few
//   tokens that can be 1% of an output, so the gated product of up to 64 is WIDE.  All products of plans that ask for exact ones
//   are: 61 tokens x 8192 x 8192 20.2 us for 17.5, 1003 x 2064 x 4112 37 for 28, 8192^3 1204 for 450, a feed-forward block of 33
//   tokens 40.6 for 38.4, of 128 50.9 for 39.8, of 4095 966 for 362, whose fp16 outputs are then 0.02% off for 0.15%.
// * Split K: the parts (fp32) go to the plan's workspace in the order in which the threads hold them, and the last workgroup
//   of a tile adds them in the order of the parts, so that the order of every sum is fixed.
//
// Bound: few tokens, the weights' bytes, and beside them a fixed 5 us (the launch, the first copies, the parts' join): 61 tokens
// x 8192 x 8192 in 17 to 18 us (3.8 to 4.0 TB/s), 33 tokens x 8192 x 4096 with 4 parts 11.8 to 15.7 us.  Some hundred tokens, the
// copies: 1003 tokens x 2064 x 4112 take 28.3 us (600 TFLOP/s) with 528 tiles of 64 x 64, the loop's copies alone 27.0, without
// copies 16.1, the products alone 12.9 and neither, a barrier a step, 6.9.  Of the copies' 27.0 us 7 go to lines that no L2 holds
// yet (19.9 with one block of K copied again and again), though the L2s answer 92% of the requests, in 291 cycles on average.
// Larger tiles ask for less, but there are fewer than CUs.
#include <type_traits>

#include "epilogue.h"
#include "f8_codec.h"
#include "f8_copy.h"
#include "f8_cut.h"
#include "handoff.h"

namespace bsg {
namespace {

// Tile and part of a workgroup.  Workgroups go to the 8 XCDs in turn; each XCD gets a contiguous range of tiles, token
// tiles first in groups of 8, so that those that share weights share an L2.
__device__ __forceinline__ int3 tile_of(int bid, int tiles_t, int tiles_n) {
  const int T = tiles_t * tiles_n, s = bid / T, b = bid - s * T;
  const int x = b & 7, q = T >> 3, r = T & 7;
  const int id = x * q + min(x, r) + (b >> 3);
  constexpr int GM = 8;
  const int per_group = GM * tiles_n, group = id / per_group, first = group * GM, size = min(tiles_t - first, GM);
  const int in_group = id - group * per_group;
  return make_int3(first + in_group % size, in_group / size, s);
}

template <int BN, int BT, int WN, int WT, int STAGES, int PER_CU, bool GATED, bool WIDE, Out O>
__global__ __launch_bounds__(64 * WN * WT, WN* WT* PER_CU / 4) void tiled_kernel(F8Args p) {
  constexpr int WAVES = WN * WT, THREADS = 64 * WAVES;
  constexpr int NT = BN / WN / 16, TT = BT / WT / 16;  // a wave's tiles of 16 rows and 16 tokens
  constexpr int STAGE = (BN + BT) * 128, COPIES = (BN + BT) / 8 / WAVES;
  constexpr int NS = GATED ? 2 : 1, BH = BN / NS;  // BH: outputs of a tile
  static_assert(COPIES * 8 * WAVES == BN + BT && BN % (8 * WAVES) == 0, "copies: whole instructions of one operand");
  static_assert(NT % 2 == 0 && 128 % (16 * NT) == 0 && TT <= 4, "a wave's rows share a block of scales");
  static_assert(STAGES * (STAGE + 256 * WAVES) * PER_CU <= 160 * 1024, "LDS");
  // stages, tokens' scales of each stage and wave; after the loop reused for a flag and the results' largest magnitudes.
  // (One variable: beside a second one every read of LDS waits for all copies.)
  __shared__ __attribute__((aligned(1024))) uint8_t lds[STAGES * (STAGE + 256 * WAVES)];
  uint8_t* const sc_all = lds + STAGES * STAGE;
  int* const sh_last = (int*)sc_all;
  uint32_t* const sh_most = (uint32_t*)sc_all + 64;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int c = lane & 15, g = lane >> 4;
  const int wn = wave / WT, wt = wave % WT;
  const int tiles_t = (p.tokens + BT - 1) / BT, tiles_n = (p.n + BH - 1) / BH;
  const int3 at = tile_of(blockIdx.x, tiles_t, tiles_n);
  const int t0 = at.x * BT, n0 = at.y * BH, k = p.k;
  const int tokens = min(BT, p.tokens - t0), outs = min(BH, p.n - n0);
  const int b0 = (int)((int64_t)at.z * p.kb / p.splits), b1 = (int)((int64_t)(at.z + 1) * p.kb / p.splits);

  // ---- copies: instruction i of the tile fills LDS rows 8 i .. 8 i + 7, eight lanes a row
  const __amdgpu_buffer_rsrc_t xb = __builtin_amdgcn_make_buffer_rsrc((void*)(p.x + (int64_t)t0 * p.x_stride), (short)0,
                                                                      (tokens - 1) * (int)p.x_stride + k, kRaw);
  __amdgpu_buffer_rsrc_t wb[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s)
    wb[s] = __builtin_amdgcn_make_buffer_rsrc((void*)(p.w + ((int64_t)s * p.n + n0) * k), (short)0, outs * k, kRaw);
  int voff[COPIES], kpos[COPIES];
#pragma unroll
  for (int i = 0; i < COPIES; ++i) {
    const int ins = wave + WAVES * i, R = 8 * ins + (lane >> 3);
    kpos[i] = 16 * ((lane & 7) ^ ((R >> 1) & 7));
    if (8 * ins < BN) {
      const int r = R & 15, i16 = R / 16 % NT, w = R / (16 * NT);  // tile i16 of wave row w
      const int row = GATED ? 8 * NT * w + 2 * NT * (r >> 2) + 4 * (i16 % (NT / 2)) + (r & 3)
                            : 16 * NT * w + 32 * (i16 >> 1) + 8 * (r >> 2) + 4 * (i16 & 1) + (r & 3);
      voff[i] = row * k + kpos[i];
    } else {
      const int Q = R - BN;
      voff[i] = (Q / (16 * TT) * 16 * TT + TT * (Q & 15) + Q / 16 % TT) * (int)p.x_stride + kpos[i];
    }
  }
  const int my_t = t0 + 16 * TT * wt;
  const int my_scales = max(0, min(16 * TT, p.tokens - my_t));
  // Every step has the same number of copies: those past the last have an offset past the buffers.
  auto copy_one = [&](int i, int b, int stage) __attribute__((always_inline)) {
    const bool real = b < b1;
    const int left = real ? k - 128 * b : 0, col = real ? 128 * b : 0;
    if (i == COPIES) {
      const __amdgpu_buffer_rsrc_t sb = __builtin_amdgcn_make_buffer_rsrc(
          (void*)(p.sx + min(b, p.kb - 1) * p.sx_stride + my_t), (short)0, real ? 4 * my_scales : 0, kRaw);
      copy4(sb, sc_all + (stage * WAVES + wave) * 256, 4 * lane, 0);
      return;
    }
    const int ins = wave + WAVES * i;
    // (instructions of one i are all of one operand: BN is a multiple of 8 WAVES)
    const bool weights = 8 * WAVES * i < BN;
    const bool up = GATED && weights && 8 * ins / 16 % NT >= NT / 2;
    copy16(weights ? (up ? wb[NS - 1] : wb[0]) : xb, lds + stage * STAGE + ins * 1024, kpos[i] < left ? voff[i] : kOut, col);
  };
  auto copy = [&](int b, int stage) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i <= COPIES; ++i) copy_one(i, b, stage);
  };
  const float* sw[NS];
  float sw_lane[NS];
#pragma unroll
  for (int s = 0; s < NS; ++s) sw[s] = p.sw + ((int64_t)s * f8_blocks(p.n) + min(n0 + BH / WN * wn, p.n - 1) / 128) * p.kb;
  auto load_sw = [&](int b) __attribute__((always_inline)) {
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      sw_lane[s] = sw[s][min(b + lane, p.kb - 1)];
      asm volatile("s_waitcnt vmcnt(0)" : "+v"(sw_lane[s])::"memory");  // (so that no wait is left in the loop)
    }
  };

  v4f acc[NT][TT];
#pragma unroll
  for (int i = 0; i < NT; ++i)
#pragma unroll
    for (int j = 0; j < TT; ++j) acc[i][j] = v4f{0, 0, 0, 0};
  const int f = (c >> 1) & 7, ch0 = 16 * (g ^ f), ch1 = 16 * ((g + 4) ^ f);
  // A step's fragments are read a step ahead, into the other of two sets of registers.
  struct Frags {
    v4i x[TT][2], w[NT][2];
    float sx[TT];
  } set[2];
  auto read = [&](Frags& q, int stage) __attribute__((always_inline)) {
    const uint8_t* tile = lds + stage * STAGE;
    const float* sc = (const float*)(sc_all + (stage * WAVES + wave) * 256) + TT * c;
#pragma unroll
    for (int j = 0; j < TT; ++j) {
      const uint8_t* row = tile + (BN + 16 * (TT * wt + j) + c) * 128;
      q.x[j][0] = *(const v4i*)(row + ch0);
      q.x[j][1] = *(const v4i*)(row + ch1);
      q.sx[j] = sc[j];
    }
#pragma unroll
    for (int i = 0; i < NT; ++i) {
      const uint8_t* row = tile + (16 * (NT * wn + i) + c) * 128;
      q.w[i][0] = *(const v4i*)(row + ch0);
      q.w[i][1] = *(const v4i*)(row + ch1);
    }
  };
  // `also(i)`, i = 0 .. COPIES, is called between the products
  auto multiply = [&](const Frags& q, int b, auto also) __attribute__((always_inline)) {
    float fct[NS][TT];
#pragma unroll
    for (int s = 0; s < NS; ++s) {
      const float one = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, sw_lane[s]), (b - b0) & 63));
#pragma unroll
      for (int j = 0; j < TT; ++j) fct[s][j] = q.sx[j] * one;
    }
    auto add = [&](int i, int j, v4f y) __attribute__((always_inline)) {
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(fct[GATED && i >= NT / 2][j], y[e], acc[i][j][e]);
    };
    if constexpr (WIDE) {
      v8h x[TT][4];
#pragma unroll
      for (int j = 0; j < TT; ++j) f8_widen(q.x[j][0], q.x[j][1], x[j]);
#pragma unroll
      for (int i = 0; i < NT; ++i) {
#pragma unroll
        for (int u = i * (COPIES + 1) / NT; u < (i + 1) * (COPIES + 1) / NT; ++u) also(u);
        v8h w[4];
        f8_widen(q.w[i][0], q.w[i][1], w);
        v4f y[TT];
#pragma unroll
        for (int u = 0; u < 4; ++u)
#pragma unroll
          for (int j = 0; j < TT; ++j)
            y[j] = __builtin_amdgcn_mfma_f32_16x16x32_f16(w[u], x[j][u], u ? y[j] : v4f{0, 0, 0, 0}, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < TT; ++j) add(i, j, y[j]);
      }
    } else {
      auto join = [](const v4i v[2]) { return v8i{v[0][0], v[0][1], v[0][2], v[0][3], v[1][0], v[1][1], v[1][2], v[1][3]}; };
      v4f y[NT * TT];
#pragma unroll
      for (int q2 = 0; q2 < NT * TT + 2; ++q2) {
        if (q2 < NT * TT) {
          y[q2] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(join(q.w[q2 / TT]), join(q.x[q2 % TT]), v4f{0, 0, 0, 0}, 0, 0, 0,
                                                                  0, 0, 0);
          __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
#pragma unroll
          for (int u = q2 * (COPIES + 1) / (NT * TT); u < (q2 + 1) * (COPIES + 1) / (NT * TT); ++u) {
            also(u);
            __builtin_amdgcn_sched_group_barrier(0x010, 1, 0);
          }
        }
        if (q2 >= 2) {
          add((q2 - 2) / TT, (q2 - 2) % TT, y[q2 - 2]);
          __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
        }
      }
      // (this empty asm that reads the sums keeps their additions here: put off, they need registers for every product)
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < TT; ++j) asm volatile("" ::"v"(acc[i][j]));
    }
  };
  // at most N copies in flight (those of later steps), LDS reads done, everyone here
  auto arrive = [](auto n) __attribute__((always_inline)) {
    asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)\n\ts_barrier" ::"n"(decltype(n)::value) : "memory");
  };
  constexpr int N = COPIES + 1;
  load_sw(b0);
#pragma unroll
  for (int d = 0; d < STAGES; ++d) copy(b0 + d, d);
  arrive(std::integral_constant<int, (STAGES - 1) * N>{});
  read(set[0], 0);
  int stage = 0;
  // Step b: the next step's copies have landed and everyone has read this step's stage, which is copied into.
  auto step = [&](const Frags& now, Frags& next, int b) __attribute__((always_inline)) {
    __builtin_amdgcn_sched_barrier(0);
    arrive(std::integral_constant<int, (STAGES - 2) * N>{});
    const int old = stage;
    stage = stage == STAGES - 1 ? 0 : stage + 1;
    read(next, stage);
    __builtin_amdgcn_sched_barrier(0);  // (left alone, the reads come last, and the next step waits for them)
    multiply(now, b, [&](int i) __attribute__((always_inline)) { copy_one(i, b + STAGES, old); });
    if (((b + 1 - b0) & 63) == 0) load_sw(b + 1);
  };
  int b = b0;
  for (; b + 2 <= b1; b += 2) {
    step(set[0], set[1], b);
    step(set[1], set[0], b + 1);
  }
  if (b < b1) multiply(set[0], b, [](int) {});
  asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");

  // ---- parts
  if (p.splits > 1) {
    const int tile = at.y * tiles_t + at.x;
    const __amdgpu_buffer_rsrc_t parts =
        handoff_buffer(p.part, (uint32_t)(tiles_t * tiles_n * p.splits) * (BN * BT * 4u));
    auto at_part = [&](int s, int r) { return (uint32_t)((tile * p.splits + s) * (BN * BT) + (r * THREADS + tid) * 4); };
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < TT; ++j) handoff_store4(parts, at_part(at.z, i * TT + j), acc[i][j]);
    if (!last_arrival(p.arrived + tile, p.splits, sh_last)) return;
    v4f sum[NT][TT];
    for (int s = 0; s < p.splits; ++s) {
      v4f y[NT][TT];
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < TT; ++j) y[i][j] = handoff_load4(parts, at_part(s, i * TT + j));
#pragma unroll
      for (int i = 0; i < NT; ++i)
#pragma unroll
        for (int j = 0; j < TT; ++j) sum[i][j] = s ? sum[i][j] + y[i][j] : y[i][j];
    }
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < TT; ++j) acc[i][j] = sum[i][j];
  }

  // ---- results
  if constexpr (GATED) {
    constexpr int H = NT / 2;
    for (int i = tid; i < BT; i += THREADS) sh_most[i] = 0;
    __syncthreads();
#pragma unroll
    for (int j = 0; j < TT; ++j) {
      uint32_t most = 0;
#pragma unroll
      for (int i = 0; i < H; ++i)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float h = f8_gated(acc[i][j][e], acc[H + i][j][e]);  // (a scalar: bits of a vector's element are its first's)
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
      for (int i = 0; i < H; ++i) q[i] = f8_not_finite(most) ? kF8Nan : f8_codes4(acc[i][j], s);
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

// More tiles than a grid may have (its threads are below 2^32; K is then not split) are done a range of tokens at a time.
template <F8Way WAY, int WN, int WT, int STAGES, bool WIDE, Out O>
hipError_t launch(F8Args a, const F8Cut& cut, hipStream_t stream) {
  constexpr F8Shape t = f8_shape(WAY);
  constexpr int THREADS = 64 * WN * WT;
  const int64_t tokens = a.tokens, at_once = f8_tokens_at_once(WAY, a.n, THREADS);
  a.splits = (int)cut.splits;
  for (int64_t first = 0;; first += at_once) {
    a.tokens = (int)(tokens - first < at_once ? tokens - first : at_once);
    const int64_t tiles = f8_tiles(t.rows, t.tokens, t.gated, a.tokens, a.n);
    void* argv[] = {&a};
    const hipError_t e = hipLaunchKernel((const void*)&tiled_kernel<t.rows, t.tokens, WN, WT, STAGES, t.per_cu, t.gated, WIDE, O>,
                                         dim3((unsigned)(tiles * cut.splits)), dim3(THREADS), argv, 0, stream);
    if (e != hipSuccess || first + at_once >= tokens) return e;
    a.x += at_once * a.x_stride;
    a.sx += at_once;
    a.out += at_once * a.out_stride * (t.gated ? 1 : 2);
    if (t.gated) a.so += at_once;
  }
}

template <Out O>
hipError_t plain(const F8Args& a, const F8Cut& cut, hipStream_t stream) {
  switch (cut.way) {
    case F8Way::T64x32: return launch<F8Way::T64x32, 2, 2, 4, false, O>(a, cut, stream);
    case F8Way::T64x64: return launch<F8Way::T64x64, 2, 2, 3, false, O>(a, cut, stream);
    case F8Way::T128x64: return launch<F8Way::T128x64, 4, 1, 3, false, O>(a, cut, stream);
    case F8Way::T64x32Wide: return launch<F8Way::T64x32Wide, 2, 2, 4, true, O>(a, cut, stream);
    case F8Way::T64x64Wide: return launch<F8Way::T64x64Wide, 2, 2, 3, true, O>(a, cut, stream);
    case F8Way::T128x128Wide: return launch<F8Way::T128x128Wide, 2, 4, 4, true, O>(a, cut, stream);
    default: return launch<F8Way::T128x128, 2, 4, 4, false, O>(a, cut, stream);
  }
}

}  // namespace

hipError_t f8_tiled_launch(const F8Args& a, bool gated, int dtype, int cus, hipStream_t stream) {
  const F8Cut cut = f8_cut(gated, a.exact != 0, a.tokens, a.n, a.k, cus);
  constexpr Out C = Out::BF16;  // (gated results are codes)
  switch (cut.way) {
    case F8Way::T256x256:
    case F8Way::G256x256: return f8_pp_launch(a, gated, dtype, cus, stream);
    case F8Way::G256x32Wide: return launch<F8Way::G256x32Wide, 4, 1, 4, true, C>(a, cut, stream);
    case F8Way::G256x64Wide: return launch<F8Way::G256x64Wide, 4, 2, 3, true, C>(a, cut, stream);
    case F8Way::G256x64: return launch<F8Way::G256x64, 4, 2, 3, false, C>(a, cut, stream);
    case F8Way::G256x128: return launch<F8Way::G256x128, 4, 2, 3, false, C>(a, cut, stream);
    default: return dtype ? plain<Out::F16>(a, cut, stream) : plain<Out::BF16>(a, cut, stream);
  }
}

}  // namespace bsg
