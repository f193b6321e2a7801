// Products in E4M3 with a scale for each block of 128, for many tokens and large weights: tiles of 256 weight rows and 256
// tokens, eight waves, two per SIMD.
//
// * Wave 4 g + s (g = group, s = SIMD) owns weight rows 128 g .. 128 g + 127 of the tile and tokens 64 s .. 64 s + 63: 8 x 4
//   accumulators of 16 x 16 (128 registers).  A group's rows are one block of the weights' scales.
// * Each product of a block of 128 is by itself (v_mfma_f32_16x16x128_f8f6f4 with a third operand of zero) and added by
//   vector operations with the factor sx sw, of which a lane has one for its token of each 16: a product takes the matrix
//   unit 32 cycles, its four additions take 16 of the vector unit.  A result is added two products after its own, when it
//   has arrived, a phase's last two in the wave's next memory phase (456 us with a wait for them, 441 without).
// * The two waves of a SIMD alternate between a memory phase (fragments of the next half of the wave's rows from LDS,
//   copies) and a compute phase (16 products, 512 cycles).  Group 1 starts one phase late, so one group computes while the
//   other moves data; one barrier per phase keeps them in step.  The tiled kernel's loop, in which both waves of a SIMD
//   read and multiply at the same times, took 577 us for 8192^3, this one 441 us (2490 TFLOP/s).
// * Memory to LDS by buffer_load_dwordx4 ... lds, two stages of 128 bytes of K, a quarter of the next one in every memory
//   phase.  A row is 8 chunks of 16 bytes; chunk q of row R is stored at q ^ ((R >> 1) & 7), so that the 16 lanes of a
//   fragment's read hit distinct banks.  Rows are ordered as in the tiled kernel, so that a lane's results are neighbours.
//   Copies past K, and of rows past the last, have an offset beyond the buffer: zeros, no traffic.
// * Workgroups go to the 8 XCDs in turn; each XCD gets a contiguous range of tiles, walked in groups of 8 rows of tiles,
//   so that what runs at once shares operands in its L2.  At most one workgroup per CU, looping over its tiles.
//
// The matrix instruction aligns the products of 8 elements to the largest and drops what lies 2^-13 below: 2e-6 of the sum of
// magnitudes for Gaussian elements, well below a rounding of bf16 or fp16.  Widening the codes to fp16 instead halves its rate;
// plans that ask for exact products have that (f8_tiled.hip).
#include <type_traits>

#include "epilogue.h"
#include "f8_codec.h"
#include "f8_copy.h"

namespace bsg {
namespace {

constexpr int BN = 256, BT = 256, BK = 128, NT = 8, TT = 4, WAVES = 8, THREADS = 64 * WAVES;
constexpr int TILE = 256 * BK;                // bytes of one operand's stage
constexpr int SCALES = 4 * TILE;               // LDS: weights' stages, tokens' stages, then tokens' scales
constexpr int SCALE_STAGE = WAVES * 64 * 4;   // each wave's own 64
constexpr int CPW = 4;                        // copy instructions of a wave in a memory phase

__device__ __forceinline__ void barrier_only() { asm volatile("s_barrier" ::: "memory"); }

// At most N loads in flight, then the barrier.
template <int N>
__device__ __forceinline__ void loads_barrier() {
  asm volatile("s_waitcnt vmcnt(%0)\n\ts_barrier" ::"n"(N) : "memory");
}

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

template <bool GATED, Out O>
__global__ __launch_bounds__(THREADS, 2) void pp_kernel(F8Args p) {
  constexpr int NS = GATED ? 2 : 1, BH = BN / NS;  // BH: outputs of a tile
  __shared__ __attribute__((aligned(1024))) uint8_t lds[SCALES + 2 * SCALE_STAGE];
  // (one variable, reused for the results' largest magnitudes: beside a second one every read of LDS waits for all copies)
  uint32_t* const sh_most = (uint32_t*)(lds + SCALES);
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int grp = wave >> 2, ws = wave & 3, c = lane & 15, g = lane >> 4;
  const int tiles_t = (p.tokens + BT - 1) / BT, tiles_n = (p.n + BH - 1) / BH, k = p.k, KT = p.kb;
  const int xs = (int)p.x_stride;
#pragma unroll 1
  for (int vb = blockIdx.x; vb < tiles_t * tiles_n; vb += gridDim.x) {
    const int2 at = tile_of(vb, tiles_t, tiles_n);
    const int t0 = at.x * BT, n0 = at.y * BH;
    const int tokens = min(BT, p.tokens - t0), outs = min(BH, p.n - n0);

    // ---- copies.  Operand 0: weights, whose LDS rows 128 g .. are read by group g only; operand 1: tokens.  In the memory
    // phase of a wave's first half, group g copies rows 0 .. 127 of operand g, in that of its second half rows 128 .. 255 of
    // the other.  Of each 128 rows, wave s of the group copies LDS rows 32 s + 8 q + lane / 8, q < 4.
    const __amdgpu_buffer_rsrc_t xb =
        __builtin_amdgcn_make_buffer_rsrc((void*)(p.x + (int64_t)t0 * p.x_stride), (short)0, (tokens - 1) * xs + k, kRaw);
    // (gated: of each group's 128 rows the first 64 are gate's, the others up's)
    const __amdgpu_buffer_rsrc_t wb = __builtin_amdgcn_make_buffer_rsrc(
        (void*)(p.w + ((int64_t)(GATED && ws >= 2 ? p.n : 0) + n0) * k), (short)0, outs * k, kRaw);
    const __amdgpu_buffer_rsrc_t first = grp == 0 ? wb : xb, second = grp == 0 ? xb : wb;
    int voff[2][CPW], kpos[2];
#pragma unroll
    for (int q = 0; q < CPW; ++q) {
      const int R = 32 * ws + 8 * q + (lane >> 3), r = R & 15, i = R / 16;
      const int chunk = 16 * ((lane & 7) ^ ((R >> 1) & 7));
      if (q < 2) kpos[q] = chunk;
      auto weight_row = [&](int half) {
        return GATED ? 64 * half + 16 * (r >> 2) + 4 * (i & 3) + (r & 3)
                     : 128 * half + 32 * (i >> 1) + 8 * (r >> 2) + 4 * (i & 1) + (r & 3);
      };
      auto token_row = [&](int half) { return 128 * half + R / 64 * 64 + 4 * (R & 15) + (R / 16 & 3); };
      voff[0][q] = (grp == 0 ? weight_row(0) * k : token_row(0) * xs) + chunk;
      voff[1][q] = (grp == 0 ? token_row(1) * xs : weight_row(1) * k) + chunk;
    }
    uint8_t* const dst0 = lds + grp * 2 * TILE + 32 * ws * BK;
    uint8_t* const dst1 = lds + (1 - grp) * 2 * TILE + (128 + 32 * ws) * BK;
    auto copy_quarter = [&](auto sc, auto hc, int kt) __attribute__((always_inline)) {
      constexpr int stage = decltype(sc)::value, half = decltype(hc)::value;
      uint8_t* dst = (half ? dst1 : dst0) + stage * TILE;
      const int left = k - BK * kt, col = kt < KT ? BK * kt : 0;  // (left <= 0 past the last)
#pragma unroll
      for (int q = 0; q < CPW; ++q)
        copy16(half ? second : first, dst + q * 8 * BK, kpos[q & 1] < left ? voff[half][q] : kOut, col);
    };
    // the scales of the wave's tokens, for itself
    const int my_t = t0 + 64 * ws, my_tokens = max(0, min(64, p.tokens - my_t));
    uint8_t* const sc_lds = lds + SCALES + wave * 256;
    auto copy_scales = [&](auto sc, int kt) __attribute__((always_inline)) {
      constexpr int stage = decltype(sc)::value;
      const __amdgpu_buffer_rsrc_t sb = __builtin_amdgcn_make_buffer_rsrc(
          (void*)(p.sx + min(kt, KT - 1) * p.sx_stride + my_t), (short)0, 4 * my_tokens, kRaw);
      copy4(sb, sc_lds + stage * SCALE_STAGE, 4 * lane, 0);
    };
    // the weights' scales of 64 K tiles, one per lane
    const float* sw[NS];
    float sw_lane[NS];
#pragma unroll
    for (int s = 0; s < NS; ++s)
      sw[s] = p.sw + ((int64_t)s * f8_blocks(p.n) + min(n0 + (GATED ? 0 : 128 * grp), p.n - 1) / 128) * KT;
    auto load_sw = [&](int kt) __attribute__((always_inline)) {
#pragma unroll
      for (int s = 0; s < NS; ++s) {
        sw_lane[s] = sw[s][min(kt + lane, KT - 1)];
        asm volatile("s_waitcnt vmcnt(0)" : "+v"(sw_lane[s])::"memory");  // (so that no wait is left in the loop)
      }
    };

    const int f = (c >> 1) & 7, ch0 = 16 * (g ^ f), ch1 = 16 * ((g + 4) ^ f);
    const uint8_t* const w_lds = lds + (128 * grp + c) * BK;
    const uint8_t* const x_lds = lds + 2 * TILE + (64 * ws + c) * BK;
    v8i wf[4], xf[TT];
    v4f xsc;
    auto frag = [&](const uint8_t* row) {
      const v4i lo = *(const v4i*)(row + ch0), hi = *(const v4i*)(row + ch1);
      return v8i{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    };
    auto read_frags = [&](auto sc, auto hc) __attribute__((always_inline)) {
      constexpr int stage = decltype(sc)::value, half = decltype(hc)::value;
      if constexpr (half == 0) {
        xsc = *(const v4f*)(sc_lds + stage * SCALE_STAGE + 16 * c);
#pragma unroll
        for (int j = 0; j < TT; ++j) xf[j] = frag(x_lds + stage * TILE + j * 16 * BK);
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) wf[i] = frag(w_lds + stage * TILE + (4 * half + i) * 16 * BK);
    };

    v4f acc[NT][TT];
#pragma unroll
    for (int i = 0; i < NT; ++i)
#pragma unroll
      for (int j = 0; j < TT; ++j) acc[i][j] = v4f{0, 0, 0, 0};

    using I0 = std::integral_constant<int, 0>;
    using I1 = std::integral_constant<int, 1>;
    load_sw(0);
    copy_quarter(I0{}, I0{}, 0);
    copy_quarter(I0{}, I1{}, 0);
    copy_scales(I0{}, 0);
    loads_barrier<0>();
    if (grp == 1) barrier_only();

    // One memory and one compute phase: rows 64 half .. of the wave's rows, K tile kt.  With phases 4 h .. 4 h + 3 those of
    // K tile t (group 0 reads at 4 h and 4 h + 2 and computes at 4 h + 1 and 4 h + 3, group 1 one later), group 0 reads the
    // next K tile at 4 h + 4, group 1 at 4 h + 5; weight rows 128 .. 255 are read by group 1 only.  Waits, before the barrier
    // that ends a phase: group 0 drains its copies after computing its second half (4 h + 3); group 1 drains those of its
    // first half at the end of its second memory phase (4 h + 3), and all after computing the second half (4 h + 4).  The
    // stage copied into was last read by group 0 at 4 h - 2 and by group 1 at 4 h - 1, before either copies into what the
    // other reads (group 0: tokens 128 .. 255 at 4 h + 2; group 1: tokens 0 .. 127 at 4 h + 1).
    float fct[TT];
    v4f late[2];  // the last two products of a compute phase, added in the next memory phase
#pragma unroll
    for (int j = 0; j < TT; ++j) fct[j] = 0.0f;
    late[0] = late[1] = v4f{0, 0, 0, 0};
    auto add = [&](int i, int j, v4f y) __attribute__((always_inline)) {
#pragma unroll
      for (int e = 0; e < 4; ++e) acc[i][j][e] = __builtin_fmaf(fct[j], y[e], acc[i][j][e]);
    };
    auto step = [&](auto sc, auto hc, int kt) __attribute__((always_inline)) {
      constexpr int stage = decltype(sc)::value, half = decltype(hc)::value;
      __builtin_amdgcn_sched_barrier(0);
      read_frags(sc, hc);
      copy_quarter(std::integral_constant<int, stage ^ 1>{}, hc, kt + 1);
      if constexpr (half == 1) copy_scales(std::integral_constant<int, stage ^ 1>{}, kt + 1);
      add(4 * (half ^ 1) + 3, 2, late[0]);
      add(4 * (half ^ 1) + 3, 3, late[1]);
      asm volatile("" ::"v"(acc[4 * (half ^ 1) + 3][2]), "v"(acc[4 * (half ^ 1) + 3][3]));  // (not later)
      __builtin_amdgcn_sched_barrier(0);
      asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
      if (half == 0 || GATED) {
        const float b = __builtin_bit_cast(
            float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, sw_lane[GATED ? half : 0]), kt & 63));
#pragma unroll
        for (int j = 0; j < TT; ++j) fct[j] = xsc[j] * b;
      }
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (half == 1) {
        if (grp == 1) loads_barrier<CPW + 1>();
        else barrier_only();
      } else {
        barrier_only();
      }
      __builtin_amdgcn_sched_barrier(0);
      __builtin_amdgcn_s_setprio(1);
      v4f y[4 * TT];
#pragma unroll
      for (int q = 0; q < 4 * TT; ++q) {
        y[q] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(wf[q / TT], xf[q % TT], v4f{0, 0, 0, 0}, 0, 0, 0, 0, 0, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        if (q >= 2) {
          add(4 * half + (q - 2) / TT, (q - 2) % TT, y[q - 2]);
          __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
        }
      }
      late[0] = y[4 * TT - 2];
      late[1] = y[4 * TT - 1];
      // (this empty asm that reads the results keeps them in this phase: they could sink past the barriers)
#define BSG_ROW(i) "v"(acc[4 * half + i][0]), "v"(acc[4 * half + i][1]), "v"(acc[4 * half + i][2]), "v"(acc[4 * half + i][3])
      asm volatile("" ::BSG_ROW(0), BSG_ROW(1), BSG_ROW(2), "v"(acc[4 * half + 3][0]), "v"(acc[4 * half + 3][1]), "v"(late[0]),
                   "v"(late[1]));
#undef BSG_ROW
      __builtin_amdgcn_s_setprio(0);
      __builtin_amdgcn_sched_barrier(0);
      if constexpr (half == 1) loads_barrier<0>();
      else barrier_only();
    };
    int kt = 0;
    auto refresh = [&] {
      if ((kt & 63) == 0) load_sw(kt);
    };
    for (; kt + 2 <= KT;) {
      step(I0{}, I0{}, kt);
      step(I0{}, I1{}, kt);
      ++kt;
      step(I1{}, I0{}, kt);
      step(I1{}, I1{}, kt);
      ++kt;
      refresh();
    }
    if (kt < KT) {
      step(I0{}, I0{}, kt);
      step(I0{}, I1{}, kt);
    }
    // Group 0 catches up with group 1's last compute phase; every wave has then drained its copies and reads.
    __builtin_amdgcn_sched_barrier(0);
    add(NT - 1, 2, late[0]);
    add(NT - 1, 3, late[1]);
    if (grp == 0) barrier_only();
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)\n\ts_barrier" ::: "memory");

    // ---- results
    if constexpr (GATED) {
      for (int i = tid; i < BT; i += THREADS) sh_most[i] = 0;
      __syncthreads();
#pragma unroll
      for (int j = 0; j < TT; ++j) {
        uint32_t most = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            const float h = f8_gated(acc[i][j][e], acc[4 + i][j][e]);  // (a scalar: bits of a vector's element are its first's)
            acc[i][j][e] = h;
            most = max(most, __builtin_bit_cast(uint32_t, h) & 0x7FFFFFFFu);
          }
        atomicMax(&sh_most[64 * ws + TT * c + j], most);
      }
      __syncthreads();
      uint32_t of_token[TT];
#pragma unroll
      for (int j = 0; j < TT; ++j) of_token[j] = sh_most[64 * ws + TT * c + j];
      __syncthreads();  // (the next tile's first copies of scales, which no other barrier precedes, go where these lay)
      const int n = n0 + 64 * grp + 16 * g;
#pragma unroll
      for (int j = 0; j < TT; ++j) {
        const int t = 64 * ws + TT * c + j;
        const uint32_t most = of_token[j];
        const float s = f8_scale(most);
        v4i q;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          q[i] = f8_not_finite(most) ? kF8Nan : f8_codes4(acc[i][j], s);
        }
        if (t < tokens) {
          if (n < p.n) *(v4i*)(p.out + (int64_t)(t0 + t) * p.out_stride + n) = q;
          if (grp == 0 && g == 0) p.so[(int64_t)(n0 / 128) * p.so_stride + t0 + t] = s;
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < NT; i += 2) {
        const int n = n0 + 128 * grp + 16 * i + 8 * g;
        if (n >= p.n) continue;
        float bias[8];
#pragma unroll
        for (int e = 0; e < 8; ++e) bias[e] = p.bias ? p.bias[n + e] : 0.0f;
#pragma unroll
        for (int j = 0; j < TT; ++j) {
          const int t = 64 * ws + TT * c + j;
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
}

template <bool GATED, Out O>
hipError_t launch(F8Args a, int cus, hipStream_t stream) {
  constexpr int BH = BN / (GATED ? 2 : 1);
  void* argv[] = {&a};
  const int64_t tiles = (int64_t)((a.tokens + BT - 1) / BT) * ((a.n + BH - 1) / BH);
  return hipLaunchKernel((const void*)&pp_kernel<GATED, O>, dim3((unsigned)(tiles < cus ? tiles : cus)), dim3(THREADS), argv, 0,
                         stream);
}

}  // namespace

hipError_t f8_pp_launch(const F8Args& a, bool gated, int dtype, int cus, hipStream_t stream) {
  if (gated) return launch<true, Out::BF16>(a, cus, stream);
  return dtype ? launch<false, Out::F16>(a, cus, stream) : launch<false, Out::BF16>(a, cus, stream);
}

}  // namespace bsg
