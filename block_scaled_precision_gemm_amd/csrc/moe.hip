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
// Decoded weights are exact: E2M1 * E4M3 has at most 6 significant bits, E4M3 * 2^e has 4.  MXFP8
// weights decode to bf16, whose exponents hold any E8M0 scale.  NVFP4 weights decode to fp16 for the
// first product (one conversion and one packed multiply for two values) and x enters it in fp16, bf16
// rows scaled by a power of two each; for the second product, whose activations have no known range
// before all of them are there, they decode to bf16.  SiLU(gate) up is held as two bf16 parts (16
// significant bits, so its rounding is far below the output's), as is fp16 x beside MXFP8 weights; each
// part is one more product per weight fragment.
//
// Three launches: the router must know every token's choice before weights can be read, and the second
// product needs all of an expert's SiLU(gate) up.
#include "codec.h"
#include "handoff.h"
#include "moe.h"

namespace bsg {
namespace {

typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));

constexpr int kSlab = 128;

template <bool F16>
__device__ __forceinline__ v4f mfma(v4i a, v4i b, v4f c) {
  if constexpr (F16)
    return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, a), __builtin_bit_cast(v8h, b), c, 0, 0, 0);
  else
    return __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(v8b, a), __builtin_bit_cast(v8b, b), c, 0, 0, 0);
}

__device__ __forceinline__ uint16_t bf16_bits(float x) { return __builtin_bit_cast(uint16_t, (__bf16)x); }
__device__ __forceinline__ float bf16_value(uint16_t b) { return __builtin_bit_cast(float, (uint32_t)b << 16); }

// ------------------------------------------------------------------------------------------- router
constexpr int kRouterThreads = 1024, kRouterWaves = kRouterThreads / 64;
constexpr int kMaxChoices = BSG_MOE_MAX_TOKENS * BSG_MOE_MAX_TOP_K;
constexpr float kLog2e = 1.44269504088896341f;

// Order of floats as unsigned: larger float, larger key; NaN above all; -0 as 0.  No logit's key is 0.
__device__ __forceinline__ uint32_t order_key(float x) {
  if (x != x) return 0xFFFFFFFFu;
  const uint32_t u = __builtin_bit_cast(uint32_t, x + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float key_value(uint32_t k) {
  return __builtin_bit_cast(float, k & 0x80000000u ? k & 0x7FFFFFFFu : ~k);
}

template <int CTRL, int ROW_MASK>
__device__ __forceinline__ uint32_t dpp(uint32_t x) {
  return (uint32_t)__builtin_amdgcn_update_dpp(0, (int)x, CTRL, ROW_MASK, 0xF, false);
}
// Largest of the wave's keys, in every lane (lanes without a source see 0).
__device__ __forceinline__ uint32_t wave_max(uint32_t x) {
  x = max(x, dpp<0x111, 0xF>(x));  // shift right within rows of 16 lanes by 1, 2, 4, 8
  x = max(x, dpp<0x112, 0xF>(x));
  x = max(x, dpp<0x114, 0xF>(x));
  x = max(x, dpp<0x118, 0xF>(x));
  x = max(x, dpp<0x142, 0xA>(x));  // lane 15 of rows 0 and 2 to rows 1 and 3
  x = max(x, dpp<0x143, 0xC>(x));  // lane 31 to rows 2 and 3
  return (uint32_t)__builtin_amdgcn_readlane((int)x, 63);
}
__device__ __forceinline__ float wave_sum(float x) {
#pragma unroll
  for (int o = 32; o > 0; o >>= 1) x += __shfl_xor(x, o);
  return x;
}

struct Choice {  // in LDS
  unsigned long long tokens_of[BSG_MOE_MAX_EXPERTS];  // bit t: token t chose the expert
  int first_row[BSG_MOE_MAX_EXPERTS];
  int chosen[kMaxChoices];  // expert and weight of each choice: tokens in order, ranks in order
  float weight[kMaxChoices];
  int sums[2 * kRouterWaves];
};
static_assert(BSG_MOE_MAX_TOKENS <= 64, "a bit for each token");
static_assert(kMaxChoices <= kRouterThreads && BSG_MOE_MAX_EXPERTS <= kRouterThreads, "one thread for each");
static_assert(BSG_MOE_MAX_TOP_K <= 64, "a lane for each of a token's choices");

// Top k of every token and the tokens of every expert; one workgroup.  A wave takes a token: lane i
// holds the logits of experts R i .. R i + R - 1, and k times the largest is found and taken out (of
// equal ones the lowest lane's and its lowest).  A choice's row follows from the bits of the tokens that
// chose its expert.
template <int R>
__device__ void choose(const MoeArgs& p, Choice& sh) {
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int E = p.experts, K = p.top_k, T = p.tokens, choices = T * K;
  if (tid < E) sh.tokens_of[tid] = 0;
  __syncthreads();
  for (int t = wave; t < T; t += kRouterWaves) {
    uint32_t key[R];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int e = lane * R + r;
      const float x = handoff_load(p.logits + (size_t)t * E + min(e, E - 1));
      key[r] = e < E ? order_key(x) : 0u;
    }
    float all = 0.0f, mine = 0.0f;
    uint32_t top = 0;
    int expert = 0;
    for (int k = 0; k < K; ++k) {
      uint32_t best = key[0];
#pragma unroll
      for (int r = 1; r < R; ++r) best = max(best, key[r]);
      const uint32_t most = wave_max(best);
      const int owner = __builtin_ctzll(__ballot(best == most));
      if (k == 0) {
        top = most;
        if (p.keep) {  // the sum over all experts, before any is taken out
          float s = 0.0f;
#pragma unroll
          for (int r = 0; r < R; ++r)
            if (key[r]) s += __builtin_amdgcn_exp2f((key_value(key[r]) - key_value(top)) * kLog2e);
          all = wave_sum(s);
        }
      }
      int place = 0;
      bool taken = lane != owner;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const bool hit = !taken && key[r] == most;
        place = hit ? r : place;
        key[r] = hit ? 0u : key[r];
        taken |= hit;
      }
      const int e = owner * R + __builtin_amdgcn_readlane(place, owner);
      if (lane == k) {
        expert = e;
        mine = __builtin_amdgcn_exp2f((key_value(most) - key_value(top)) * kLog2e);
      }
    }
    const float sum = p.keep ? all : wave_sum(mine);
    if (lane < K) {
      const int c = t * K + lane;
      sh.chosen[c] = expert;
      sh.weight[c] = mine / sum;
      atomicOr(&sh.tokens_of[expert], 1ull << t);
    }
  }
  __syncthreads();
  // rows of each expert, and its slots of up to slot_rows rows: a scan over the experts
  const int count = tid < E ? __popcll(sh.tokens_of[tid]) : 0, mine = (count + p.slot_rows - 1) / p.slot_rows;
  int rows = count, slots = mine;
#pragma unroll
  for (int o = 1; o < 64; o <<= 1) {
    const int a = __shfl_up(rows, o), b = __shfl_up(slots, o);
    if (lane >= o) rows += a, slots += b;
  }
  if (lane == 63) sh.sums[wave] = rows, sh.sums[kRouterWaves + wave] = slots;
  __syncthreads();
#pragma unroll
  for (int w = 0; w < kRouterWaves; ++w)
    if (w < wave) rows += sh.sums[w], slots += sh.sums[kRouterWaves + w];
  if (tid < E) {
    sh.first_row[tid] = rows - count;
    for (int k = 0; k < mine; ++k)
      p.slots[slots - mine + k] = int4{tid, rows - count + k * p.slot_rows, min(count - k * p.slot_rows, p.slot_rows), 0};
  }
  if (tid == kRouterThreads - 1) *p.active = slots;
  __syncthreads();
  if (tid < choices) {
    const int t = tid / K, e = sh.chosen[tid];
    const float w = sh.weight[tid];
    const int row = sh.first_row[e] + __popcll(sh.tokens_of[e] & ((1ull << t) - 1));
    p.row_token[row] = t;
    p.row_weight[row] = w;
    p.row_of[tid] = row;
    if (p.ids) p.ids[tid] = e;
    if (p.weights) p.weights[tid] = w;
  }
}

// The form in which the first product takes x: as it is, bf16 rows as fp16 scaled by a power of two each
// (NVFP4 weights decode to fp16 in half the operations of bf16), or fp16 rows as two bf16 parts (MXFP8
// weights need bf16's range).
enum class Prep { kNone, kScaled, kParts };
template <bool NV, bool F16>
constexpr Prep kPrep = NV ? (F16 ? Prep::kNone : Prep::kScaled) : (F16 ? Prep::kParts : Prep::kNone);

// One token's row, by a whole workgroup.
template <Prep PREP>
__device__ __forceinline__ void prepare_row(const MoeArgs& p, int t, uint32_t* shared) {
  const int tid = threadIdx.x;
  const uint16_t* x = p.x + t * p.x_stride;
  uint16_t* dst = p.xs + (int64_t)t * p.hidden;
  float scale = 1.0f;
  v4i w = {0, 0, 0, 0};
  if constexpr (PREP == Prep::kScaled) {
    uint32_t most = 0;  // largest magnitude, as bits
    for (int i = 8 * tid; i < p.hidden; i += 8 * kRouterThreads) {
      w = *(const v4i*)(x + i);
#pragma unroll
      for (int k = 0; k < 4; ++k) most = max(most, max((uint32_t)w[k] & 0x7FFFu, ((uint32_t)w[k] >> 16) & 0x7FFFu));
    }
    most = wave_max(most);
    if ((tid & 63) == 0) shared[tid >> 6] = most;
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kRouterWaves; ++k) most = max(most, shared[k]);
    // largest magnitude to [2^7, 2^8): exact in fp16 down to 2^-32 of it, and products with decoded
    // weights (below 2^4) stay far inside fp32; rows with an infinity or a NaN are left as they are
    const int e = (int)(most >> 7) - 127, up = e > 127 ? 0 : max(7 - e, -110);
    if (tid == 0) p.x_exp[t] = up;
    scale = __builtin_amdgcn_ldexpf(1.0f, min(up, 127));  // (rows of bf16 subnormals: short of it, still exact)
    if (up > 127 && tid == 0) p.x_exp[t] = 127;
  }
  for (int i = 8 * tid; i < p.hidden; i += 8 * kRouterThreads) {
    if (PREP != Prep::kScaled || p.hidden > 8 * kRouterThreads) w = *(const v4i*)(x + i);  // else still held
    v4i hi, lo;
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t u = (uint32_t)w[k];
      if constexpr (PREP == Prep::kScaled) {
        const v2f f = {__builtin_bit_cast(float, u << 16) * scale, __builtin_bit_cast(float, u & 0xFFFF0000u) * scale};
        hi[k] = __builtin_bit_cast(int, __builtin_convertvector(f, v2h));
      } else {
        const v2h v = __builtin_bit_cast(v2h, u);
        const float f0 = (float)v[0], f1 = (float)v[1];
        const uint16_t h0 = bf16_bits(f0), h1 = bf16_bits(f1);
        const bool fin0 = __builtin_fabsf(f0) < 65536.0f, fin1 = __builtin_fabsf(f1) < 65536.0f;  // else no low part
        hi[k] = h0 | h1 << 16;
        lo[k] = (fin0 ? bf16_bits(f0 - bf16_value(h0)) : 0) | (fin1 ? bf16_bits(f1 - bf16_value(h1)) : 0) << 16;
      }
    }
    *(v4i*)(dst + i) = hi;
    if constexpr (PREP == Prep::kParts) *(v4i*)(dst + (int64_t)p.tokens * p.hidden + i) = lo;
  }
}

// Workgroups 0 .. tiles - 1: the logits of one tile of 16 experts and 16 tokens, the waves taking
// alternate steps of 32 k, kBatch of them in flight; the last of these workgroups to finish chooses.  The
// others prepare one token's row each.
template <bool NV, bool F16>
__global__ __launch_bounds__(kRouterThreads) void router_kernel(MoeArgs p) {
  __shared__ union {
    float part[kRouterWaves][64][4];
    Choice choice;
    uint32_t most[kRouterWaves];
  } sh;
  __shared__ int last;
  constexpr int kBatch = 8;
  const int tiles_e = (p.experts + 15) / 16, tiles = tiles_e * ((p.tokens + 15) / 16);
  if ((int)blockIdx.x >= tiles) {
    if constexpr (kPrep<NV, F16> != Prep::kNone) prepare_row<kPrep<NV, F16>>(p, blockIdx.x - tiles, sh.most);
    return;
  }
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, c = lane & 15, g = lane >> 4;
  const int e0 = blockIdx.x % tiles_e * 16, t0 = blockIdx.x / tiles_e * 16;
  const uint16_t* a = p.router + (size_t)min(e0 + c, p.experts - 1) * p.hidden + 8 * g;
  const uint16_t* b = p.x + (int64_t)min(t0 + c, p.tokens - 1) * p.x_stride + 8 * g;
  v4f acc = {0, 0, 0, 0};
  const int steps = p.hidden / 32;
  for (int s0 = wave; s0 < steps; s0 += kRouterWaves * kBatch) {
    v4i aw[kBatch], bw[kBatch];
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const int s = min(s0 + k * kRouterWaves, steps - 1);
      aw[k] = *(const v4i*)(a + 32 * s);
      bw[k] = *(const v4i*)(b + 32 * s);
    }
#pragma unroll
    for (int k = 0; k < kBatch; ++k) {
      const bool in = s0 + k * kRouterWaves < steps;  // repeated steps count as zero
      aw[k] = in ? aw[k] : v4i{0, 0, 0, 0};
      bw[k] = in ? bw[k] : v4i{0, 0, 0, 0};
      acc = mfma<F16>(aw[k], bw[k], acc);
    }
  }
  *(v4f*)sh.part[wave][lane] = acc;
  __syncthreads();
  if (wave == 0) {
    v4f s = *(v4f*)sh.part[0][lane];
#pragma unroll
    for (int w = 1; w < kRouterWaves; ++w) s += *(v4f*)sh.part[w][lane];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (t0 + c < p.tokens && e0 + 4 * g + i < p.experts)
        handoff_store(p.logits + (size_t)(t0 + c) * p.experts + e0 + 4 * g + i, s[i]);
  }
  if (!last_arrival(p.arrived, tiles, &last)) return;
  if (p.experts <= 64) choose<1>(p, sh.choice);
  else if (p.experts <= 128) choose<2>(p, sh.choice);
  else choose<BSG_MOE_MAX_EXPERTS / 64>(p, sh.choice);
}

// ------------------------------------------------------------------------------------------- weights
constexpr int kThreads = 256;

// How codes become fragments of a product.
enum class Dec { kNvF16, kNvBf16, kMxBf16 };

template <Dec DEC>
struct Codes {
  static constexpr bool NV = DEC != Dec::kMxBf16, F16 = DEC == Dec::kNvF16;
  static constexpr int kBlock = NV ? 16 : 32;                   // elements per scale
  static constexpr int kSlabBytes = NV ? kSlab / 2 : kSlab;     // code bytes of a slab of a row
  static constexpr int kSlabScales = kSlab / kBlock;
  static constexpr int kRegs = NV ? 4 : 8;
  static constexpr int kDepth = 2;                              // slabs of weights in flight
};

// A lane's 32 codes of one row.
template <Dec DEC>
struct Row {
  using C = Codes<DEC>;
  uint32_t q[C::kRegs];
  __device__ __forceinline__ void load(const uint8_t* w) {
    const v4i a = *(const v4i*)w;
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = (uint32_t)a[i];
    if constexpr (!C::NV) {
      const v4i b = *(const v4i*)(w + 16);
#pragma unroll
      for (int i = 0; i < 4; ++i) q[4 + i] = (uint32_t)b[i];
    }
  }
  __device__ __forceinline__ void clear() {
#pragma unroll
    for (int i = 0; i < C::kRegs; ++i) q[i] = 0;
  }
  // Fragment j of four; `s`: the two scale codes of the 32 elements (NVFP4), or the one.
  __device__ __forceinline__ v4i fragment(int j, uint32_t s) const {
    if constexpr (DEC == Dec::kNvF16) {  // times 2^-8 (codec.h)
      const uint32_t s2 = e4m3x2_scale_f16x2(s);
      return e2m1x8_scaled_f16x8(q[j], j < 2 ? f16x2_splat_lo(s2) : f16x2_splat_hi(s2));
    } else if constexpr (DEC == Dec::kNvBf16) {
      const float f = j < 2 ? __builtin_amdgcn_cvt_f32_fp8((int)s, 0) : __builtin_amdgcn_cvt_f32_fp8((int)s, 1);
      const v2f a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[j], 1.0f, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[j], 1.0f, 1);
      const v2f c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[j], 1.0f, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q[j], 1.0f, 3);
      // products of at most 6 significant bits: their upper halves are the bf16 values
      auto pair = [&](float x, float y) {
        return (int)__builtin_amdgcn_perm(__builtin_bit_cast(uint32_t, y * f), __builtin_bit_cast(uint32_t, x * f), 0x07060302u);
      };
      const float a0 = a[0], a1 = a[1], b0 = b[0], b1 = b[1], c0 = c[0], c1 = c[1], d0 = d[0], d1 = d[1];
      return v4i{pair(a0, a1), pair(b0, b1), pair(c0, c1), pair(d0, d1)};
    } else {
      const float f = __builtin_bit_cast(float, s << 23);
      const int lo = (int)q[2 * j], hi = (int)q[2 * j + 1];
      return v4i{__builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, f, false)),
                 __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, f, true)),
                 __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, f, false)),
                 __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, f, true))};
    }
  }
};

// Scale codes of a workgroup's rows for kChunk k at a time, in LDS: read from memory a row's codes are
// a few bytes per slab in 16 rows at once, and those reads cost more than the codes' (gate/up of 33
// tokens, 64 experts of 4096 x 2048 in NVFP4: 191 us with them, 155 us with constant scales).  Rows are
// padded so that the 16 rows of a tile lie in different banks.
constexpr int kChunk = 4096;
template <Dec DEC, int TILES>
struct Scales {
  static constexpr int kRowBytes = kChunk / Codes<DEC>::kBlock, kPitch = kRowBytes + (Codes<DEC>::NV ? 8 : 4);
  uint8_t rows[TILES * 16][kPitch];
};

// Copy the codes of chunk k0 .. k0 + n - 1 of tiles whose first rows start at sc[m].
template <Dec DEC, int TILES>
__device__ __forceinline__ void stage_scales(Scales<DEC, TILES>& sh, const uint8_t* const sc[TILES], int K, int k0, int n, int tid) {
  const int row_bytes = K / Codes<DEC>::kBlock, first = k0 / Codes<DEC>::kBlock, bytes = n / Codes<DEC>::kBlock;
  auto copy = [&](auto unit) {
    using U = decltype(unit);
    const int per_row = bytes / (int)sizeof(U);
#pragma unroll
    for (int m = 0; m < TILES; ++m)
#pragma unroll 2
      for (int i = tid; i < 16 * per_row; i += kThreads) {
        const int r = i / per_row, at = (i - r * per_row) * (int)sizeof(U);
        const U v = *(const U*)(sc[m] + r * row_bytes + first + at);
        __builtin_memcpy(&sh.rows[16 * m + r][at], &v, sizeof(U));
      }
  };
  if (row_bytes % 8 == 0) copy(uint2{});  // (chunks start at multiples of 8 codes; scales are 4-byte aligned at least)
  else if constexpr (Codes<DEC>::NV) copy(uint16_t{});
  else copy(uint8_t{});
}

// acc[tile][nt] += rows x columns: tile m's 16 rows start at w[m] (codes) and sc[m] (scales), the lane's
// column is at b[nt], PARTS parts `part` elements apart.  Slabs of 128 k go to the four waves in turn.
template <Dec DEC, int TILES, int NT, int PARTS>
__device__ __forceinline__ void products(Scales<DEC, TILES>& sh, const uint8_t* const w[TILES], const uint8_t* const sc[TILES],
                                         int K, int tid, int wave, const uint16_t* const b[NT], int64_t part, int nts,
                                         v4f acc[TILES][NT]) {
  using C = Codes<DEC>;
  constexpr int DEPTH = C::kDepth;
  static_assert(DEPTH % 2 == 0, "the activations' buffers alternate");
  const int lane = tid & 63, c = lane & 15, g = lane >> 4;
  const int row_bytes = C::NV ? K / 2 : K;
  const uint32_t at0 = c * row_bytes + g * (C::kSlabBytes / 4);
  Row<DEC> buf[DEPTH][TILES];
  v4i x[2][PARTS][NT][4];
  auto fetch = [&](Row<DEC>* r, int s) {
#pragma unroll
    for (int m = 0; m < TILES; ++m) r[m].load(w[m] + (at0 + (uint32_t)s * C::kSlabBytes));
  };
  auto fetch_x = [&](v4i (*v)[NT][4], int s) {
#pragma unroll
    for (int q = 0; q < PARTS; ++q)
#pragma unroll
      for (int n = 0; n < NT; ++n)
        if (n < nts) {
#pragma unroll
          for (int j = 0; j < 4; ++j) v[q][n][j] = *(const v4i*)(b[n] + q * part + s * kSlab + 32 * g + 8 * j);
        }
  };
  auto multiply = [&](const Row<DEC>* r, const v4i (*v)[NT][4], int chunk_slab) {
#pragma unroll
    for (int m = 0; m < TILES; ++m) {
      const uint8_t* codes = &sh.rows[16 * m + c][chunk_slab * C::kSlabScales + g * (C::kSlabScales / 4)];
      const uint32_t s = C::NV ? (uint32_t)*(const uint16_t*)codes : (uint32_t)*codes;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const v4i a = r[m].fragment(j, s);
#pragma unroll
        for (int n = 0; n < NT; ++n)
          if (n < nts) {
#pragma unroll
            for (int q = 0; q < PARTS; ++q) acc[m][n] = mfma<C::F16>(a, v[q][n][j], acc[m][n]);
          }
      }
    }
  };
  for (int k0 = 0; k0 < K; k0 += kChunk) {
    const int n = min(kChunk, K - k0), first = k0 / kSlab, full = first + n / kSlab;
    const int s1 = first + wave;
#pragma unroll
    for (int d = 0; d < DEPTH; ++d)
      if (s1 + 4 * d < full) fetch(buf[d], s1 + 4 * d);
    if (s1 < full) fetch_x(x[0], s1);
    if (k0) __syncthreads();
    stage_scales<DEC, TILES>(sh, sc, K, k0, n, tid);
    __syncthreads();
    for (int s0 = s1; s0 < full; s0 += 4 * DEPTH) {
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) {
        const int s = s0 + 4 * d;
        if (s < full) {
          if (s + 4 < full) fetch_x(x[(d + 1) & 1], s + 4);
          multiply(buf[d], x[d & 1], s - first);
          if (s + 4 * DEPTH < full) fetch(buf[d], s + 4 * DEPTH);
        }
      }
    }
    if (n % kSlab && wave == full % 4) {  // the rest: lanes past the end count as zero
      const bool in = full * kSlab + 32 * g < K;
#pragma unroll
      for (int m = 0; m < TILES; ++m) buf[0][m].clear();
#pragma unroll
      for (int q = 0; q < PARTS; ++q)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int j = 0; j < 4; ++j) x[0][q][nt][j] = v4i{0, 0, 0, 0};
      if (in) {
        fetch_x(x[0], full);
        fetch(buf[0], full);
      } else {
        // their scales are whatever LDS holds: zero them, so that no NaN comes of it
#pragma unroll
        for (int m = 0; m < TILES; ++m)
#pragma unroll
          for (int i = 0; i < C::kSlabScales / 4; ++i)
            sh.rows[16 * m + c][(full - first) * C::kSlabScales + g * (C::kSlabScales / 4) + i] = 0;
      }
      multiply(buf[0], x[0], full - first);
    }
  }
}

// Workgroup (x, slot): SiLU(gate) up of dims 32x .. 32x+31 for the tokens of the slot's expert.
template <bool NV, bool F16, int NT>
__global__ __launch_bounds__(kThreads, NT > 1 ? 1 : NV ? 3 : 2) void gate_up_kernel(MoeArgs p) {
  constexpr int TILES = 4;  // gate rows 0..15, 16..31, up rows 0..15, 16..31
  constexpr Dec DEC = NV ? Dec::kNvF16 : Dec::kMxBf16;
  constexpr Prep PREP = kPrep<NV, F16>;
  constexpr int PARTS = PREP == Prep::kParts ? 2 : 1;
  __shared__ union {
    Scales<DEC, TILES> scales;
    v4f acc[4][TILES][NT][64];
  } sh;
  const int4 slot = p.slots[blockIdx.y];
  if ((int)blockIdx.y >= *p.active) return;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, c = lane & 15;
  const int e = __builtin_amdgcn_readfirstlane(slot.x), start = __builtin_amdgcn_readfirstlane(slot.y);
  const int count = __builtin_amdgcn_readfirstlane(slot.z);
  const int nts = (count + 15) / 16, i0 = blockIdx.x * 32;
  const uint8_t *w[TILES], *sc[TILES];
#pragma unroll
  for (int m = 0; m < TILES; ++m) {
    const int64_t row = (int64_t)e * 2 * p.inter + (m < 2 ? 0 : p.inter) + i0 + (m & 1) * 16;
    w[m] = p.w13 + row * (NV ? p.hidden / 2 : p.hidden);
    sc[m] = p.s13 + row * (NV ? p.hidden / 16 : p.hidden / 32);
  }
  const uint16_t* b[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const int t = p.row_token[start + min(16 * n + c, count - 1)];
    b[n] = PREP == Prep::kNone ? p.x + t * p.x_stride : p.xs + (int64_t)t * p.hidden;
  }
  v4f acc[TILES][NT] = {};
  products<DEC, TILES, NT, PARTS>(sh.scales, w, sc, p.hidden, tid, wave, b, (int64_t)p.tokens * p.hidden, nts, acc);
  __syncthreads();  // the scales are done with
#pragma unroll
  for (int m = 0; m < TILES; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) sh.acc[wave][m][n][lane] = acc[m][n];
  __syncthreads();
  const float alpha = p.alpha13 ? p.alpha13[e] : 1.0f;
  const int64_t rows = (int64_t)p.tokens * p.top_k;
  for (int k = tid; k < 2 * nts * 64; k += kThreads) {
    const int l = k & 63, m = (k >> 6) & 1, n = k >> 7, col = 16 * n + (l & 15), i = i0 + 16 * m + 4 * (l >> 4);
    v4f gate = sh.acc[0][m][n][l], up = sh.acc[0][m + 2][n][l];
#pragma unroll
    for (int w = 1; w < 4; ++w) gate += sh.acc[w][m][n][l], up += sh.acc[w][m + 2][n][l];
    if (col >= count || i >= p.inter) continue;
    // powers of two that the operands carry: decoded weights 2^-8, scaled rows of x 2^x_exp
    const int back = (NV ? 8 : 0) - (PREP == Prep::kScaled ? p.x_exp[p.row_token[start + col]] : 0);
    uint16_t hi[4], lo[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float x = alpha * __builtin_amdgcn_ldexpf(gate[r], back), u = alpha * __builtin_amdgcn_ldexpf(up[r], back);
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
__global__ __launch_bounds__(kThreads, NT > 1 ? 1 : NV ? 3 : 2) void down_kernel(MoeArgs p) {
  constexpr int TILES = 4;
  constexpr Dec DEC = NV ? Dec::kNvBf16 : Dec::kMxBf16;
  __shared__ union {
    Scales<DEC, TILES> scales;
    v4f acc[4][TILES][NT][64];
  } sh;
  __shared__ int last;
  const int active = *p.active;
  const int4 slot = p.slots[blockIdx.y];
  if ((int)blockIdx.y >= active) return;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, c = lane & 15;
  const int e = __builtin_amdgcn_readfirstlane(slot.x), start = __builtin_amdgcn_readfirstlane(slot.y);
  const int count = __builtin_amdgcn_readfirstlane(slot.z);
  const int nts = (count + 15) / 16, d0 = blockIdx.x * 64;
  const uint8_t *w[TILES], *sc[TILES];
#pragma unroll
  for (int m = 0; m < TILES; ++m) {
    const int64_t row = (int64_t)e * p.hidden + min(d0 + 16 * m, p.hidden - 16);  // (tiles past the end repeat the last)
    w[m] = p.w2 + row * (NV ? p.inter / 2 : p.inter);
    sc[m] = p.s2 + row * (NV ? p.inter / 16 : p.inter / 32);
  }
  const uint16_t* b[NT];
#pragma unroll
  for (int n = 0; n < NT; ++n) b[n] = p.h + (int64_t)(start + min(16 * n + c, count - 1)) * p.inter;
  v4f acc[TILES][NT] = {};
  products<DEC, TILES, NT, 2>(sh.scales, w, sc, p.inter, tid, wave, b, (int64_t)p.tokens * p.top_k * p.inter, nts, acc);
  __syncthreads();  // the scales are done with
#pragma unroll
  for (int m = 0; m < TILES; ++m)
#pragma unroll
    for (int n = 0; n < NT; ++n) sh.acc[wave][m][n][lane] = acc[m][n];
  __syncthreads();
  const float alpha = p.alpha2 ? p.alpha2[e] : 1.0f;
  // (a few tokens' rows: far below 2^31 bytes)
  const __amdgpu_buffer_rsrc_t ybuf = handoff_buffer(p.y, (uint32_t)(p.tokens * p.top_k) * (uint32_t)p.hidden * 4u);
  for (int k = tid; k < TILES * nts * 64; k += kThreads) {
    const int l = k & 63, m = (k >> 6) % TILES, n = (k >> 6) / TILES, col = 16 * n + (l & 15), d = d0 + 16 * m + 4 * (l >> 4);
    v4f y = sh.acc[0][m][n][l];
#pragma unroll
    for (int w = 1; w < 4; ++w) y += sh.acc[w][m][n][l];
    if (col >= count || d >= p.hidden) continue;
    handoff_store4(ybuf, (uint32_t)(start + col) * p.hidden + d, y * (alpha * p.row_weight[start + col]));
  }
  if (!last_arrival(p.arrived + 1 + blockIdx.x, active, &last)) return;
  for (int k = tid; k < p.tokens * 16; k += kThreads) {
    const int t = k >> 4, d = d0 + 4 * (k & 15);
    if (d >= p.hidden) continue;
    v4f y = {0, 0, 0, 0};
    for (int j0 = 0; j0 < p.top_k; j0 += 8) {
      v4f v[8];
#pragma unroll
      for (int j = 0; j < 8; ++j)  // all in flight
        v[j] = handoff_load4(ybuf, (uint32_t)p.row_of[t * p.top_k + min(j0 + j, p.top_k - 1)] * p.hidden + d);
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (j0 + j < p.top_k) y += v[j];
    }
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
  const unsigned tiles = (a.experts + 15) / 16 * ((a.tokens + 15) / 16);
  hipError_t e = hipLaunchKernel((const void*)&router_kernel<NV, F16>,
                                 dim3(tiles + (kPrep<NV, F16> != Prep::kNone ? a.tokens : 0)), dim3(kRouterThreads), argv, 0,
                                 stream);
  if (e != hipSuccess) return e;
  // at most one slot per choice, and one per expert and slot_rows choices
  const int choices = a.tokens * a.top_k, bound = a.experts + choices / a.slot_rows;
  const unsigned slots = choices < bound ? choices : bound;
  e = hipLaunchKernel((const void*)&gate_up_kernel<NV, F16, NT>, dim3((a.inter + 31) / 32, slots), dim3(kThreads),
                      argv, 0, stream);
  if (e != hipSuccess) return e;
  return hipLaunchKernel((const void*)&down_kernel<NV, F16, NT>, dim3((a.hidden + 63) / 64, slots), dim3(kThreads), argv, 0,
                         stream);
}

template <bool NV, bool F16>
hipError_t launch_nt(const MoeArgs& a, hipStream_t stream) {
  return a.slot_rows == 16 ? launch<NV, F16, 1>(a, stream) : launch<NV, F16, 2>(a, stream);
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
  a->xs = (uint16_t*)take(2 * T * p.hidden * 2);
  a->x_exp = (int*)take(T * 4);
  a->h = (uint16_t*)take(2 * rows * p.inter * 2);
  a->y = (float*)take(rows * p.hidden * 4);
  a->active = (int*)take(4);
  a->slots = (int4*)take((p.experts + rows / 16 + 1) * sizeof(int4));
  a->row_token = (int*)take(rows * 4);
  a->row_weight = (float*)take(rows * 4);
  a->row_of = (int*)take(rows * 4);
  *counters_at = at;
  *counters_bytes = (1 + ((size_t)p.hidden + 63) / 64) * 4;
  a->arrived = (int*)take(*counters_bytes);
  return at;
}

}  // namespace bsg
