// Mixture-of-experts layer for few tokens: router, gate/up with SiLU, down with the weighted sum.
//
// Few tokens read many weights, so the layer is bound by the bytes of the chosen experts' weights,
// and every kernel streams weight rows through registers into v_mfma_f32_16x16x32: rows of weights are
// the product's first operand (16 rows), tokens the second (16 columns, unused ones zero).  A lane loads
// the codes of 32 consecutive k of one row (16 bytes of E2M1, 32 of E4M3) and uses them in four products;
// the k order of a product is free, and the tokens' operand follows it.  A workgroup's waves take alternate
// slabs of 128 k and are summed through LDS.
//
// Decoded weights are exact: E2M1 * E4M3 has at most 6 significant bits, E4M3 * 2^e has 4.  MXFP8
// weights decode to bf16, whose exponents hold any E8M0 scale.  NVFP4 weights decode to fp16 for the
// first product (one conversion and one packed multiply for two values) and x enters it in fp16, bf16
// rows scaled by a power of two each; for the second product, whose activations have no known range
// before all of them are there, they decode to bf16.  SiLU(gate) up is held as two bf16 parts (16
// significant bits, so its rounding is far below the output's), as is fp16 x beside MXFP8 weights; each
// part is one more product per weight fragment.
//
// Measured (weights read per product's time): 33 tokens, 64 experts of (4096, 2048), 8 chosen, NVFP4: router 14 us,
// gate/up 126 us (4.8 TB/s), down 91 us (3.3 TB/s; without arithmetic 115 and 69 us); one token 4, 18 and 15 us;
// 7 tokens, 16 experts of (2048, 4096), 2 chosen, MXFP8: 8, 40 and 29 us.
//
// Three launches: the router must know every token's choice before weights can be read, and the second
// product needs all of an expert's SiLU(gate) up.
#include <type_traits>

#include "codec.h"
#include "handoff.h"
#include "moe.h"

namespace bsg {
namespace {

typedef __bf16 v8b __attribute__((ext_vector_type(8)));
typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));

constexpr int kSlab = 128;
constexpr int kSlotRows = 16;  // rows of a slot: the columns of a product

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
constexpr int kRouterParts = 4;  // most parts that the logits' sums are cut into

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

// The top k of one token, by a wave: lane i holds the logits x of experts R i .. R i + R - 1 (the last
// expert's again beyond it), and k times the largest is found and taken out (of equal ones the lowest
// lane's, and its lowest).  Lane i ends with the expert of rank i and its weight (i < K); the last rank
// looked for is `last`.
template <int R>
__device__ __forceinline__ void top_k(const float x[R], int E, int last, bool keep, int lane, int& expert, float& weight) {
  uint32_t key[R];
#pragma unroll
  for (int r = 0; r < R; ++r) key[r] = lane * R + r < E ? order_key(x[r]) : 0u;
  float all = 0.0f;
  uint32_t top = 0;
  uint32_t mine = 0;
  expert = 0;
  for (int k = 0; k <= last; ++k) {
    uint32_t best = key[0];
#pragma unroll
    for (int r = 1; r < R; ++r) best = max(best, key[r]);
    const uint32_t most = wave_max(best);
    const int owner = __builtin_ctzll(__ballot(best == most));
    if (k == 0) {
      top = most;
      if (keep) {  // the sum over all experts, before any is taken out
        float s = 0.0f;
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (key[r]) s += __builtin_amdgcn_exp2f((key_value(key[r]) - key_value(top)) * kLog2e);
        all = wave_sum(s);
      }
    }
    int place = 0;
    if constexpr (R == 1) {
      key[0] = lane == owner ? 0u : key[0];
    } else {
      bool taken = lane != owner;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const bool hit = !taken && key[r] == most;
        place = hit ? r : place;
        key[r] = hit ? 0u : key[r];
        taken |= hit;
      }
      place = __builtin_amdgcn_readlane(place, owner);
    }
    expert = lane == k ? owner * R + place : expert;
    mine = lane == k ? most : mine;
  }
  weight = lane <= last ? __builtin_amdgcn_exp2f((key_value(mine) - key_value(top)) * kLog2e) : 0.0f;
  weight /= keep ? all : wave_sum(weight);
}

// Top k of every token and the tokens of every expert; one workgroup, a wave for each token.  A choice's
// row follows from the bits of the tokens that chose its expert.
template <int R>
__device__ void choose(const MoeArgs& p, Choice& sh) {
  const int tid = threadIdx.x, lane = tid & 63, wave = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int E = p.experts, K = p.top_k, T = p.tokens, choices = T * K;
  constexpr int N = BSG_MOE_MAX_TOKENS / kRouterWaves;
  float x[N][R];  // the logits of all of the wave's tokens, in flight together
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (wave + i * kRouterWaves < T) {
#pragma unroll
      for (int r = 0; r < R; ++r)
        x[i][r] = handoff_load(p.logits + (size_t)(wave + i * kRouterWaves) * E + min(lane * R + r, E - 1));
    }
  for (int part = 1; part < p.router_parts; ++part)
#pragma unroll
    for (int i = 0; i < N; ++i)
      if (wave + i * kRouterWaves < T) {
#pragma unroll
        for (int r = 0; r < R; ++r)
          x[i][r] += handoff_load(p.logits + (size_t)(part * T + wave + i * kRouterWaves) * E + min(lane * R + r, E - 1));
      }
  if (tid < E) sh.tokens_of[tid] = 0;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const int t = wave + i * kRouterWaves;
    if (t >= T) break;
    int expert;
    float weight;
    top_k<R>(x[i], E, K - 1, p.keep, lane, expert, weight);
    if (lane < K) {
      const int c = t * K + lane;
      sh.chosen[c] = expert;
      sh.weight[c] = weight;
      atomicOr(&sh.tokens_of[expert], 1ull << t);
    }
  }
  __syncthreads();
  // rows of each expert, and its slots of up to kSlotRows rows: a scan over the experts
  const int count = tid < E ? __popcll(sh.tokens_of[tid]) : 0, mine = (count + kSlotRows - 1) / kSlotRows;
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
      p.slots[slots - mine + k] = int4{tid, rows - count + k * kSlotRows, min(count - k * kSlotRows, kSlotRows), 0};
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

// The form in which the first product takes x, in rows without gaps: as it is, bf16 rows as fp16 scaled
// by a power of two each (NVFP4 weights decode to fp16 in half the operations of bf16), or fp16 rows as
// two bf16 parts (MXFP8 weights need bf16's range).
enum class Prep { kAsIs, kScaled, kParts };
template <bool NV, bool F16>
constexpr Prep kPrep = NV ? (F16 ? Prep::kAsIs : Prep::kScaled) : (F16 ? Prep::kParts : Prep::kAsIs);

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
    // Largest magnitude to [2^7, 2^8): fp16's steps are then 2^-31 of it and less, all 8 bits of an element are kept
    // down to 2^-24 of it, and products with decoded weights (below 2^4) stay far inside fp32.  (Rows of bf16 subnormals:
    // short of it, still exact.  Rows with an infinity or a NaN: as if their largest were 2^127.)
    const int up = min(7 - min((int)(most >> 7) - 127, 127), 127);
    if (tid == 0) p.x_exp[t] = up;
    scale = __builtin_amdgcn_ldexpf(1.0f, up);
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
      } else if constexpr (PREP == Prep::kAsIs) {
        hi[k] = (int)u;
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

// The first workgroups: a part of the sums of one tile of 16 experts and 16 tokens' logits, the waves taking
// alternate steps of 32 k, up to eight of them in flight; the last of these workgroups to finish chooses.  The
// others prepare one token's row each.
template <bool NV, bool F16>
__global__ __launch_bounds__(kRouterThreads) void router_kernel(MoeArgs p) {
  __shared__ union {
    float part[kRouterWaves][64][4];
    Choice choice;
    uint32_t most[kRouterWaves];
  } sh;
  __shared__ int last;
  const int tiles_e = (p.experts + 15) / 16, tiles = tiles_e * ((p.tokens + 15) / 16), logits = tiles * p.router_parts;
  if ((int)blockIdx.x >= logits) {
    prepare_row<kPrep<NV, F16>>(p, blockIdx.x - logits, sh.most);
    return;
  }
  const int tid = threadIdx.x, wave = tid >> 6, lane = tid & 63, c = lane & 15, g = lane >> 4;
  const int tile = blockIdx.x % tiles, part = blockIdx.x / tiles;
  const int e0 = tile % tiles_e * 16, t0 = tile / tiles_e * 16;
  const uint16_t* a = p.router + (size_t)min(e0 + c, p.experts - 1) * p.hidden + 8 * g;
  const uint16_t* b = p.x + (int64_t)min(t0 + c, p.tokens - 1) * p.x_stride + 8 * g;
  v4f acc = {0, 0, 0, 0};
  const int all = p.hidden / 32, each = (all + p.router_parts - 1) / p.router_parts;
  const int steps = min(all, (part + 1) * each);
  int s0 = part * each + wave;
  auto batch = [&](auto size) __attribute__((always_inline)) {
    constexpr int B = decltype(size)::value;
    v4i aw[B], bw[B];
#pragma unroll
    for (int k = 0; k < B; ++k) {
      const int s = min(s0 + k * kRouterWaves, steps - 1);
      aw[k] = *(const v4i*)(a + 32 * s);
      bw[k] = *(const v4i*)(b + 32 * s);
    }
#pragma unroll
    for (int k = 0; k < B; ++k) {
      const bool in = s0 + k * kRouterWaves < steps;  // repeated steps count as zero
      aw[k] = in ? aw[k] : v4i{0, 0, 0, 0};
      bw[k] = in ? bw[k] : v4i{0, 0, 0, 0};
      acc = mfma<F16>(aw[k], bw[k], acc);
    }
    s0 += B * kRouterWaves;
  };
  // (always eight at once repeated steps of short rows: 6.9 us for one token, 32 experts, hidden 1024, 3.5 us so)
  while (s0 + 4 * kRouterWaves < steps) batch(std::integral_constant<int, 8>{});
  if (s0 + 2 * kRouterWaves < steps) batch(std::integral_constant<int, 4>{});
  if (s0 < steps) batch(std::integral_constant<int, 2>{});
  *(v4f*)sh.part[wave][lane] = acc;
  __syncthreads();
  if (wave == 0) {
    v4f s = *(v4f*)sh.part[0][lane];
#pragma unroll
    for (int w = 1; w < kRouterWaves; ++w) s += *(v4f*)sh.part[w][lane];
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (t0 + c < p.tokens && e0 + 4 * g + i < p.experts)
        handoff_store(p.logits + (size_t)(part * p.tokens + t0 + c) * p.experts + e0 + 4 * g + i, s[i]);
  }
  if (p.tokens == 1 || !last_arrival(p.arrived, logits, &last)) return;  // (one token: gate_up_kernel chooses)
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

// Copy the codes of chunk k0 .. k0 + n - 1 of tiles whose first rows start at sc[m]: 16 threads a row.
template <Dec DEC, int TILES>
__device__ __forceinline__ void stage_scales(Scales<DEC, TILES>& sh, const uint8_t* const sc[TILES], int K, int k0, int n, int tid) {
  const int row_bytes = K / Codes<DEC>::kBlock, bytes = n / Codes<DEC>::kBlock, r = tid >> 4;
  const uint32_t first = r * row_bytes + k0 / Codes<DEC>::kBlock;
  auto copy = [&](auto unit) {
    using U = decltype(unit);
    for (int at = (tid & 15) * (int)sizeof(U); at < bytes; at += 16 * (int)sizeof(U)) {
      U v[TILES];
#pragma unroll
      for (int m = 0; m < TILES; ++m) v[m] = *(const U*)(sc[m] + first + at);
#pragma unroll
      for (int m = 0; m < TILES; ++m) __builtin_memcpy(&sh.rows[16 * m + r][at], &v[m], sizeof(U));
    }
  };
  // whole rows of 8 codes keep every row at 4 bytes or better (scales are 4-byte aligned), chunks start
  // at multiples of 8 codes
  if (row_bytes % 8 == 0) copy(uint2{});
  else if constexpr (Codes<DEC>::NV) copy(uint16_t{});
  else copy(uint8_t{});
}

// A wave's slab of the activations in LDS: 16 columns of 128 k, padded so that the 16 lanes of a fragment
// read lie in different banks.  Read straight from memory in fragment order each lane would touch a
// line of its own four times over (64 lines in each of four loads, against 64 of all the weights').
constexpr int kXPitch = 2 * kSlab + 16;
struct Slab {
  uint8_t at[4][16 * kXPitch];  // [wave]; parts of the activations follow each other in it
};

// acc[tile] += rows x columns: tile m's 16 rows start at w[m] (codes) and sc[m] (scales); the columns are
// rows of `x` (bf16 or fp16, K long), column i's at byte column[i] (of the lane's columns 4 i + lane / 16;
// kNoColumn: none, zeros), part q `part` bytes further.  Slabs of 128 k go to the four waves in turn.
constexpr uint32_t kNoColumn = 0x80000000u;
template <Dec DEC, int TILES, int PARTS>
__device__ __forceinline__ void products(Scales<DEC, TILES>& sh, Slab& slab, const uint8_t* const w[TILES],
                                         const uint8_t* const sc[TILES], int K, int tid, int wave, const void* x,
                                         uint32_t x_bytes, const uint32_t column[4], uint32_t part, v4f acc[TILES]) {
  using C = Codes<DEC>;
  const int lane = tid & 63, c = lane & 15, g = lane >> 4;
  const uint32_t at0 = c * (C::NV ? K / 2 : K) + g * (C::kSlabBytes / 4);
  const __amdgpu_buffer_rsrc_t xbuf = handoff_buffer(x, x_bytes);
  Row<DEC> rows[TILES];  // the next slab's weights
  v4u_t raw[PARTS][4];
  auto fetch = [&](int s) {
#pragma unroll
    for (int m = 0; m < TILES; ++m) rows[m].load(w[m] + (at0 + (uint32_t)s * C::kSlabBytes));
  };
  auto fetch_x = [&](int s) {
    const uint32_t k = s * kSlab + 8 * c;  // the lane's 8 k of each of its columns
#pragma unroll
    for (int q = 0; q < PARTS; ++q)
#pragma unroll
      for (int i = 0; i < 4; ++i)  // beyond the buffer: zeros, and no memory access
        raw[q][i] = __builtin_amdgcn_raw_buffer_load_b128(xbuf, (int)(k < (uint32_t)K ? column[i] + 2 * k + q * part : kNoColumn), 0, 0);
  };
  auto multiply = [&](int chunk_slab, int next) {
    v4i v[PARTS][4];
#pragma unroll
    for (int q = 0; q < PARTS; ++q) {  // (one wave's LDS accesses are in order: the fences only keep them so)
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
#pragma unroll
      for (int i = 0; i < 4; ++i) *(v4u_t*)&slab.at[wave][(4 * i + g) * kXPitch + 16 * c] = raw[q][i];
      __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
      __builtin_amdgcn_wave_barrier();
#pragma unroll
      for (int j = 0; j < 4; ++j) v[q][j] = *(const v4i*)&slab.at[wave][c * kXPitch + 64 * g + 16 * j];
    }
    fetch_x(next);
    uint32_t s[TILES];
#pragma unroll
    for (int m = 0; m < TILES; ++m) {
      const uint8_t* codes = &sh.rows[16 * m + c][chunk_slab * C::kSlabScales + g * (C::kSlabScales / 4)];
      s[m] = C::NV ? (uint32_t)*(const uint16_t*)codes : (uint32_t)*codes;
    }
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int m = 0; m < TILES; ++m) {
        const v4i a = rows[m].fragment(j, s[m]);
#pragma unroll
        for (int q = 0; q < PARTS; ++q) acc[m] = mfma<C::F16>(a, v[q][j], acc[m]);
      }
  };
  for (int k0 = 0; k0 < K; k0 += kChunk) {
    const int n = min(kChunk, K - k0), first = k0 / kSlab, full = first + n / kSlab;
    const int s1 = first + wave;
    // slabs past the last are read again as the last and not used
    const int mine = s1 < full ? (full - s1 + 3) / 4 : 0, last = s1 + 4 * (mine - 1);
    if (mine) {
      fetch(s1);
      fetch_x(s1);
    }
    if (k0) __syncthreads();
    stage_scales<DEC, TILES>(sh, sc, K, k0, n, tid);
    __syncthreads();
    // One slab of weights ahead and four waves per SIMD: two slabs and three waves were slower (33 tokens,
    // 64 experts of 4096 x 2048 in NVFP4: 134 and 94 us for the two products, 126 and 89 us so).
    for (int i = 0; i < mine; ++i) {
      const int s = s1 + 4 * i, next = min(s + 4, last);
      multiply(s - first, next);
      fetch(next);
    }
    if (n % kSlab && wave == full % 4) {  // the rest: lanes past the end count as zero
      fetch_x(full);
      if (full * kSlab + 32 * g < K) {
        fetch(full);
      } else {
        // their scales are whatever LDS holds: zero them too, so that no NaN comes of it
#pragma unroll
        for (int m = 0; m < TILES; ++m) {
          rows[m].clear();
#pragma unroll
          for (int b = 0; b < C::kSlabScales / 4; ++b)
            sh.rows[16 * m + c][(full - first) * C::kSlabScales + g * (C::kSlabScales / 4) + b] = 0;
        }
      }
      multiply(full - first, full);
    }
  }
}

// Workgroup (x, slot): SiLU(gate) up of dims 32x .. 32x+31 for the tokens of the slot's expert.
template <bool NV, bool F16, bool ONE>
__global__ __launch_bounds__(kThreads, NV ? 4 : 3) void gate_up_kernel(MoeArgs p) {
  constexpr int TILES = 4;  // gate rows 0..15, 16..31, up rows 0..15, 16..31
  constexpr Dec DEC = NV ? Dec::kNvF16 : Dec::kMxBf16;
  constexpr Prep PREP = kPrep<NV, F16>;
  constexpr int PARTS = PREP == Prep::kParts ? 2 : 1;
  __shared__ union {
    struct {
      Scales<DEC, TILES> scales;
      Slab slab;
    };
    v4f acc[4][TILES][64];
  } sh;
  int4 slot;
  if (ONE) {
    // one token: slot y is its choice of rank y, found by each workgroup for itself while it would wait
    // for the router's last workgroup otherwise; the first workgroup of a slot keeps it for the next kernel
    const int lane = threadIdx.x & 63, y = blockIdx.y, last = blockIdx.x ? y : p.top_k - 1;
    int expert;
    float weight;
    auto choose_one = [&](auto each) {
      constexpr int R = decltype(each)::value;
      float x[R];
#pragma unroll
      for (int r = 0; r < R; ++r) x[r] = p.logits[min(lane * R + r, p.experts - 1)];
      for (int part = 1; part < p.router_parts; ++part)
#pragma unroll
        for (int r = 0; r < R; ++r) x[r] += p.logits[part * p.experts + min(lane * R + r, p.experts - 1)];
      top_k<R>(x, p.experts, last, p.keep, lane, expert, weight);
    };
    if (p.experts <= 64) choose_one(std::integral_constant<int, 1>{});
    else choose_one(std::integral_constant<int, BSG_MOE_MAX_EXPERTS / 64>{});
    slot = int4{__builtin_amdgcn_readlane(expert, y), y, 1, 0};
    if (blockIdx.x == 0 && (int)threadIdx.x == y) {
      p.slots[y] = slot;
      p.row_weight[y] = weight;
      p.row_of[y] = y;
      if (y == 0) *p.active = p.top_k;
      if (p.ids) p.ids[y] = expert;
      if (p.weights) p.weights[y] = weight;
    }
  } else {
    slot = p.slots[blockIdx.y];
    if ((int)blockIdx.y >= *p.active) return;
  }
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, c = lane & 15;
  const int e = __builtin_amdgcn_readfirstlane(slot.x), start = __builtin_amdgcn_readfirstlane(slot.y);
  const int count = __builtin_amdgcn_readfirstlane(slot.z);
  const int i0 = blockIdx.x * 32;
  const uint8_t *w[TILES], *sc[TILES];
#pragma unroll
  for (int m = 0; m < TILES; ++m) {
    const int64_t row = (int64_t)e * 2 * p.inter + (m < 2 ? 0 : p.inter) + i0 + (m & 1) * 16;
    w[m] = p.w13 + row * (NV ? p.hidden / 2 : p.hidden);
    sc[m] = p.s13 + row * (NV ? p.hidden / 16 : p.hidden / 32);
  }
  uint32_t column[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int col = 4 * i + (lane >> 4), t = ONE ? 0 : p.row_token[start + min(col, count - 1)];
    column[i] = col < count ? (uint32_t)t * p.hidden * 2 : kNoColumn;
  }
  v4f acc[TILES] = {};
  const uint32_t part = (uint32_t)p.tokens * p.hidden * 2;
  products<DEC, TILES, PARTS>(sh.scales, sh.slab, w, sc, p.hidden, tid, wave, p.xs, PARTS * part, column, part, acc);
  __syncthreads();  // the scales and the slabs are done with
#pragma unroll
  for (int m = 0; m < TILES; ++m) sh.acc[wave][m][lane] = acc[m];
  __syncthreads();
  const float alpha = p.alpha13 ? p.alpha13[e] : 1.0f;
  const int64_t rows = (int64_t)p.tokens * p.top_k;
  if (tid < 128) {
    const int m = tid >> 6, col = c, i = i0 + 16 * m + 4 * (lane >> 4);
    v4f gate = sh.acc[0][m][lane], up = sh.acc[0][m + 2][lane];
#pragma unroll
    for (int w = 1; w < 4; ++w) gate += sh.acc[w][m][lane], up += sh.acc[w][m + 2][lane];
    if (col >= count || i >= p.inter) return;
    // powers of two that the operands carry: decoded weights 2^-8, scaled rows of x 2^x_exp
    const int back = (NV ? 8 : 0) - (PREP == Prep::kScaled ? p.x_exp[ONE ? 0 : p.row_token[start + col]] : 0);
    uint16_t hi[4], lo[4];
#pragma unroll
    for (int r = 0; r < 4; ++r) {
      const float x = alpha * __builtin_amdgcn_ldexpf(gate[r], back), u = alpha * __builtin_amdgcn_ldexpf(up[r], back);
      const float v = x / (1.0f + __builtin_amdgcn_exp2f(-x * kLog2e)) * u;
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
template <bool NV, bool F16>
__global__ __launch_bounds__(kThreads, 3) void down_kernel(MoeArgs p) {
  constexpr int TILES = 4;
  constexpr Dec DEC = NV ? Dec::kNvBf16 : Dec::kMxBf16;
  __shared__ union {
    struct {
      Scales<DEC, TILES> scales;
      Slab slab;
    };
    v4f acc[4][TILES][64];
  } sh;
  __shared__ int last;
  const int active = *p.active;
  const int4 slot = p.slots[blockIdx.y];
  if ((int)blockIdx.y >= active) return;
  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63, c = lane & 15;
  const int e = __builtin_amdgcn_readfirstlane(slot.x), start = __builtin_amdgcn_readfirstlane(slot.y);
  const int count = __builtin_amdgcn_readfirstlane(slot.z);
  const int d0 = blockIdx.x * 64;
  const uint8_t *w[TILES], *sc[TILES];
#pragma unroll
  for (int m = 0; m < TILES; ++m) {
    const int64_t row = (int64_t)e * p.hidden + min(d0 + 16 * m, p.hidden - 16);  // (tiles past the end repeat the last)
    w[m] = p.w2 + row * (NV ? p.inter / 2 : p.inter);
    sc[m] = p.s2 + row * (NV ? p.inter / 16 : p.inter / 32);
  }
  uint32_t column[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const int col = 4 * i + (lane >> 4);
    column[i] = col < count ? (uint32_t)(start + col) * p.inter * 2 : kNoColumn;
  }
  v4f acc[TILES] = {};
  const uint32_t part = (uint32_t)(p.tokens * p.top_k) * p.inter * 2;
  products<DEC, TILES, 2>(sh.scales, sh.slab, w, sc, p.inter, tid, wave, p.h, 2 * part, column, part, acc);
  __syncthreads();  // the scales and the slabs are done with
#pragma unroll
  for (int m = 0; m < TILES; ++m) sh.acc[wave][m][lane] = acc[m];
  __syncthreads();
  const float alpha = p.alpha2 ? p.alpha2[e] : 1.0f;
  const __amdgpu_buffer_rsrc_t ybuf = handoff_buffer(p.y, (uint32_t)(p.tokens * p.top_k) * (uint32_t)p.hidden * 4u);
  {
    const int m = wave, col = c, d = d0 + 16 * m + 4 * (lane >> 4);
    v4f y = sh.acc[0][m][lane];
#pragma unroll
    for (int w = 1; w < 4; ++w) y += sh.acc[w][m][lane];
    if (col < count && d < p.hidden)
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

template <bool NV, bool F16>
hipError_t launch(const MoeArgs& a, hipStream_t stream) {
  MoeArgs args = a;
  void* argv[] = {&args};
  const unsigned tiles = (a.experts + 15) / 16 * ((a.tokens + 15) / 16);
  // Parts of 1024 k where there are few tiles: a compute unit reads a tile's 256 KB (hidden 4096) in 3.5 us (1 token, 64
  // experts: 7.1 us whole, 4.5 in 4 parts; 33 tokens: 16.8 and 14.4).  Many tiles fill more compute units, and
  // their parts would all pass through the one that chooses.
  const int parts = (a.hidden + 1023) / 1024;
  args.router_parts = tiles > 32 ? 1 : parts < kRouterParts ? parts : kRouterParts;
  hipError_t e = hipLaunchKernel((const void*)&router_kernel<NV, F16>, dim3(tiles * args.router_parts + a.tokens),
                                 dim3(kRouterThreads), argv, 0, stream);
  if (e != hipSuccess) return e;
  // at most one slot per choice, and one per expert and kSlotRows choices
  const int choices = a.tokens * a.top_k, bound = a.experts + choices / kSlotRows;
  const unsigned slots = choices < bound ? choices : bound;
  const void* gate_up = a.tokens == 1 ? (const void*)&gate_up_kernel<NV, F16, true> : (const void*)&gate_up_kernel<NV, F16, false>;
  e = hipLaunchKernel(gate_up, dim3((a.inter + 31) / 32, slots), dim3(kThreads), argv, 0, stream);
  if (e != hipSuccess) return e;
  return hipLaunchKernel((const void*)&down_kernel<NV, F16>, dim3((a.hidden + 63) / 64, slots), dim3(kThreads), argv, 0, stream);
}

}  // namespace

hipError_t moe_launch(const MoeArgs& a, int format, int dtype, hipStream_t stream) {
  if (format) return dtype ? launch<true, true>(a, stream) : launch<true, false>(a, stream);
  return dtype ? launch<false, true>(a, stream) : launch<false, false>(a, stream);
}

size_t moe_workspace(const bsg_moe_problem& p, uint8_t* base, MoeArgs* a, size_t* counters_at, size_t* counters_bytes) {
  const size_t T = (size_t)p.max_tokens, rows = T * p.top_k;
  size_t at = 0;
  auto take = [&](size_t bytes) {
    const size_t here = at;
    at += (bytes + 255) & ~(size_t)255;
    return base ? base + here : nullptr;
  };
  a->logits = (float*)take(kRouterParts * T * p.experts * 4);
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
