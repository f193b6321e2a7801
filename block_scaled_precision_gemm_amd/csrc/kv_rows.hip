// Attention over the paged NVFP4 cache for many query rows per key/value head: prompt chunks.
//
// A workgroup holds R = 32 WAVES query rows (new tokens x the heads that share a key/value head) of one
// sequence and walks the positions that they see in tiles of 64.  Each tile is decoded once by the
// workgroup, from packed codes in registers to fp16 fragments in LDS (two buffers, one barrier per tile).
// Fragments are stored in the order in which the lanes of a product read them, so every LDS access is 1 KB
// in a row:
// * keys: 16 positions x 32 dims per fragment, S^T = K Q^T;
// * values: 16 dims x 32 positions, O^T += V^T P^T, with P^T straight from S^T's registers.
// The lane layouts and the decoding are those of the few-row kernel (kv_attend.hip).  Each wave keeps 32
// rows, so a fragment read from LDS feeds two products.
//
// Bound: per tile and wave 64 products (about 1040 cycles of the SIMD's matrix unit) and 230 vector
// operations (about 1150 cycles).  A SIMD holds two waves, and they only overlap if one multiplies while
// the other does its softmax: half of the waves go through a tile in the other order (run, below), products
// have priority, and fragments are read six ahead.  2 x 2048 tokens against 8192 and 3351 positions, 32
// heads on 8 of 128: 361 us with all waves in step, 338 us half a tile apart, 306 us with priority, 270 to 278 us
// with fragments six ahead and fewer rescalings (kSlack; 1150 to 1180 TFLOP/s); the products alone, without decoding, loads and softmax, 203 us.
//
// Workgroups that share a sequence and head run on one XCD where that can be arranged, and share its L2
// (the same case: 618 us with sequences in turn, 458 us so).  Where the rows alone give too few workgroups,
// positions are split and a second kernel joins the parts.
#include <type_traits>

#include "kv_attend.h"

namespace bsg {
namespace {

// P is held as 2^kPBias P, relative to a row's reference m: a maximum of its products, which is only replaced (and the
// row's sums rescaled) once some product lies more than kSlack above it.  P then stays below 2^15, and weights down to
// 2^-34 of the largest are kept (fp16 steps are 2^-24).  This costs accuracy: rounding P to fp16 costs every weight up to
// 2^-11 of itself, and a stale reference adds the largest one, which would be exact as a power of two.  Beside a reference
// that is always the maximum (and 2^14, kept down to 2^-38): 2 x 2048 tokens 296 us, heads of 64 229 us, against 278 and 203;
// root mean square error of fp16 outputs of order 0.1 3.34e-5 against 3.40e-5, and 2.83e-5 with weights in fp32, most of
// it the output's own rounding; of bf16 ones the same.
constexpr float kPBias = 10.0f, kSlack = 5.0f;

// Where the results of row block rb of a sequence and head go.
template <Out O, int D, int R>
struct Results {
  const KvArgs& p;
  int first_token, h, rb;
  __device__ void store_lse(int row, float top, float sum) const {
    const int i = (rb * R + row) / p.group, hq = rb * R + row - i * p.group;
    p.lse[(int64_t)(first_token + i) * p.q_heads + h * p.group + hq] =
        sum == 0.0f ? kNegInf : (top - kPBias + __builtin_amdgcn_logf(sum)) * kLn2;
  }
  __device__ uint16_t* out_at(int row, int d) const {
    const int i = (rb * R + row) / p.group, hq = rb * R + row - i * p.group;
    return (uint16_t*)p.out.ptr + (int64_t)(first_token + i) * p.out.token_stride + (int64_t)(h * p.group + hq) * p.out.head_stride + d;
  }
  // Four outputs from sums of weighted values, 256 over the weights' sum, and whether that is zero.
  __device__ uint2 pack4(v4f y, float f, bool none) const {
    uint32_t bits[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) bits[i] = out_bits<O>(none ? 0.0f : y[i] * f * p.v_scale);  // (v_scale may be near fp32's ends)
    return make_uint2(bits[0] | bits[1] << 16, bits[2] | bits[3] << 16);
  }
};

// Row block `at` of a group: its sequence, head, and which of the sequence's blocks of R rows, the last one first.
struct RowBlock {
  int b, h, first_token, q_len;
  int rb;  // < 0: none
};

template <int R>
__device__ __forceinline__ RowBlock row_block(const KvArgs& p, int group, int at, int lane) {
  RowBlock s;
  if (p.row_listed) {
    int lo = 0;
    for (int n = p.num_seqs; n > 1;) {  // the last sequence that starts at or before the slot: 64 pivots a step
      const int step = (n + 63) / 64, i = lane * step;
      const bool le = i < n && row_slot(seq_start(p, lo + i), lo + i, p.group, R) <= at;
      const int parts = max(__popcll(__ballot(le)), 1) - 1;
      lo += parts * step;
      n = min(step, n - parts * step);
    }
    s.b = __builtin_amdgcn_readfirstlane(lo);
    s.h = group;
    at -= row_slot(seq_start(p, s.b), s.b, p.group, R);
  } else {
    s.b = group / p.kv_heads;
    s.h = group - s.b * p.kv_heads;
  }
  s.first_token = p.one_each ? s.b : seq_start(p, s.b);
  s.q_len = p.one_each ? 1 : min(max(seq_start(p, s.b + 1) - s.first_token, 0), p.max_q);
  const int blocks = (s.q_len * p.group + R - 1) / R;
  const bool other = p.mixed && s.q_len * p.group <= kFewRows;  // the few-row kernel's
  s.rb = other || at < 0 ? -1 : blocks - 1 - at;
  return s;
}

template <Out O, int D, int WAVES>
__global__ __launch_bounds__(64 * WAVES, 2) void rows_kernel(KvArgs p) {
  constexpr int RT = 2, R = 32 * WAVES;
  constexpr int NJ = D / 32, E = D / 16;
  constexpr int SLOT = R * (D + 2);  // a part: its rows' outputs, then their maxima and sums
  using L = PageLayout<D>;
  struct Buffer {
    v4i k[4][NJ][64];  // [16 positions][32 dims][lane]
    v4i v[2][E][64];   // [32 positions][dims E m + e][lane]
  };
  __shared__ Buffer sh[2];
  __shared__ int sh_nan[4];  // tile n's first position at n % 4, if it has such a NaN block (below)

  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int c = lane & 15, g = lane >> 4;
  const int H = p.kv_heads, G = p.group, P = 1 << p.page_shift;
  const bool causal = !(p.flags & BSG_KV_NONCAUSAL);

  // ---- block and split.  Groups (kv_split.h) are a multiple of 8: workgroup x is on XCD x % 8 and so is all of a
  // group, whose blocks follow each other there, each sequence's from the last (the longest) to the first.
  // Otherwise groups alternate.
  const int per_group = p.row_width * p.splits;
  int group, rest;
  if (p.row_groups % 8 == 0) {
    const int at = blockIdx.x >> 3;
    group = at / per_group * 8 + (blockIdx.x & 7);
    rest = at % per_group;
  } else {
    group = blockIdx.x % p.row_groups;
    rest = blockIdx.x / p.row_groups;
  }
  const int split = rest % p.splits;
  const RowBlock block = row_block<R>(p, group, rest / p.splits, lane);
  if (block.rb < 0) return;
  const int b = block.b, h = block.h, rb = block.rb, first_token = block.first_token, q_len = block.q_len;
  const int len = seq_len(p, b);
  const int rows = min(R, q_len * G - rb * R), pos0 = len - q_len;
  const int i_first = rb * R / G, i_last = (rb * R + rows - 1) / G;
  const int lo = p.window > 0 ? max(0, pos0 + i_first - p.window + 1) : 0;
  const int hi = causal ? max(0, pos0 + i_last + 1) : len;
  const int base = lo & ~15, all = hi > base ? (hi - base + kTile - 1) / kTile : 0;
  const int per = (all + p.splits - 1) / p.splits;
  const int t_begin = base + split * per * kTile, t_end = min(hi, t_begin + per * kTile);

  // ---- queries
  const int w_row = 32 * wave;  // the wave's first row
  v8h q[RT][NJ];
  float mul[RT];
  int pos[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int r = w_row + 16 * t + c, row = rb * R + (r < rows ? r : 0);
    v4i raw[NJ];
    load_query<D>(p, first_token, h, row, g, raw);
    convert_query<O, D>(p, raw, q[t], mul[t]);
    pos[t] = causal ? pos0 + row / G : len - 1;
  }
  // positions that all, and any, of the wave's rows see up to
  const int w_first = causal ? pos0 + (rb * R + min(w_row, rows - 1)) / G : len - 1;
  const int w_last = causal ? pos0 + (rb * R + min(w_row + 31, rows - 1)) / G : len - 1;
  v4f o[RT][E];
  float m[RT], l[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    m[t] = kNegInf;
    l[t] = 0.0f;
#pragma unroll
    for (int e = 0; e < E; ++e) o[t][e] = v4f{0, 0, 0, 0};
  }

  if (t_begin < t_end) {
    const int* table = p.pages + (int64_t)b * p.pages_stride;
    const int last_pos = hi - 1, chunk = L::chunk(P);
    // Decoding a tile is cut in tasks for four waves: the values of positions 32 (task / 2) .. + 31 for even
    // or odd dims, and the keys of 16 positions.  Of eight waves the first four decode values, the others keys.
    const int task = wave & 3;
    uint32_t kq[NJ], ks = 0, vq[2][4], vs[2];
    // Page numbers of 64 pages from page_base on, one per lane
    int page_base = t_begin >> p.page_shift;
    int page_ids = clamp_page(p, table[min(page_base + lane, last_pos >> p.page_shift)]);
    auto keep_pages = [&](int t0) {  // those of two tiles from t0 on (at most 9) are among them
      const int first = min(t0, last_pos) >> p.page_shift;
      if (first - page_base >= 48) {
        page_base = first;
        page_ids = clamp_page(p, table[min(page_base + lane, last_pos >> p.page_shift)]);
      }
    };
    const uint8_t* head = p.cache + (int64_t)h * chunk;
    auto group_at = [&](int t, int& slot) -> const uint8_t* {  // (clamped into the context)
      t = min(t, last_pos & ~15);
      slot = t & (P - 1);
      return head + (int64_t)__builtin_amdgcn_readlane(page_ids, (t >> p.page_shift) - page_base) * p.page_stride;
    };
    // a lane's offsets from a group's codes and scales
    const uint32_t v_lane = 4 * g * L::kRow + c * (E / 2), vs_lane = (c * E / 16) * P + 4 * g;
    const uint32_t k_lane = c * L::kRow + g * (4 * NJ), ks_lane = c * L::kBlocks + g * (D / 64);
    auto load_v = [&](int t0) __attribute__((always_inline)) {
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        int slot;
        const uint8_t* at = group_at(t0 + 32 * (task >> 1) + 16 * u, slot);
        const uint8_t *codes = at + L::v_codes(P) + slot * L::kRow, *scales = at + L::v_scales(P) + slot;
#pragma unroll
        for (int j = 0; j < 4; ++j)
          vq[u][j] = E == 8 ? *(const uint32_t*)(codes + v_lane + j * L::kRow) : *(const uint16_t*)(codes + v_lane + j * L::kRow);
        vs[u] = *(const uint32_t*)(scales + vs_lane);
      }
    };
    auto load_k = [&](int t0) __attribute__((always_inline)) {
      int slot;
      const uint8_t* at = group_at(t0 + 16 * task, slot);
      const uint8_t *codes = at + slot * L::kRow, *scales = at + L::k_scales(P) + slot * L::kBlocks;
      if constexpr (D == 128) {
        const v4i w = *(const v4i*)(codes + k_lane);
#pragma unroll
        for (int j = 0; j < NJ; ++j) kq[j] = (uint32_t)w[j];
        ks = *(const uint16_t*)(scales + ks_lane);
      } else {
        const uint2 w = *(const uint2*)(codes + k_lane);
        kq[0] = w.x;
        kq[1] = w.y;
        ks = scales[ks_lane];
      }
    };
    // some row of the workgroup does not see all of the tile at t0
    const int all_first = causal ? pos0 + i_first : len - 1, any_last = causal ? pos0 + i_last : len - 1;
    auto partly_hidden = [&](int t0) {
      return t0 + kTile - 1 > min(all_first, t_end - 1) || (p.window > 0 && t0 <= any_last - p.window);
    };
    // Of a tile that is partly hidden, positions outside the workgroup's count as zero, whatever their slots hold,
    // and NaN blocks that only some rows see are taken out and given to those rows by the waves (take_nans).
    auto mask_v = [&](int t0) __attribute__((always_inline)) {
      if (!partly_hidden(t0)) return;
      const int g4 = 4 * rare(g);
      uint32_t bad = 0;
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t keep = 0;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const int at = t0 + 32 * (task >> 1) + 16 * u + g4 + i;
          if (at >= lo && at < t_end) keep |= 0xFFu << (8 * i);
        }
        vs[u] &= keep;
        const uint32_t hit = ((vs[u] + 0x01010101u) & 0x80808080u) >> 7;
        bad |= hit;
        vs[u] &= ~(hit * 0x7Fu);
      }
      if (__any(bad) && lane == 0) sh_nan[(t0 - t_begin) / kTile & 3] = t0;
    };
    // Fragment e of the wave's decoded values (positions pairs[2u], pairs[2u + 1]: u = 0, 1), and j of its keys
    uint32_t pairs[4];
    v2h v_s[4];
    const int odd = task & 1, down = 4 * odd;
    auto decode_v = [&](int e, int buf) __attribute__((always_inline)) {
      if (e == 0) {
#pragma unroll
        for (int jj = 0; jj < 4; ++jj) {
          const int u = jj / 2, j = (jj & 1) * 2;
          v_s[jj] = __builtin_bit_cast(v2h, (jj & 1) ? scale_pair<kHigh>(vs[u]) : scale_pair<kLow>(vs[u]));
          const uint32_t mask = 0x0F0F0F0Fu;
          pairs[jj] = ((vq[u][j] >> down) & mask) | ((vq[u][j + 1] << (4 - down)) & ~mask);
        }
      }
      v4i frag;
#pragma unroll
      for (int jj = 0; jj < 4; ++jj) frag[jj] = __builtin_bit_cast(int, fp4_pair(pairs[jj], e) * v_s[jj]);
      sh[buf].v[task >> 1][2 * e + odd][lane] = frag;
    };
    auto decode_k = [&](int j, int buf) __attribute__((always_inline)) {
      const uint32_t sp = scale_pair<kLow>(ks);
      sh[buf].k[task][j][lane] = e2m1x8_scaled_f16x8(kq[j], j < 2 ? f16x2_splat_lo(sp) : f16x2_splat_hi(sp));
    };
    v4f sc[RT][4];
    v8h pt[RT][2];
    if (tid < 4) sh_nan[tid] = -1;
    // before the first tile there are no weights and values: zeros
#pragma unroll
    for (int t = 0; t < RT; ++t) pt[t][0] = pt[t][1] = v8h{};
    for (int i = tid; i < 2 * E * 64; i += 64 * WAVES) (&sh[1].v[0][0][0])[i] = v4i{0, 0, 0, 0};
    __syncthreads();
    // A tile's products: the last tile's outputs, then this tile's scores, each fragment read from LDS
    // kFly fragments before its two products.  Between them the wave decodes its part of this tile's values into
    // buffer buf and of the next tile's keys into the other, and loads the following ones: its vector operations
    // run beside its products.
    auto products = [&](auto scores, auto do_v, auto do_k, int t0, int buf) __attribute__((always_inline)) {
      constexpr int NO = 2 * E, N = NO + (scores.value ? 4 * NJ : 0);
      constexpr int NV = do_v.value ? E / 2 : 0, NU = NV + (do_k.value ? NJ : 0);
      constexpr int kFly = 6;
      v8h frag[kFly];
      auto read = [&](int i) {
        return __builtin_bit_cast(v8h, i < NO ? sh[buf ^ 1].v[i / E][i % E][lane] : sh[buf].k[(i - NO) % 4][(i - NO) / 4][lane]);
      };
#pragma unroll
      for (int i = 0; i < kFly; ++i) frag[i] = read(i);
      __builtin_amdgcn_sched_group_barrier(0x100, kFly, 0);
#pragma unroll
      for (int i = 0; i < N; ++i) {
        const v8h a = frag[i % kFly];
        if (i + kFly < N) frag[i % kFly] = read(i + kFly);
        if (i < NO) {
#pragma unroll
          for (int t = 0; t < RT; ++t) o[t][i % E] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, pt[t][i / E], o[t][i % E], 0, 0, 0);
        } else {
          const int j = (i - NO) / 4, gr = (i - NO) % 4;
#pragma unroll
          for (int t = 0; t < RT; ++t)
            sc[t][gr] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, q[t][j], j ? sc[t][gr] : v4f{0, 0, 0, 0}, 0, 0, 0);
        }
#pragma unroll
        for (int u = 0; u < NU; ++u)
          if (i == (u + 1) * N / (NU + 2)) {
            if (u < NV) decode_v(u, buf);
            else decode_k(u - NV, buf ^ 1);
          }
        if (NU && i == (NU + 1) * N / (NU + 2)) {
          if (do_v.value) load_v(t0 + kTile);
          if (do_k.value) load_k(t0 + 2 * kTile);
        }
        __builtin_amdgcn_sched_group_barrier(0x008, RT, 0);
        if (i + kFly < N) __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      }
    };
    auto softmax = [&](int t0) __attribute__((always_inline)) {
      const bool edge = t0 + kTile - 1 > min(w_first, t_end - 1) || (p.window > 0 && t0 <= w_last - p.window);
#pragma unroll
      for (int t = 0; t < RT; ++t) {
        const float scale = mul[t];
        if (p.cap > 0.0f) soft_cap<4>(p, scale, sc[t]);
        if (edge) {
          const int first = t0 + 4 * rare(g), top = min(pos[t], t_end - 1), bottom = p.window > 0 ? pos[t] - p.window : -1;
#pragma unroll
          for (int gr = 0; gr < 4; ++gr)
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int at = first + 16 * gr + i;
              sc[t][gr][i] = at <= top && at > bottom ? sc[t][gr][i] : kNegInf;
            }
        }
        float top = sc[t][0][0];
#pragma unroll
        for (int gr = 0; gr < 4; ++gr)
#pragma unroll
          for (int i = 0; i < 4; ++i) top = __builtin_fmaxf(top, sc[t][gr][i]);
        if (__any((top - m[t]) * scale > kSlack)) {
          const float grown = __builtin_fmaxf(m[t], max_over_g(top));
          const float f = grown == kNegInf ? 1.0f : __builtin_amdgcn_exp2f((m[t] - grown) * scale);
          m[t] = grown;
          l[t] *= f;
#pragma unroll
          for (int e = 0; e < E; ++e) o[t][e] *= f;
        }
        const float off = m[t] == kNegInf ? 0.0f : kPBias - m[t] * scale;
#pragma unroll
        for (int k = 0; k < 2; ++k)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            float e4[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              e4[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[t][2 * k + half][i], scale, off));
              l[t] += e4[i];
            }
            const v2h x = __builtin_convertvector((v2f{e4[0], e4[1]}), v2h), y = __builtin_convertvector((v2f{e4[2], e4[3]}), v2h);
            pt[t][k][4 * half] = x[0];
            pt[t][k][4 * half + 1] = x[1];
            pt[t][k][4 * half + 2] = y[0];
            pt[t][k][4 * half + 3] = y[1];
          }
      }
    };
    auto take_nans = [&](int t0) __attribute__((always_inline)) {
      if (partly_hidden(t0) && __builtin_amdgcn_readfirstlane(sh_nan[(t0 - t_begin) / kTile & 3]) == t0) {
        // rare: a NaN block among positions that not every row sees.  Output element i of tile e is
        // dim E (4g + i) + e, so element i lies in block E (4g + i) / 16.
        for (int at = max(t0, lo); at < min(t0 + kTile, t_end); ++at) {
          const int page = clamp_page(p, table[at >> p.page_shift]), sl = at & (P - 1);
          const uint8_t* codes = p.cache + (int64_t)page * p.page_stride + (int64_t)h * chunk + L::v_scales(P) + sl;
          const int g4 = 4 * rare(g);
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const bool bad = codes[E * (g4 + i) / 16 * P] == 0x7F;
#pragma unroll
            for (int t = 0; t < RT; ++t)
              if (bad && at <= pos[t] && (p.window <= 0 || at > pos[t] - p.window))
#pragma unroll
                for (int e = 0; e < E; ++e) o[t][e][i] = __builtin_nanf("");
          }
        }
      }
    };
    // One barrier per tile.  Between two of them the first waves do tile t's products (and the outputs of tile
    // t - 1) and then its softmax; of eight waves the last four do the softmax of tile t - 1 first, so that
    // each SIMD has one wave in matrix products and one in vector operations.  Values of tile t and keys of
    // tile t + 1 are decoded meanwhile, into the buffers that were read before the last barrier.
    auto tile_end = [] {
      __builtin_amdgcn_sched_barrier(0);
      __syncthreads();
      __builtin_amdgcn_sched_barrier(0);
    };
    auto run = [&](auto do_v, auto do_k) __attribute__((always_inline)) {
      constexpr bool late = !do_v.value;
      if (do_v.value) {
        load_v(t_begin);
        mask_v(t_begin);
      }
      if (do_k.value) {
        load_k(t_begin);
#pragma unroll
        for (int j = 0; j < NJ; ++j) decode_k(j, 0);
        load_k(t_begin + kTile);
      }
      tile_end();
      int buf = 0;
      for (int t0 = t_begin; t0 < t_end; t0 += kTile, buf ^= 1) {
        if (late && t0 > t_begin) softmax(t0 - kTile);
        __builtin_amdgcn_s_setprio(1);  // products first: the other wave's operations fit between them
        products(std::true_type{}, do_v, do_k, t0, buf);
        __builtin_amdgcn_s_setprio(0);
        if (t0 > t_begin) take_nans(t0 - kTile);
        if (!late) softmax(t0);
        keep_pages(t0 + 2 * kTile);
        if (do_v.value) mask_v(t0 + kTile);
        tile_end();
      }
      const int t_last = t_begin + (t_end - 1 - t_begin) / kTile * kTile;
      if (late) softmax(t_last);
      products(std::false_type{}, std::false_type{}, std::false_type{}, t_end, buf);
      take_nans(t_last);
    };
    if constexpr (WAVES == 4) run(std::true_type{}, std::true_type{});
    else if (wave < 4) run(std::true_type{}, std::false_type{});
    else run(std::false_type{}, std::true_type{});
  }

  // ---- results
  const Results<O, D, R> results{p, first_token, h, rb};
  float* part = p.part + (int64_t)(group * per_group + rest) * SLOT;
#pragma unroll
  for (int t = 0; t < RT; ++t) {
    const int r = w_row + 16 * t + c;
    const float sum = sum_over_g(l[t]), top = m[t] == kNegInf ? kNegInf : m[t] * mul[t];
    if (r >= rows) continue;
    if (p.splits == 1) {
      const float f = 256.0f / sum;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint16_t* dst = results.out_at(r, E * (4 * g + i));
#pragma unroll
        for (int e = 0; e < E; e += 4)
          *(uint2*)(dst + e) = results.pack4(v4f{o[t][e][i], o[t][e + 1][i], o[t][e + 2][i], o[t][e + 3][i]}, f, sum == 0.0f);
      }
      if (p.lse && g == 0) results.store_lse(r, top, sum);
    } else {
#pragma unroll
      for (int i = 0; i < 4; ++i)
#pragma unroll
        for (int e = 0; e < E; e += 4)
          *(v4f*)(part + r * D + E * (4 * g + i) + e) = v4f{o[t][e][i], o[t][e + 1][i], o[t][e + 2][i], o[t][e + 3][i]};
      if (g == 0) *(v2f*)(part + R * D + 2 * r) = v2f{top, sum};
    }
  }
}

// Joins the parts of split row blocks, with one thread for four dims of a row.  A kernel of its own, so that
// the whole chip reads the parts: joined by the last workgroup of each block, 2 x 482 tokens, 8 heads on
// 4 of 128 dims and a window of 781 took 67 us against 34.
template <Out O, int D, int R>
__global__ __launch_bounds__(256) void join_kernel(KvArgs p) {
  constexpr int ROWS = 256 / (D / 4), SLOT = R * (D + 2), AT_ONCE = 8;
  const int unit = blockIdx.x / (R / ROWS), group = unit / p.row_width;
  const RowBlock block = row_block<R>(p, group, unit - group * p.row_width, threadIdx.x & 63);
  if (block.rb < 0) return;
  const int h = block.h, rb = block.rb, first_token = block.first_token, q_len = block.q_len;
  const int r = blockIdx.x % (R / ROWS) * ROWS + threadIdx.x / (D / 4), d = threadIdx.x % (D / 4) * 4;
  if (r >= min(R, q_len * p.group - rb * R)) return;
  const float* part = p.part + (int64_t)unit * p.splits * SLOT;
  const int last = p.splits - 1;
  float top = kNegInf, sum = 0.0f;
  v4f y = {0, 0, 0, 0};
  for (int s0 = 0; s0 <= last; s0 += AT_ONCE) {
    v2f ms[AT_ONCE];
    v4f ys[AT_ONCE];
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {  // all in flight; parts past the last repeat it and count nothing
      const float* at = part + (int64_t)min(s0 + i, last) * SLOT;
      ms[i] = *(const v2f*)(at + R * D + 2 * r);
      ys[i] = *(const v4f*)(at + r * D + d);
    }
    float grown = top;
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) grown = __builtin_fmaxf(grown, ms[i][0]);
    const float f0 = top == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(top - grown);
    sum *= f0;
    y *= f0;
    top = grown;
#pragma unroll
    for (int i = 0; i < AT_ONCE; ++i) {
      if (s0 + i > last) continue;
      const float f = ms[i][0] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(ms[i][0] - top);
      sum += f * ms[i][1];
      y += f * ys[i];
    }
  }
  const Results<O, D, R> results{p, first_token, h, rb};
  *(uint2*)results.out_at(r, d) = results.pack4(y, 256.0f / sum, sum == 0.0f);
  if (p.lse && d == 0) results.store_lse(r, top, sum);
}

template <Out O, int D, int WAVES>
hipError_t launch(const KvArgs& a, int cus, hipStream_t stream) {
  constexpr int R = 32 * WAVES;
  KvArgs args = a;
  const RowsGrid grid = rows_grid(R, a.num_tokens, a.num_seqs, a.max_q, a.group, a.kv_heads);
  const int64_t places = grid.groups * grid.width;
  args.row_groups = (int)grid.groups;
  args.row_width = (int)grid.width;
  args.row_listed = grid.listed;
  // units that exist, at most: ragged sequences leave some of the places without rows
  const int64_t rows = (int64_t)a.num_tokens * a.group, most = a.mixed ? rows / kFewRows : a.num_seqs;
  int64_t units = (rows / R + (most < a.num_seqs ? most : a.num_seqs)) * a.kv_heads;
  if (units > places) units = places;
  const int64_t fill = (int64_t)cus * (8 / WAVES);  // workgroups that run at once
  const int64_t seen = a.window > 0 ? (int64_t)a.window + a.max_q : a.max_kv;
  const int64_t tiles = ((seen < a.max_kv ? seen : a.max_kv) + kTile - 1) / kTile;
  // The number of parts that takes the fewest tiles' time.  A workgroup's beginning and end cost about three
  // tiles, the join two and one more for 8 parts.  At least two tiles per part; the workspace holds twice
  // the workgroups that run at once.  (2 x 134 tokens, 8 heads on 4 of 128 dims, 2133 positions: one part
  // 86 us, so 26 us; one sequence of 1575 tokens, 4 heads on 1, 3756 positions: 141 and 40 us.)
  int64_t splits = 1, best = 0;
  for (int64_t s = 1; s == 1 || (s <= tiles / 2 && places * s <= 2 * fill); ++s) {
    const int64_t cost = (units * s + fill - 1) / fill * ((tiles + s - 1) / s + 3) + (s > 1 ? 2 + s / 8 : 0);
    if (s == 1 || cost < best) {
      best = cost;
      splits = s;
    }
  }
  args.splits = (int)splits;
  void* argv[] = {&args};
  hipError_t err = hipLaunchKernel((const void*)&rows_kernel<O, D, WAVES>, dim3((unsigned)(places * splits)),
                                   dim3(64 * WAVES), argv, 0, stream);
  if (err != hipSuccess || splits == 1) return err;
  return hipLaunchKernel((const void*)&join_kernel<O, D, R>, dim3((unsigned)(places * (R * (D / 4) / 256))), dim3(256),
                         argv, 0, stream);
}

template <Out O, int D>
hipError_t launch(const KvArgs& a, int cus, hipStream_t stream) {
  return rows_waves(a.max_q, a.group) == 8 ? launch<O, D, 8>(a, cus, stream) : launch<O, D, 4>(a, cus, stream);
}

}  // namespace

hipError_t kv_attend_rows_launch(const KvArgs& a, int dtype, int head_dim, int cus, hipStream_t stream) {
  if (head_dim == 64) return dtype ? launch<Out::F16, 64>(a, cus, stream) : launch<Out::BF16, 64>(a, cus, stream);
  return dtype ? launch<Out::F16, 128>(a, cus, stream) : launch<Out::BF16, 128>(a, cus, stream);
}

size_t kv_rows_part_floats(const bsg_kv_problem& p, int cus) {
  if (p.max_tokens * (p.q_heads / p.kv_heads) <= kFewRows) return 0;
  return (size_t)2 * cus * 256 * (p.head_dim + 2);  // 2 x 8 waves per CU, 32 rows each
}

}  // namespace bsg
