// Attention over the paged NVFP4 cache for few query rows per key/value head.
//
// A unit of work is a block of R = 16 RT query rows (new tokens x the query heads that share a
// key/value head) of one sequence and key/value head, over that sequence's positions, which are cut into
// tiles of 64.  Where there are few units each is cut into pieces, one per workgroup, all about as long;
// where there are many, the tiles of all units, and a fixed cost for each unit, form one line, and each
// workgroup takes an equal run of it.  Either way one launch balances any mixture of lengths.  A unit
// that lies in several workgroups is joined by the last of them to finish, in the workgroups' order, from
// the parts (output, maximum, sum) that the others left in the plan's workspace, so the order of every
// sum is fixed.
//
// Inside a workgroup the four waves take consecutive quarters of a run and are joined through LDS.  A
// wave handles 32 positions at a time, everything in registers, while the next two steps' codes arrive:
// * S^T = K Q^T on v_mfma_f32_16x16x32_f16: a lane loads D/4 consecutive dims of one position (16
//   bytes for D = 128) -- the k order of the product is free, so those are its k values.  K is decoded
//   exactly (codec.h); Q is exact in fp16 once each row is scaled by a power of two (bf16 rows).
// * The result has position 4g + i (g = lane / 16) of each 16 in element i and the row in lane % 16,
//   which is the layout in which P^T enters O^T += V^T P^T as the second operand: softmax needs no
//   data movement but the maximum over g.
// * For that product a lane needs 8 positions of one dim.  It loads 4 bytes (D = 128: 8 dims) of each
//   of 8 positions, interleaves the nibbles of two positions (4 operations for 16 values), and decodes
//   each byte to the pair (position j, position j + 1), which one packed multiply scales by the pair of
//   scales, stored with the position fastest for this purpose.
// Softmax: maximum m and sum l per row, in fp32 and base 2.  P is rounded to fp16 for its product, 2^-11 of itself at most (a
// second product for what is left would double the work beside the loads); l sums the unrounded values.
//
// Bound: bytes of the cache (D 9/8 bytes per position and head) where contexts are long; for short ones the
// chain of dependent trips to memory (lengths, page numbers, codes, the join), about 10 us.  Measured, heads
// of 128: 64 tokens over up to 16384 positions, 64 heads on 8: 80 us (4.3 TB/s); one token over 131072
// positions, 32 heads on 4: 28 us (2.7 TB/s); one over 1001 positions, 32 heads on 8: 10 us.
#include "handoff.h"
#include "kv_attend.h"

namespace bsg {
namespace {

constexpr int kThreads = 256;
constexpr int kMinTiles = 2;    // a piece is at least a step of each wave
constexpr int kWgPerCu = 2;
// P is held as 2^kPBias P, relative to the row's maximum in the wave's run so far: at most 2^14, and weights down to 2^-38 of
// the largest are kept (fp16 steps are 2^-24).
constexpr float kPBias = 14.0f;

template <int CTRL, int ROWS>
__device__ __forceinline__ int dpp_add(int x) {
  return x + __builtin_amdgcn_update_dpp(0, x, CTRL, ROWS, 0xF, false);
}
// Inclusive sums over the wave's lanes.
__device__ __forceinline__ int wave_scan(int x) {
  x = dpp_add<0x111, 0xF>(x);  // shift right within rows of 16 lanes by 1, 2, 4, 8
  x = dpp_add<0x112, 0xF>(x);
  x = dpp_add<0x114, 0xF>(x);
  x = dpp_add<0x118, 0xF>(x);
  x = dpp_add<0x142, 0xA>(x);  // lane 15 of rows 0 and 2 to rows 1 and 3
  return dpp_add<0x143, 0xC>(x);  // lane 31 to rows 2 and 3
}

// What a unit covers.
struct Span {
  int q_len, len;  // new tokens and context of the sequence
  int lo, tiles;   // first position read (a multiple of 16), and tiles of each of its units
  int blocks;      // its blocks of R rows
};

template <int R>
__device__ __forceinline__ Span span_of(const KvArgs& p, int b) {
  Span s;
  s.len = seq_len(p, b);
  s.q_len = p.one_each ? 1 : min(max(seq_start(p, b + 1) - seq_start(p, b), 0), p.max_q);
  s.lo = p.window > 0 ? max(0, s.len - s.q_len - p.window + 1) & ~15 : 0;
  s.tiles = max(1, (s.len - s.lo + kTile - 1) / kTile);
  s.blocks = p.mixed && s.q_len * p.group > kFewRows ? 0 : (s.q_len * p.group + R - 1) / R;
  return s;
}

template <Out O, int D, int RT>
__global__ __launch_bounds__(kThreads, 2) void few_kernel(KvArgs p) {
  constexpr int R = 16 * RT;
  constexpr int NG = 2, DEPTH = 2;   // groups of 16 positions in a wave's step, steps in flight
  constexpr int kStep = 16 * NG;
  constexpr int NJ = D / 32;       // k steps of Q K^T; dwords of K codes a lane loads per position
  constexpr int E = D / 16;        // dims of a lane in V; output tiles
  constexpr int OS = D + 4;        // LDS row of the joining buffer (padded)
  constexpr int SLOT = R * (D + 4);  // floats of a part
  using L = PageLayout<D>;
  __shared__ float sh_o[4][R][OS];
  __shared__ float sh_m[4][R], sh_l[4][R];
  __shared__ int sh_sum[2][4], sh_at[2], sh_last;

  const int tid = threadIdx.x, wave = __builtin_amdgcn_readfirstlane(tid >> 6), lane = tid & 63;
  const int c = lane & 15, g = lane >> 4;
  const int H = p.kv_heads, G = p.group;
  const int P = 1 << p.page_shift;

  // ---- how the work is divided: all threads look at the sequences together
  const int per_thread = (p.num_seqs + kThreads - 1) / kThreads;
  auto block_sums = [&](int a, int b2, int& sum_a, int& sum_b, int& before) {  // and a's sum over earlier threads
    int incl = wave_scan(a);
    b2 = wave_scan(b2);
    if (lane == 63) sh_sum[0][wave] = incl, sh_sum[1][wave] = b2;
    __syncthreads();
    sum_a = sum_b = 0;
#pragma unroll
    for (int w = 0; w < 4; ++w) {
      if (w < wave) incl += sh_sum[0][w];
      sum_a += sh_sum[0][w];
      sum_b += sh_sum[1][w];
    }
    before = incl - a;
    __syncthreads();
  };
  int tiles = 0, units = 0;
  for (int i = 0; i < per_thread; ++i) {
    const int b = tid * per_thread + i;
    if (b < p.num_seqs) {
      const Span s = span_of<R>(p, b);
      const int n = s.blocks * H;
      tiles += n * s.tiles;
      units += n;
    }
  }
  int all_tiles, all_units, before;
  block_sums(tiles, units, all_tiles, all_units, before);
  // Few units: each is cut in pieces of about `piece` tiles, one piece per workgroup.  Many: their tiles
  // and kUnitCost more for each form one line, of which every workgroup takes an equal run.
  const bool pieces = 2 * all_units <= (int)gridDim.x;
  const int piece = pieces ? max(kMinTiles, (all_tiles + (int)gridDim.x - all_units - 1) / ((int)gridDim.x - all_units)) : 1;
  auto items = [&](const Span& s) { return pieces ? (s.tiles + piece - 1) / piece : s.tiles + kUnitCost; };
  int mine = 0;
  for (int i = 0; i < per_thread; ++i) {
    const int b = tid * per_thread + i;
    if (b < p.num_seqs) {
      const Span s = span_of<R>(p, b);
      mine += s.blocks * H * items(s);
    }
  }
  int total, unused;
  block_sums(mine, 0, total, unused, before);
  const int per = pieces ? 1 : (total + (int)gridDim.x - 1) / (int)gridDim.x;
  const int run0 = blockIdx.x * per;
  if (run0 >= total) return;
  const int run1 = min(run0 + per, total);
  if (before <= run0 && run0 < before + mine) {  // the one thread whose sequences hold the run's start
    int at = before, b = tid * per_thread;
    for (;; ++b) {
      const Span s = span_of<R>(p, b);
      const int n = s.blocks * H * items(s);
      if (run0 < at + n) break;
      at += n;
    }
    sh_at[0] = b;
    sh_at[1] = at;
  }
  __syncthreads();
  int b = __builtin_amdgcn_readfirstlane(sh_at[0]);
  int seq0 = __builtin_amdgcn_readfirstlane(sh_at[1]);  // line position of sequence b's first item

  for (int x = run0; x < run1;) {
    Span s = span_of<R>(p, b);
    int len = items(s);
    while (x >= seq0 + s.blocks * H * len) {
      seq0 += s.blocks * H * len;
      ++b;
      s = span_of<R>(p, b);
      len = items(s);
    }
    const int unit = (x - seq0) / len;
    const int u0 = seq0 + unit * len, u1 = u0 + len;  // the unit's items on the line
    const int rb = unit / H, h = unit - rb * H;
    const int x1 = min(run1, u1);
    const int real = pieces ? u0 : u0 + kUnitCost;  // the first item that is work
    if (x1 <= real) {
      x = x1;
      continue;
    }
    // its tiles here
    const int tile0 = pieces ? piece_begin(x - u0, len, s.tiles) : max(x - real, 0);
    const int tile1 = pieces ? piece_begin(x1 - u0, len, s.tiles) : x1 - real;
    const int first_token = p.one_each ? b : seq_start(p, b);
    const int rows = min(R, s.q_len * G - rb * R);
    const bool causal = !(p.flags & BSG_KV_NONCAUSAL);
    const int pos0 = s.len - s.q_len;  // position of the sequence's first new token
    // positions seen by some row of the block
    const int i_first = rb * R / G, i_last = (rb * R + rows - 1) / G;
    const int lo = p.window > 0 ? max(0, pos0 + i_first - p.window + 1) : 0;
    const int hi = causal ? max(0, pos0 + i_last + 1) : s.len;
    const int s0 = max(s.lo + tile0 * kTile, lo & ~15), s1 = min(s.lo + tile1 * kTile, hi);

    // ---- this wave's positions
    const int steps = s1 > s0 ? (s1 - s0 + kStep - 1) / kStep : 0;
    const int per_wave = (steps + 3) / 4;
    const int w0 = s0 + wave * per_wave * kStep, w1 = min(s1, w0 + per_wave * kStep);
    const int* table = p.pages + (int64_t)b * p.pages_stride;
    const int last_pos = max(hi - 1, 0), chunk = L::chunk(P);
    // page numbers of the next 64 pages, one per lane
    int page_base = min(w0, last_pos) >> p.page_shift;
    int page_ids = clamp_page(p, table[min(page_base + lane, last_pos >> p.page_shift)]);
    // the queries' loads are issued before the codes', and used after them
    v4i raw[RT][NJ];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int r = 16 * t + c;
      load_query<D>(p, first_token, h, rb * R + (r < rows ? r : 0), g, raw[t]);
    }
    // a step's codes: NG groups of 16 positions, DEPTH steps in flight
    uint32_t kq[DEPTH][NG][NJ], ks[DEPTH][NG], vq[DEPTH][NG][4], vs[DEPTH][NG];
    // a lane's offsets from a group's codes and scales
    const uint32_t k_lane = c * L::kRow + g * (4 * NJ), ks_lane = c * L::kBlocks + g * (D / 64);
    const uint32_t v_lane = 4 * g * L::kRow + c * (E / 2), vs_lane = (c * E / 16) * P + 4 * g;
    auto load = [&](int d, int t0) {
#pragma unroll
      for (int gr = 0; gr < NG; ++gr) {
        const int t = min(t0 + 16 * gr, last_pos & ~15);  // (clamped into the context)
        const int page = t >> p.page_shift;
        if (page - page_base >= 64) {
          page_base = page;
          page_ids = clamp_page(p, table[min(page_base + lane, last_pos >> p.page_shift)]);
        }
        const int slot = t & (P - 1);
        const uint8_t* at = p.cache + (int64_t)__builtin_amdgcn_readlane(page_ids, page - page_base) * p.page_stride +
                            (int64_t)h * chunk;
        const uint8_t *k_codes = at + slot * L::kRow, *k_scales = at + L::k_scales(P) + slot * L::kBlocks;
        const uint8_t *v_codes = at + L::v_codes(P) + slot * L::kRow, *v_scales = at + L::v_scales(P) + slot;
        if constexpr (D == 128) {
          const v4i w = *(const v4i*)(k_codes + k_lane);
#pragma unroll
          for (int k = 0; k < NJ; ++k) kq[d][gr][k] = (uint32_t)w[k];
          ks[d][gr] = *(const uint16_t*)(k_scales + ks_lane);
        } else {
          const uint2 w = *(const uint2*)(k_codes + k_lane);
          kq[d][gr][0] = w.x;
          kq[d][gr][1] = w.y;
          ks[d][gr] = k_scales[ks_lane];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
          vq[d][gr][k] = E == 8 ? *(const uint32_t*)(v_codes + v_lane + k * L::kRow) : *(const uint16_t*)(v_codes + v_lane + k * L::kRow);
        vs[d][gr] = *(const uint32_t*)(v_scales + vs_lane);
      }
    };
    v8h q[RT][NJ];
    float mul[RT];   // base-2 score of one accumulator unit
    int pos[RT];     // the row's position: it sees (pos - window, pos]
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const int r = 16 * t + c, row = rb * R + (r < rows ? r : 0);
      convert_query<O, D>(p, raw[t], q[t], mul[t]);
      pos[t] = causal ? pos0 + row / G : s.len - 1;
    }

    v4f o[RT][E];
    float m[RT], l[RT];
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      m[t] = kNegInf;
      l[t] = 0.0f;
#pragma unroll
      for (int e = 0; e < E; ++e) o[t][e] = v4f{0, 0, 0, 0};
    }

    if (w0 < w1) {
      const int first_pos = causal ? pos0 + i_first : s.len - 1, last_row_pos = causal ? pos0 + i_last : s.len - 1;
      auto step = [&](int d, int t0) {
        // -- scores
        v4f sc[RT][NG];
#pragma unroll
        for (int gr = 0; gr < NG; ++gr) {
          const uint32_t sp = scale_pair<kLow>(ks[d][gr]);
          const uint32_t sp0 = f16x2_splat_lo(sp), sp1 = f16x2_splat_hi(sp);
#pragma unroll
          for (int t = 0; t < RT; ++t) sc[t][gr] = v4f{0, 0, 0, 0};
#pragma unroll
          for (int k = 0; k < NJ; ++k) {
            const v8h a = __builtin_bit_cast(v8h, e2m1x8_scaled_f16x8(kq[d][gr][k], k < 2 ? sp0 : sp1));
#pragma unroll
            for (int t = 0; t < RT; ++t)
              sc[t][gr] = __builtin_amdgcn_mfma_f32_16x16x32_f16(a, q[t][k], sc[t][gr], 0, 0, 0);
          }
        }
        // -- masks: only where a row does not see the whole step
        const bool edge = t0 + kStep - 1 > min(first_pos, w1 - 1) || (p.window > 0 && t0 <= last_row_pos - p.window);
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          if (p.cap > 0.0f) soft_cap<NG>(p, mul[t], sc[t]);
          if (edge) {
            const int first = t0 + 4 * rare(g), top = min(pos[t], w1 - 1), bottom = p.window > 0 ? pos[t] - p.window : -1;
#pragma unroll
            for (int gr = 0; gr < NG; ++gr)
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const int at = first + 16 * gr + i;
                sc[t][gr][i] = at <= top && at > bottom ? sc[t][gr][i] : kNegInf;
              }
          }
        }
        uint32_t nan_codes = 0;
        if (edge) {
          // positions that no row sees count as zero, whatever their slots hold; NaN blocks seen by
          // some rows only are taken out here and given to those rows below
          const int first = t0 + 4 * rare(g), from = max(lo, w0), to = w1;
#pragma unroll
          for (int gr = 0; gr < NG; ++gr) {
            uint32_t keep = 0;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int at = first + 16 * gr + i;
              if (at >= from && at < to) keep |= 0xFFu << (8 * i);
            }
            vs[d][gr] &= keep;
            const uint32_t bad = ((vs[d][gr] + 0x01010101u) & 0x80808080u) >> 7;  // 1 in each byte that is 0x7F
            nan_codes |= bad;
            vs[d][gr] &= ~(bad * 0x7Fu);
          }
        }
        // -- softmax
        v8h pt[RT][NG / 2];
#pragma unroll
        for (int t = 0; t < RT; ++t) {
          float top = sc[t][0][0];
#pragma unroll
          for (int gr = 0; gr < NG; ++gr)
#pragma unroll
            for (int i = 0; i < 4; ++i) top = __builtin_fmaxf(top, sc[t][gr][i]);
          if (__any(top > m[t])) {  // (replacing m less often saves nothing here: 79.9 and 79.6 us for the 64 tokens above)
            const float grown = __builtin_fmaxf(m[t], max_over_g(top));
            const float f = grown == kNegInf ? 1.0f : __builtin_amdgcn_exp2f((m[t] - grown) * mul[t]);
            m[t] = grown;
            l[t] *= f;
#pragma unroll
            for (int e = 0; e < E; ++e) o[t][e] *= f;
          }
          const float off = m[t] == kNegInf ? 0.0f : kPBias - m[t] * mul[t];
#pragma unroll
          for (int k = 0; k < NG / 2; ++k)
#pragma unroll
            for (int half = 0; half < 2; ++half) {
              float e4[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                e4[i] = __builtin_amdgcn_exp2f(__builtin_fmaf(sc[t][2 * k + half][i], mul[t], off));
                l[t] += e4[i];
              }
              const v2h a = __builtin_convertvector((v2f{e4[0], e4[1]}), v2h), bb = __builtin_convertvector((v2f{e4[2], e4[3]}), v2h);
              pt[t][k][4 * half] = a[0];
              pt[t][k][4 * half + 1] = a[1];
              pt[t][k][4 * half + 2] = bb[0];
              pt[t][k][4 * half + 3] = bb[1];
            }
        }
        // -- O^T += V^T P^T
#pragma unroll
        for (int k = 0; k < NG / 2; ++k) {
          v4i frag[E];
#pragma unroll
          for (int jj = 0; jj < 4; ++jj) {  // pairs of positions: two of each 16
            const int gr = 2 * k + jj / 2, x2 = (jj & 1) * 2;
            const v2h s2 = __builtin_bit_cast(v2h, (jj & 1) ? scale_pair<kHigh>(vs[d][gr]) : scale_pair<kLow>(vs[d][gr]));
            const uint32_t a = vq[d][gr][x2], bb = vq[d][gr][x2 + 1], mask = 0x0F0F0F0Fu;
            const uint32_t even = (a & mask) | ((bb << 4) & ~mask), odd = ((a >> 4) & mask) | (bb & ~mask);
#pragma unroll
            for (int e = 0; e < E; e += 2) {
              frag[e][jj] = __builtin_bit_cast(int, fp4_pair(even, e / 2) * s2);
              frag[e + 1][jj] = __builtin_bit_cast(int, fp4_pair(odd, e / 2) * s2);
            }
          }
#pragma unroll
          for (int e = 0; e < E; ++e)
#pragma unroll
            for (int t = 0; t < RT; ++t)
              o[t][e] = __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(v8h, frag[e]), pt[t][k], o[t][e], 0, 0, 0);
        }
        if (__any(nan_codes)) {
          // rare: a NaN block among positions that not every row sees.  Output element i of tile e is
          // dim E (4g + i) + e, so element i lies in block E (4g + i) / 16.
          for (int at = max(t0, max(lo, w0)); at < min(t0 + kStep, w1); ++at) {
            const int page = clamp_page(p, table[at >> p.page_shift]), sl = at & (P - 1);
            const uint8_t* codes = p.cache + (int64_t)page * p.page_stride + (int64_t)h * chunk + L::v_scales(P) + sl;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const bool bad = codes[E * (4 * rare(g) + i) / 16 * P] == 0x7F;
#pragma unroll
              for (int t = 0; t < RT; ++t)
                if (bad && at <= pos[t] && (p.window <= 0 || at > pos[t] - p.window))
#pragma unroll
                  for (int e = 0; e < E; ++e) o[t][e][i] = __builtin_nanf("");
            }
          }
        }
      };
#pragma unroll
      for (int d = 0; d < DEPTH; ++d) load(d, w0 + d * kStep);
      int t0 = w0;
      for (; t0 + (DEPTH - 1) * kStep < w1; t0 += DEPTH * kStep) {
#pragma unroll
        for (int d = 0; d < DEPTH; ++d) {
          step(d, t0 + d * kStep);
          load(d, t0 + (d + DEPTH) * kStep);
        }
      }
#pragma unroll
      for (int d = 0; d < DEPTH - 1; ++d)
        if (t0 + d * kStep < w1) step(d, t0 + d * kStep);
    }

    // a scaled maximum from here on
#pragma unroll
    for (int t = 0; t < RT; ++t)
      if (m[t] != kNegInf) m[t] *= mul[t];

    // ---- join the waves
#pragma unroll
    for (int t = 0; t < RT; ++t) {
      const float sum = sum_over_g(l[t]);
      const int r = 16 * t + c;
      if (g == 0) {
        sh_m[wave][r] = m[t];
        sh_l[wave][r] = sum;
      }
      if (sum != 0.0f) {  // a NaN row counts
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int e = 0; e < E; e += 4)
            *(v4f*)&sh_o[wave][r][E * (4 * g + i) + e] = v4f{o[t][e][i], o[t][e + 1][i], o[t][e + 2][i], o[t][e + 3][i]};
      }
    }
    __syncthreads();
    const bool whole = x <= real && x1 >= u1;
    const int wg0 = real / per, wgs = (u1 - 1) / per - wg0 + 1;  // the workgroups that share the unit
    // Slot of the part that workgroup wg0 + k left: 2 (wg0 + k), or one more where the unit starts inside
    // that workgroup's run.
    auto slot_of = [&](int k) { return 2 * (wg0 + k) + (real >= (wg0 + k) * per ? 1 : 0); };
    const __amdgpu_buffer_rsrc_t parts = handoff_buffer(p.part, 2u * gridDim.x * SLOT * 4u);
    // element (row r, dims d .. d+3)
    auto store_out = [&](int r, int d, v4f y, float top, float sum) {
      const int i = (rb * R + r) / G, hq = rb * R + r - i * G;
      const float f = 256.0f / sum, gain = p.v_scale;  // (one after the other: v_scale may be near fp32's ends)
      const bool none = sum == 0.0f;                   // an empty row gives zeros
      uint16_t* dst = (uint16_t*)p.out.ptr + (int64_t)(first_token + i) * p.out.token_stride +
                      (int64_t)(h * G + hq) * p.out.head_stride + d;
      const uint32_t a = out_bits<O>(none ? 0.0f : y[0] * f * gain), bq = out_bits<O>(none ? 0.0f : y[1] * f * gain);
      const uint32_t cc = out_bits<O>(none ? 0.0f : y[2] * f * gain), dd = out_bits<O>(none ? 0.0f : y[3] * f * gain);
      *(uint2*)dst = make_uint2(a | bq << 16, cc | dd << 16);
      if (p.lse && d == 0)
        p.lse[(int64_t)(first_token + i) * p.q_heads + h * G + hq] =
            none ? kNegInf : (top - kPBias + __builtin_amdgcn_logf(sum)) * 0.693147180559945309f;
    };
    // part: R rows of D outputs, then (maximum, sum) of each row in a group of four floats
    auto store_part = [&](int slot, int r, int d, v4f y, float top, float sum) {
      handoff_store4(parts, slot * SLOT + r * D + d, y);
      if (d == 0) handoff_store4(parts, slot * SLOT + R * D + 4 * r, v4f{top, sum, 0.0f, 0.0f});
    };
    for (int k = tid; k < rows * (D / 4); k += kThreads) {
      const int r = k / (D / 4), d = k % (D / 4) * 4;
      float top = kNegInf, sum = 0.0f;
#pragma unroll
      for (int w = 0; w < 4; ++w) top = __builtin_fmaxf(top, sh_m[w][r]);
      v4f y = {0, 0, 0, 0};
#pragma unroll
      for (int w = 0; w < 4; ++w)
        if (sh_l[w][r] != 0.0f) {
          const float f = sh_m[w][r] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(sh_m[w][r] - top);
          sum += f * sh_l[w][r];
          y += f * *(const v4f*)&sh_o[w][r][d];
        }
      if (whole) store_out(r, d, y, top, sum);
      else store_part(slot_of(blockIdx.x - wg0), r, d, y, top, sum);
    }
    if (!whole) {
      // ---- the last workgroup of the unit joins the parts: in groups of kJoin, each joined by its own
      // last one, where there are many
      // joined part of workgroups wg0 + first + step * i, i < n, for this thread's elements
      auto join = [&](int first, int step, int n, bool final, int slot) {
        for (int k = tid; k < rows * (D / 4); k += kThreads) {
          const int r = k / (D / 4), d = k % (D / 4) * 4;
          float top = kNegInf, sum = 0.0f;
          v4f y = {0, 0, 0, 0};
          for (int i0 = 0; i0 < n; i0 += kJoin) {
            v4f ms[kJoin], ys[kJoin];
#pragma unroll
            for (int i = 0; i < kJoin; ++i) {  // all loads in flight at once; a repeated last part counts nothing
              const uint32_t at = slot_of(first + step * min(i0 + i, n - 1)) * SLOT;
              ms[i] = handoff_load4(parts, at + R * D + 4 * r);
              ys[i] = handoff_load4(parts, at + r * D + d);
            }
            float grown = top;
#pragma unroll
            for (int i = 0; i < kJoin; ++i) grown = __builtin_fmaxf(grown, ms[i][0]);
            const float f0 = top == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(top - grown);
            y *= f0;
            sum *= f0;
#pragma unroll
            for (int i = 0; i < kJoin; ++i)
              if (i0 + i < n) {
                const float f = ms[i][0] == kNegInf ? 0.0f : __builtin_amdgcn_exp2f(ms[i][0] - grown);
                sum += f * ms[i][1];
                y += f * ys[i];
              }
            top = grown;
          }
          if (final) store_out(r, d, y, top, sum);
          else store_part(slot, r, d, y, top, sum);
        }
      };
      int* unit_counter = p.arrived + ((int64_t)first_token * G + (int64_t)rb * R) * H + h;
      if (wgs <= kJoin) {
        if (last_arrival(unit_counter, wgs, &sh_last)) join(0, 1, wgs, true, 0);
      } else {
        const int k0 = (blockIdx.x - wg0) / kJoin * kJoin, n = min(kJoin, wgs - k0);
        if (last_arrival(p.group_arrived + slot_of(k0), n, &sh_last)) {
          join(k0, 1, n, false, slot_of(k0));
          if (last_arrival(unit_counter, (wgs + kJoin - 1) / kJoin, &sh_last)) join(0, kJoin, (wgs + kJoin - 1) / kJoin, true, 0);
        }
      }
    }
    __syncthreads();  // the joining buffers are free again
    x = x1;
  }
}

template <Out O, int D>
hipError_t launch(const KvArgs& a, int cus, hipStream_t stream) {
  KvArgs args = a;
  void* argv[] = {&args};
  // Of a mixed batch most short sequences have one new token: 16 rows, and two blocks for the others.
  const int64_t rows = (int64_t)(a.mixed ? 1 : a.max_q) * a.group;
  const int R = rows <= 16 ? 16 : 32;
  const int64_t tiles = (context_positions(a.window, a.max_q, a.max_kv) + kTile - 1) / kTile + 1;
  // units: sum over sequences of ceil(tokens * group / R), at most one partial block each
  const int64_t units = ((int64_t)a.num_tokens * a.group / R + a.num_seqs) * a.kv_heads;
  const int64_t want = units * ((tiles + kMinTiles - 1) / kMinTiles), most = (int64_t)cus * kWgPerCu;
  const dim3 grid((unsigned)(want < most ? want : most));
  const void* fn = R == 16 ? (const void*)&few_kernel<O, D, 1> : (const void*)&few_kernel<O, D, 2>;
  return hipLaunchKernel(fn, grid, dim3(kThreads), argv, 0, stream);
}

}  // namespace

// One token and whole prompts may share a batch.  Sequences of up to kFewRows rows are then left to the
// few-row kernel and the others to the many-row kernel, which would walk a long context for a few rows with
// one workgroup (a prompt of 512 tokens beside 63 single tokens at 1000 to 16000 positions, 32 heads on 8 of
// 128 dims: 2073 us by that kernel alone, 208 by both).  The host does not know the sequences' tokens: it
// looks for uneven batches in which the sequences besides a longest one must be short on average, or of eight and
// more.  Eight is a compromise: a launch that finds nothing to do costs 2 to 3 us at any number (8 prompts of 100 to 500
// tokens 84 us by one kernel, 87 by both), and what short sequences gain depends on their contexts, which the host does not
// know (4 prompts of 300 tokens and 4 single ones, 32 heads on 8 of 128 dims: single ones over 4000 positions 105 and 54
// us, over 1000 38 and 48 us; with 2 of each 70 and 56, 42 and 51 us).
hipError_t kv_attend_launch(const KvArgs& args, int dtype, int head_dim, int cus, hipStream_t stream) {
  KvArgs a = args;
  a.mixed = mixed_batch(a.num_tokens, a.num_seqs, a.max_q, a.group);
  if ((int64_t)a.max_q * a.group > kFewRows) {
    const hipError_t e = kv_attend_rows_launch(a, dtype, head_dim, cus, stream);
    if (e != hipSuccess || !a.mixed) return e;
  }
  if (head_dim == 64) return dtype ? launch<Out::F16, 64>(a, cus, stream) : launch<Out::BF16, 64>(a, cus, stream);
  return dtype ? launch<Out::F16, 128>(a, cus, stream) : launch<Out::BF16, 128>(a, cus, stream);
}

void kv_workspace(const bsg_kv_problem& p, int cus, size_t* part_floats, size_t* counters, size_t* group_counters) {
  const size_t slots = (size_t)cus * kWgPerCu * 2;
  const size_t rows = kv_rows_part_floats(p, cus);
  *part_floats = slots * 32 * (p.head_dim + 4);
  if (*part_floats < rows) *part_floats = rows;
  *counters = slots + (size_t)p.max_tokens * p.q_heads;
  *group_counters = slots;
}

}  // namespace bsg
