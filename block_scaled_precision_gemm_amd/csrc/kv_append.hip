// Storing new keys and values in the paged NVFP4 cache, rotating keys and queries on the way, and
// reading stored positions back.
//
// A lane holds 8 consecutive dims of one head row, so D/8 lanes hold a row and two neighbours a
// block of 16.  The rotation partner of a lane's dims is in its own 8 dims (interleaved pairs) or
// R/2 dims away (halves); the latter are read from memory a second time, which hits the L1 line
// that the partner lane fetches.
//
// Quantisation (bsg_kv.h) without a division per element: with s of at most 4 significant bits and
// r = fl(1/s), z0 = fl(y r) and z = fl(z0 + r fl(y - z0 s)) is the correctly rounded y / s.  Its
// rounding to E2M1 is then the rounding of the exact quotient: E2M1's halfway points t and s are
// short enough that t s is exact, so y / s = t (1 + e) with e != 0 never rounds to t itself.
// Products and sums of the rotation are rounded one by one (no fused multiply-add), so that a value
// does not depend on which of its two products a compiler would fuse.
//
// Bound: bytes.  Per token (q_heads + 2 kv_heads) D 16-bit values in, q_heads D 16-bit values and
// 2 kv_heads D 9/16 bytes out.  Measured: 4096 tokens of 32 + 2 x 8 heads of 128 in 22.8 us (4.1 TB/s), reading
// them back 7.8 us (3.3 TB/s); one token 4.2 and 2.8 us, a launch's own time for the most part.
#include "kv.h"

namespace bsg {
namespace {

#pragma clang fp contract(off)

constexpr int kThreads = 256;

template <Out O>
__device__ __forceinline__ void unpack8(v4i w, float x[8]) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t u = (uint32_t)w[i];
    if constexpr (O == Out::BF16) {
      x[2 * i] = __builtin_bit_cast(float, u << 16);
      x[2 * i + 1] = __builtin_bit_cast(float, u & 0xFFFF0000u);
    } else {
      const v2h h = __builtin_bit_cast(v2h, u);
      x[2 * i] = (float)h[0];
      x[2 * i + 1] = (float)h[1];
    }
  }
}

typedef float v2f __attribute__((ext_vector_type(2)));
typedef __bf16 v2b __attribute__((ext_vector_type(2)));

template <Out O>
__device__ __forceinline__ v4i pack8(const float x[8]) {
  v4i w;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const v2f p = {x[2 * i], x[2 * i + 1]};
    if constexpr (O == Out::BF16) w[i] = __builtin_bit_cast(int, __builtin_convertvector(p, v2b));
    else w[i] = __builtin_bit_cast(int, __builtin_convertvector(p, v2h));
  }
  return w;
}

// The sequence of token t: the last b with q_start[b] <= t, found by the W lanes of a row together
// (each step compares W pivots and keeps one of the W parts).
template <int W>
__device__ __forceinline__ int seq_of(const KvArgs& p, int t, int lane_in_row, int row_shift) {
  if (p.one_each) return t;
  int lo = 0, n = p.num_seqs;
  while (n > 1) {
    const int step = (n + W - 1) / W;
    const int idx = lane_in_row * step;
    const bool le = idx < n && p.q_start[lo + idx] <= t;
    const uint32_t mask = (uint32_t)(__ballot(le) >> row_shift) & ((1u << W) - 1u);
    const int parts = max(__popc(mask), 1) - 1;
    lo += parts * step;
    n = min(step, n - parts * step);
  }
  return lo;
}

// Where token t is stored: position, and the byte offset of its page's head 0 chunk plus its slot.
struct Place {
  int pos;        // position (rotation), may be negative for a token that is not stored
  int slot;       // slot in the page
  int64_t page;   // byte offset of the page, or -1: not stored
};

template <int W>
__device__ __forceinline__ Place place_of(const KvArgs& p, int t, int lane_in_row, int row_shift) {
  const int b = seq_of<W>(p, t, lane_in_row, row_shift);
  Place r;
  int first, next, len = p.kv_len[b];
  if (p.one_each) {
    first = t;
    next = t + 1;
  } else {
    first = p.q_start[b];
    next = p.q_start[b + 1];
  }
  r.pos = len - (next - first) + (t - first);
  r.slot = r.pos & ((1 << p.page_shift) - 1);
  r.page = -1;
  if (r.pos >= 0 && r.pos < p.max_kv) {
    const int page = p.pages[(int64_t)b * p.pages_stride + (r.pos >> p.page_shift)];
    if (page >= 0 && page < p.num_pages) r.page = (int64_t)page * p.page_stride;
  }
  return r;
}

// Rotate the 8 dims of a lane: x, with y the partner dims (halves) or unused (neighbours).
__device__ __forceinline__ void rotate8(float x[8], const float y[8], const float cs[8], const float sn[8], bool inter, bool upper) {
  if (inter) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = x[2 * i], b = x[2 * i + 1];
      x[2 * i] = a * cs[i] - b * sn[i];
      x[2 * i + 1] = b * cs[i] + a * sn[i];
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float mine = x[i] * cs[i], other = y[i] * sn[i];
      x[i] = upper ? mine + other : mine - other;
    }
  }
}

// A block's eight elements of this lane (the neighbour lane has the other eight): packed codes, and the
// scale's code.
__device__ __forceinline__ uint32_t quantize8(float x[8], float inv, int& code) {
  float amax = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    x[i] = x[i] * inv;
    amax = __builtin_elementwise_maximum(amax, __builtin_fabsf(x[i]));  // keeps a NaN
  }
  amax = __builtin_elementwise_maximum(amax, __shfl_xor(amax, 1));
  const bool nan = amax != amax;
  const float s_raw = fminf(amax * (1.0f / 6.0f), 448.0f);
  code = nan ? 0x7F : __builtin_amdgcn_cvt_pk_fp8_f32(s_raw, 0.0f, 0, false) & 0x7F;
  const float s = nan ? 0.0f : __builtin_amdgcn_cvt_f32_fp8(code, 0);
  const float r = s > 0.0f ? 1.0f / s : 0.0f;
  uint32_t q = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float z[2];
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      // beyond 3 * 448 * 6 every element saturates: the clamp keeps infinities out of the correction
      const float y = __builtin_amdgcn_fmed3f(x[2 * i + j], -8192.0f, 8192.0f);
      const float z0 = y * r;
      z[j] = __builtin_copysignf(__builtin_fmaf(__builtin_fmaf(-z0, s, y), r, z0), y);  // (of y = -0 the correction is +0)
    }
    // the byte to replace is an immediate
    if (i == 0) q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, z[0], z[1], 1.0f, 0);
    if (i == 1) q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, z[0], z[1], 1.0f, 1);
    if (i == 2) q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, z[0], z[1], 1.0f, 2);
    if (i == 3) q = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(q, z[0], z[1], 1.0f, 3);
  }
  return q;
}

// Workgroup (x, y): ROWS tokens, and heads NB y .. NB y + NB - 1 of (keys, values, queries).  A lane's
// rotation factors and place serve all of them, and their loads are in flight together.
template <Out O, int D, int NB>
__global__ __launch_bounds__(kThreads) void append_kernel(KvArgs p, int heads) {
  constexpr int W = D / 8, ROWS = kThreads / W;
  const int tid = threadIdx.x, c = tid % W, row_shift = (tid & 63) / W * W;
  const int t = blockIdx.x * ROWS + tid / W;
  const bool live = t < p.num_tokens;
  const int tt = live ? t : p.num_tokens - 1;  // idle rows follow the last token, and store nothing
  const int R = 2 * p.rope_half, d0 = 8 * c;
  const bool inter = p.flags & BSG_KV_ROPE_INTERLEAVED, turns = d0 < R;
  const bool upper = d0 >= p.rope_half;  // halves: this lane holds the second of each pair
  const int d1 = !turns || inter ? d0 : upper ? d0 - p.rope_half : d0 + p.rope_half;  // the partners' dims
  v4i w[NB], w2[NB];
#pragma unroll
  for (int k = 0; k < NB; ++k) {
    const int h = min((int)blockIdx.y * NB + k, heads - 1);
    const int kind = h < p.kv_heads ? 0 : h < 2 * p.kv_heads ? 1 : 2;
    const int hh = kind == 0 ? h : kind == 1 ? h - p.kv_heads : h - 2 * p.kv_heads;
    const HeadsArg& src = kind == 0 ? p.k : kind == 1 ? p.v : p.q;
    const uint16_t* row = (const uint16_t*)src.ptr + (int64_t)tt * src.token_stride + (int64_t)hh * src.head_stride;
    w[k] = *(const v4i*)(row + d0);
    w2[k] = kind == 1 || inter ? w[k] : *(const v4i*)(row + d1);
  }
  const Place at = place_of<W>(p, tt, c, row_shift);
  float cs[8], sn[8];
  if (turns) {
    const float* tab = p.rope + (int64_t)min(max(at.pos, 0), p.max_kv - 1) * R;
    const int i0 = inter ? d0 / 2 : upper ? d0 - p.rope_half : d0;
    const v4f c0 = *(const v4f*)(tab + i0), s0 = *(const v4f*)(tab + p.rope_half + i0);
    const int i1 = inter ? i0 : i0 + 4;
    const v4f c1 = *(const v4f*)(tab + i1), s1 = *(const v4f*)(tab + p.rope_half + i1);
#pragma unroll
    for (int i = 0; i < 4; ++i) cs[i] = c0[i], cs[4 + i] = c1[i], sn[i] = s0[i], sn[4 + i] = s1[i];
  }
#pragma unroll
  for (int k = 0; k < NB; ++k) {
    const int h = blockIdx.y * NB + k;
    if (h >= heads) break;
    const int kind = h < p.kv_heads ? 0 : h < 2 * p.kv_heads ? 1 : 2;
    const int hh = kind == 0 ? h : kind == 1 ? h - p.kv_heads : h - 2 * p.kv_heads;
    float x[8];
    unpack8<O>(w[k], x);
    if (turns && kind != 1) {
      float y[8];
      unpack8<O>(w2[k], y);
      rotate8(x, y, cs, sn, inter, upper);
    }
    if (kind == 2) {
      v4i* dst = (v4i*)((uint16_t*)p.out.ptr + (int64_t)t * p.out.token_stride + (int64_t)hh * p.out.head_stride + d0);
      if (live) {
        if constexpr (NB > 1) __builtin_nontemporal_store(pack8<O>(x), dst);  // (more than the L2s hold; 24.1 -> 22.8 us)
        else *dst = pack8<O>(x);
      }
      continue;
    }
    int code;
    const uint32_t q = quantize8(x, kind == 0 ? p.k_inv : p.v_inv, code);
    if (!live || at.page < 0) continue;
    using L = PageLayout<D>;
    const int P = 1 << p.page_shift;
    uint8_t* chunk = p.cache + at.page + (int64_t)hh * L::chunk(P);
    *(uint32_t*)(chunk + (kind ? L::v_codes(P) : 0) + at.slot * L::kRow + 4 * c) = q;
    if (!(c & 1)) {
      if (kind) chunk[L::v_scales(P) + (c >> 1) * P + at.slot] = (uint8_t)code;
      else chunk[L::k_scales(P) + at.slot * L::kBlocks + (c >> 1)] = (uint8_t)code;
    }
  }
}

// Eight E2M1 codes times s, in fp32 (exact), times the global scale g (one rounding).
__device__ __forceinline__ void values8(uint32_t q, float s, float g, float x[8]) {
  const v2f a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 0), b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 1);
  const v2f c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 2), d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(q, 1.0f, 3);
  const float v[8] = {a[0], a[1], b[0], b[1], c[0], c[1], d[0], d[1]};
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] = v[i] * s * g;
}

template <Out O, int D>
__global__ __launch_bounds__(kThreads) void read_kernel(KvArgs p) {
  constexpr int W = D / 8, ROWS = kThreads / W;
  const int tid = threadIdx.x, c = tid % W, row_shift = (tid & 63) / W * W;
  const int t = blockIdx.x * ROWS + tid / W;
  const bool is_v = (int)blockIdx.y >= p.kv_heads;
  const int h = is_v ? blockIdx.y - p.kv_heads : blockIdx.y;
  const int tt = min(t, p.num_tokens - 1);
  const Place at = place_of<W>(p, tt, c, row_shift);
  float x[8] = {};
  if (at.page >= 0) {
    using L = PageLayout<D>;
    const int P = 1 << p.page_shift;
    const uint8_t* chunk = p.cache + at.page + (int64_t)h * L::chunk(P);
    const uint32_t q = *(const uint32_t*)(chunk + (is_v ? L::v_codes(P) : 0) + at.slot * L::kRow + 4 * c);
    const int code = is_v ? chunk[L::v_scales(P) + (c >> 1) * P + at.slot]
                          : chunk[L::k_scales(P) + at.slot * L::kBlocks + (c >> 1)];
    values8(q, __builtin_amdgcn_cvt_f32_fp8(code, 0), is_v ? p.v_scale : p.k_scale, x);
  }
  const HeadsArg& dst = is_v ? p.v : p.k;
  if (t < p.num_tokens)
    *(v4i*)((uint16_t*)dst.ptr + (int64_t)t * dst.token_stride + (int64_t)h * dst.head_stride + 8 * c) = pack8<O>(x);
}

template <Out O, int D>
hipError_t launch_append(const KvArgs& a, bool with_q, hipStream_t stream) {
  constexpr int ROWS = kThreads / (D / 8), NB = 4;
  KvArgs args = a;
  int heads = 2 * a.kv_heads + (with_q ? a.q_heads : 0);
  void* argv[] = {&args, &heads};
  const unsigned x = (a.num_tokens + ROWS - 1) / ROWS;
  // Four heads to a workgroup share the rotation factors (4096 tokens, 48 heads of 128: 27.8 us with one
  // head, 24.1 us with four); few tokens are spread over more workgroups, all being latency.
  if ((int64_t)x * heads <= 2048)
    return hipLaunchKernel((const void*)&append_kernel<O, D, 1>, dim3(x, heads), dim3(kThreads), argv, 0, stream);
  return hipLaunchKernel((const void*)&append_kernel<O, D, NB>, dim3(x, (heads + NB - 1) / NB), dim3(kThreads), argv, 0, stream);
}

template <Out O, int D>
hipError_t launch_read(const KvArgs& a, hipStream_t stream) {
  constexpr int ROWS = kThreads / (D / 8);
  KvArgs args = a;
  void* argv[] = {&args};
  const dim3 grid((a.num_tokens + ROWS - 1) / ROWS, 2 * a.kv_heads);
  return hipLaunchKernel((const void*)&read_kernel<O, D>, grid, dim3(kThreads), argv, 0, stream);
}

}  // namespace

hipError_t kv_append_launch(const KvArgs& a, int dtype, int head_dim, bool with_q, hipStream_t stream) {
  if (head_dim == 64)
    return dtype ? launch_append<Out::F16, 64>(a, with_q, stream) : launch_append<Out::BF16, 64>(a, with_q, stream);
  return dtype ? launch_append<Out::F16, 128>(a, with_q, stream) : launch_append<Out::BF16, 128>(a, with_q, stream);
}

hipError_t kv_read_launch(const KvArgs& a, int dtype, int head_dim, hipStream_t stream) {
  if (head_dim == 64) return dtype ? launch_read<Out::F16, 64>(a, stream) : launch_read<Out::BF16, 64>(a, stream);
  return dtype ? launch_read<Out::F16, 128>(a, stream) : launch_read<Out::BF16, 128>(a, stream);
}

}  // namespace bsg
