// C ABI of the products in 8-bit floating point with a scale for each block of 128 (include/bsg_f8.h): plans, argument
// checks and launches.
#include <hip/hip_runtime.h>
#include <stdio.h>
#include <stdlib.h>

#include <new>

#include "f8.h"
#include "f8_cut.h"
#include "plan.h"

struct bsg_f8_plan_s {
  uint32_t magic;
  bsg_f8_problem problem;
  int device, cus, dtype, log_level;
  void* workspace;  // parts of products whose K is split, and their counters, or null
  uint64_t workspace_bytes;
  float* part;
  int* arrived;
};

struct bsg_f8_ffn_plan_s {
  uint32_t magic;
  bsg_f8_ffn_problem problem;
  int device, cus, dtype, log_level;
  void* workspace;
  uint64_t workspace_bytes;
  // parts of the workspace
  uint8_t* x_codes;   // [max_tokens][hidden]
  uint8_t* h_codes;   // [max_tokens][inter]
  float* x_scales;    // [B(hidden)][padded tokens]
  float* h_scales;    // [B(inter)][padded tokens]
  float* h;           // [up to kF8OneTile][inter]: SiLU(gate) up where it is not made codes at once
  float* part;        // as in bsg_f8_plan_s
  int* arrived;
};

namespace {

using bsg::set_error;

constexpr uint32_t kF8Magic = 0x42534738u, kFfnMagic = 0x42534746u;  // "BSG8", "BSGF"
constexpr int64_t kStrideLimit = (int64_t)1 << 22, kScaleStrideLimit = (int64_t)1 << 25;

bool bad_size(int64_t n) { return n < 16 || n % 16 || n > BSG_F8_MAX_SIZE; }

bsg_status check_common(int32_t dtype, uint32_t flags, uint32_t known, const char* a, int64_t an, const char* b, int64_t bn,
                        int64_t max_tokens) {
  if (dtype != BSG_OUT_BF16 && dtype != BSG_OUT_F16) {
    set_error("unsupported dtype %d (BF16 or F16 only)", dtype);
    return BSG_ERR_ABI;
  }
  if (flags & ~known) {
    set_error("unknown flag bits 0x%x", flags);
    return BSG_ERR_ABI;
  }
  if (bad_size(an) || bad_size(bn) || max_tokens < 1 || max_tokens > BSG_F8_MAX_TOKENS) {
    set_error("%s and %s must be multiples of 16 in [16, %d] and max_tokens in [1, %d] (got %lld, %lld, %lld)", a, b,
              BSG_F8_MAX_SIZE, BSG_F8_MAX_TOKENS, (long long)an, (long long)bn, (long long)max_tokens);
    return BSG_ERR_SHAPE;
  }
  return BSG_OK;
}

bsg_status check_tokens(int64_t tokens, int64_t max_tokens) {
  if (tokens >= 0 && tokens <= max_tokens) return BSG_OK;
  set_error("tokens must be in [0, max_tokens = %lld] (got %lld)", (long long)max_tokens, (long long)tokens);
  return BSG_ERR_SHAPE;
}

// A 16-bit tensor of rows: pointer, and elements from row to row.
bsg_status check_rows(const char* name, const void* p, int64_t stride, int64_t cols) {
  if (!p) {
    set_error("null %s", name);
    return BSG_ERR_NULL;
  }
  if (((uintptr_t)p & 15u) || (stride & 7)) {
    set_error("%s must be 16-byte aligned with a stride that is a multiple of 8 elements (got %p, %lld)", name, p,
              (long long)stride);
    return BSG_ERR_ALIGN;
  }
  if (stride < cols || stride >= kStrideLimit) {
    set_error("the stride of %s must be in [%lld, 2^22) (got %lld)", name, (long long)cols, (long long)stride);
    return BSG_ERR_SHAPE;
  }
  return BSG_OK;
}

bsg_status check_codes(const char* name, const void* codes, int64_t stride, const float* scales, int64_t scale_stride,
                       int64_t rows, int64_t cols, bool wide) {
  if (!codes || !scales) {
    set_error("null codes or scales of %s", name);
    return BSG_ERR_NULL;
  }
  if (((uintptr_t)codes & 15u) || ((uintptr_t)scales & (wide ? 15u : 3u)) || (stride & 15) || (scale_stride & 3)) {
    set_error("codes of %s must be 16-byte aligned with a stride that is a multiple of 16, scales %d-byte aligned with a "
              "scale_stride that is a multiple of 4 (got %p, %lld, %p, %lld)", name, wide ? 16 : 4, codes, (long long)stride,
              (const void*)scales, (long long)scale_stride);
    return BSG_ERR_ALIGN;
  }
  if (stride < cols || stride >= kStrideLimit || scale_stride < rows || scale_stride >= kScaleStrideLimit) {
    set_error("the stride of %s must be in [%lld, 2^22) and its scale_stride in [%lld, 2^25) (got %lld, %lld)", name,
              (long long)cols, (long long)rows, (long long)stride, (long long)scale_stride);
    return BSG_ERR_SHAPE;
  }
  return BSG_OK;
}

bsg_status launched(hipError_t e, const char* what) {
  if (e == hipSuccess) return BSG_OK;
  set_error("%s: launch failed: %s", what, hipGetErrorString(e));
  return BSG_ERR_HIP;
}

int log_level() {
  const char* log = getenv("BSG_LOG");
  return log ? atoi(log) : 0;
}

int64_t padded(int64_t tokens) { return (tokens + 3) / 4 * 4; }

}  // namespace

extern "C" {

bsg_status bsg_f8_quantize(int32_t dtype, int64_t rows, int64_t cols, const void* x, int64_t x_stride, void* codes,
                           int64_t codes_stride, float* scales, int64_t scale_stride, void* stream) {
  bsg_status st = check_common(dtype, 0, 0, "cols", cols, "cols", cols, 1);
  if (st == BSG_OK) st = check_tokens(rows, BSG_F8_MAX_TOKENS);
  if (st != BSG_OK || rows == 0) return st;
  if ((st = check_rows("x", x, x_stride, cols)) != BSG_OK) return st;
  if ((st = check_codes("the result", codes, codes_stride, scales, scale_stride, rows, cols, false)) != BSG_OK) return st;
  return launched(bsg::f8_quantize_launch(dtype == BSG_OUT_F16 ? bsg::Src::F16 : bsg::Src::BF16, rows, cols, x, x_stride, codes,
                                          codes_stride, scales, scale_stride, (hipStream_t)stream),
                  "bsg_f8_quantize");
}

bsg_status bsg_f8_plan_create(const bsg_f8_problem* problem, bsg_f8_plan* out_plan) {
  if (!problem || !out_plan) {
    set_error("null problem or out_plan");
    return BSG_ERR_NULL;
  }
  *out_plan = nullptr;
  if (problem->struct_size != sizeof(bsg_f8_problem)) {
    set_error("bsg_f8_problem.struct_size is %u, expected %zu", problem->struct_size, sizeof(bsg_f8_problem));
    return BSG_ERR_ABI;
  }
  bsg_status st = check_common(problem->dtype, problem->flags, BSG_F8_BIAS | BSG_F8_EXACT, "n", problem->n, "k", problem->k, problem->max_tokens);
  if (st != BSG_OK) return st;
  int dev = -1, cus = 0;
  if ((st = bsg::resolve_device(problem->device, &dev, &cus)) != BSG_OK) return st;
  bsg_f8_plan_s* plan = new (std::nothrow) bsg_f8_plan_s();
  if (!plan) {
    set_error("out of host memory");
    return BSG_ERR_ALLOC;
  }
  plan->magic = kF8Magic;
  plan->problem = *problem;
  plan->problem.device = plan->device = dev;
  plan->cus = cus;
  plan->dtype = problem->dtype == BSG_OUT_F16;
  plan->log_level = log_level();
  const bsg::F8Parts parts = bsg::f8_parts(false, problem->flags & BSG_F8_EXACT, problem->max_tokens, problem->n, problem->k, cus);
  const uint64_t part = 4 * (uint64_t)parts.floats, counters = 4 * (uint64_t)parts.counters;
  plan->workspace_bytes = part + counters;
  if (plan->workspace_bytes) {
    st = bsg::device_alloc(dev, plan->workspace_bytes, &plan->workspace);
    if (st == BSG_OK) {
      plan->part = (float*)plan->workspace;
      plan->arrived = (int*)((uint8_t*)plan->workspace + part);
      st = bsg::device_clear(dev, plan->arrived, counters);
      if (st != BSG_OK) bsg::device_free(dev, plan->workspace);
    }
    if (st != BSG_OK) {
      delete plan;
      return st;
    }
  }
  if (plan->log_level >= 1)
    fprintf(stderr, "bsg: f8 plan n=%lld k=%lld workspace %llu B on device %d\n", (long long)problem->n, (long long)problem->k,
            (unsigned long long)plan->workspace_bytes, dev);
  *out_plan = plan;
  return BSG_OK;
}

bsg_status bsg_f8_plan_destroy(bsg_f8_plan plan) {
  if (!plan) return BSG_OK;
  if (plan->magic != kF8Magic) {
    set_error("invalid plan");
    return BSG_ERR_NULL;
  }
  plan->magic = 0;
  bsg::device_free(plan->device, plan->workspace);  // hipFree waits for work still using it
  delete plan;
  return BSG_OK;
}

bsg_status bsg_f8_plan_workspace(bsg_f8_plan plan, uint64_t* bytes) {
  if (!plan || plan->magic != kF8Magic || !bytes) {
    set_error("invalid plan or null bytes");
    return BSG_ERR_NULL;
  }
  *bytes = plan->workspace_bytes;
  return BSG_OK;
}

bsg_status bsg_f8_run(bsg_f8_plan plan, int64_t tokens, const bsg_f8_rows* x, const void* w, const float* sw,
                      const float* bias, void* out, int64_t out_stride, void* stream) {
  if (!plan || plan->magic != kF8Magic) {
    set_error("invalid plan");
    return BSG_ERR_NULL;
  }
  const bsg_f8_problem& p = plan->problem;
  bsg_status st = check_tokens(tokens, p.max_tokens);
  if (st != BSG_OK || tokens == 0) return st;
  const bool with_bias = p.flags & BSG_F8_BIAS;
  if (!x || !w || !sw || (with_bias && !bias)) {
    set_error("null operand (x=%p w=%p sw=%p bias=%p)", (const void*)x, w, (const void*)sw, (const void*)bias);
    return BSG_ERR_NULL;
  }
  if ((st = check_codes("x", x->codes, x->stride, x->scales, x->scale_stride, tokens, p.k, true)) != BSG_OK) return st;
  if ((st = check_rows("out", out, out_stride, p.n)) != BSG_OK) return st;
  if (((uintptr_t)w & 15u) || (((uintptr_t)sw | (with_bias ? (uintptr_t)bias : 0)) & 3u)) {
    set_error("w must be 16-byte aligned, sw and bias 4-byte aligned");
    return BSG_ERR_ALIGN;
  }
  bsg::F8Args a = {};
  a.tokens = (int)tokens;
  a.n = (int)p.n;
  a.k = (int)p.k;
  a.kb = bsg::f8_blocks(p.k);
  a.x = (const uint8_t*)x->codes;
  a.sx = x->scales;
  a.x_stride = x->stride;
  a.sx_stride = x->scale_stride;
  a.w = (const uint8_t*)w;
  a.sw = sw;
  a.bias = with_bias ? bias : nullptr;
  a.out = (uint8_t*)out;
  a.out_stride = out_stride;
  a.part = plan->part;
  a.arrived = plan->arrived;
  a.exact = (p.flags & BSG_F8_EXACT) != 0;
  if (plan->log_level >= 2) fprintf(stderr, "bsg: f8 run tokens=%lld stream=%p\n", (long long)tokens, stream);
  const hipStream_t s = (hipStream_t)stream;
  return launched(tokens <= bsg::kF8OneTile ? bsg::f8_few_launch(a, bsg::Src::CODES, false, plan->dtype, s)
                                            : bsg::f8_tiled_launch(a, false, plan->dtype, plan->cus, s),
                  "bsg_f8_run");
}

bsg_status bsg_f8_ffn_plan_create(const bsg_f8_ffn_problem* problem, bsg_f8_ffn_plan* out_plan) {
  if (!problem || !out_plan) {
    set_error("null problem or out_plan");
    return BSG_ERR_NULL;
  }
  *out_plan = nullptr;
  if (problem->struct_size != sizeof(bsg_f8_ffn_problem)) {
    set_error("bsg_f8_ffn_problem.struct_size is %u, expected %zu", problem->struct_size, sizeof(bsg_f8_ffn_problem));
    return BSG_ERR_ABI;
  }
  bsg_status st = check_common(problem->dtype, problem->flags, BSG_F8_EXACT, "hidden", problem->hidden, "inter", problem->inter,
                               problem->max_tokens);
  if (st != BSG_OK) return st;
  int dev = -1, cus = 0;
  if ((st = bsg::resolve_device(problem->device, &dev, &cus)) != BSG_OK) return st;
  bsg_f8_ffn_plan_s* plan = new (std::nothrow) bsg_f8_ffn_plan_s();
  if (!plan) {
    set_error("out of host memory");
    return BSG_ERR_ALLOC;
  }
  plan->magic = kFfnMagic;
  plan->problem = *problem;
  plan->problem.device = plan->device = dev;
  plan->cus = cus;
  plan->dtype = problem->dtype == BSG_OUT_F16;
  plan->log_level = log_level();
  const int64_t t = problem->max_tokens, few = t < bsg::kF8OneTile ? t : bsg::kF8OneTile;
  const bool exact = problem->flags & BSG_F8_EXACT;
  const bsg::F8Parts up = bsg::f8_parts(true, exact, t, problem->inter, problem->hidden, cus);
  const bsg::F8Parts down = bsg::f8_parts(false, exact, t, problem->hidden, problem->inter, cus);
  const uint64_t part_bytes = 4 * (uint64_t)(up.floats > down.floats ? up.floats : down.floats);
  const uint64_t counter_bytes = 4 * (uint64_t)(up.counters > down.counters ? up.counters : down.counters);
  uint64_t at = 0;
  auto take = [&](uint64_t bytes) {
    const uint64_t here = at;
    at += (bytes + 255) / 256 * 256;
    return here;
  };
  const uint64_t x_codes = take(t * problem->hidden), h_codes = take(t * problem->inter);
  const uint64_t x_scales = take(4 * padded(t) * bsg::f8_blocks(problem->hidden));
  const uint64_t h_scales = take(4 * padded(t) * bsg::f8_blocks(problem->inter)), h = take(4 * few * problem->inter);
  const uint64_t part = take(part_bytes), arrived = take(counter_bytes);
  plan->workspace_bytes = at;
  if ((st = bsg::device_alloc(dev, at, &plan->workspace)) != BSG_OK) {
    delete plan;
    return st;
  }
  uint8_t* base = (uint8_t*)plan->workspace;
  plan->x_codes = base + x_codes;
  plan->h_codes = base + h_codes;
  plan->x_scales = (float*)(base + x_scales);
  plan->h_scales = (float*)(base + h_scales);
  plan->h = (float*)(base + h);
  plan->part = (float*)(base + part);
  plan->arrived = (int*)(base + arrived);
  if (counter_bytes && (st = bsg::device_clear(dev, plan->arrived, counter_bytes)) != BSG_OK) {
    bsg::device_free(dev, plan->workspace);
    delete plan;
    return st;
  }
  if (plan->log_level >= 1)
    fprintf(stderr, "bsg: f8 ffn plan hidden=%lld inter=%lld workspace %llu B on device %d\n", (long long)problem->hidden,
            (long long)problem->inter, (unsigned long long)at, dev);
  *out_plan = plan;
  return BSG_OK;
}

bsg_status bsg_f8_ffn_plan_destroy(bsg_f8_ffn_plan plan) {
  if (!plan) return BSG_OK;
  if (plan->magic != kFfnMagic) {
    set_error("invalid plan");
    return BSG_ERR_NULL;
  }
  plan->magic = 0;
  bsg::device_free(plan->device, plan->workspace);  // hipFree waits for work still using it
  delete plan;
  return BSG_OK;
}

bsg_status bsg_f8_ffn_plan_workspace(bsg_f8_ffn_plan plan, uint64_t* bytes) {
  if (!plan || plan->magic != kFfnMagic || !bytes) {
    set_error("invalid plan or null bytes");
    return BSG_ERR_NULL;
  }
  *bytes = plan->workspace_bytes;
  return BSG_OK;
}

bsg_status bsg_f8_ffn_run(bsg_f8_ffn_plan plan, int64_t tokens, const void* x, int64_t x_stride,
                          const bsg_f8_ffn_weights* w, void* out, int64_t out_stride, void* stream) {
  if (!plan || plan->magic != kFfnMagic) {
    set_error("invalid plan");
    return BSG_ERR_NULL;
  }
  const bsg_f8_ffn_problem& p = plan->problem;
  bsg_status st = check_tokens(tokens, p.max_tokens);
  if (st != BSG_OK || tokens == 0) return st;
  if (!w) {
    set_error("null weights");
    return BSG_ERR_NULL;
  }
  if (w->struct_size != sizeof(bsg_f8_ffn_weights) || w->reserved != 0) {
    set_error("bsg_f8_ffn_weights.struct_size is %u, expected %zu (reserved 0)", w->struct_size, sizeof(bsg_f8_ffn_weights));
    return BSG_ERR_ABI;
  }
  if (!w->w13 || !w->s13 || !w->w2 || !w->s2) {
    set_error("null weights (w13=%p s13=%p w2=%p s2=%p)", w->w13, (const void*)w->s13, w->w2, (const void*)w->s2);
    return BSG_ERR_NULL;
  }
  if ((((uintptr_t)w->w13 | (uintptr_t)w->w2) & 15u) || (((uintptr_t)w->s13 | (uintptr_t)w->s2) & 3u)) {
    set_error("w13 and w2 must be 16-byte aligned, s13 and s2 4-byte aligned");
    return BSG_ERR_ALIGN;
  }
  if ((st = check_rows("x", x, x_stride, p.hidden)) != BSG_OK) return st;
  if ((st = check_rows("out", out, out_stride, p.hidden)) != BSG_OK) return st;
  if (plan->log_level >= 2) fprintf(stderr, "bsg: f8 ffn run tokens=%lld stream=%p\n", (long long)tokens, stream);
  const hipStream_t s = (hipStream_t)stream;
  const bsg::Src src = plan->dtype ? bsg::Src::F16 : bsg::Src::BF16;
  const int64_t pad = padded(tokens);
  bsg::F8Args a = {};  // gate and up
  a.tokens = (int)tokens;
  a.n = (int)p.inter;
  a.k = (int)p.hidden;
  a.kb = bsg::f8_blocks(p.hidden);
  a.x = plan->x_codes;
  a.x_stride = p.hidden;
  a.sx = plan->x_scales;
  a.sx_stride = pad;
  a.w = (const uint8_t*)w->w13;
  a.sw = w->s13;
  a.out_stride = p.inter;
  a.so_stride = pad;
  bsg::F8Args b = {};  // down
  b.tokens = (int)tokens;
  b.n = (int)p.hidden;
  b.k = (int)p.inter;
  b.kb = bsg::f8_blocks(p.inter);
  b.x = plan->h_codes;
  b.x_stride = p.inter;
  b.sx = plan->h_scales;
  b.sx_stride = pad;
  b.w = (const uint8_t*)w->w2;
  b.sw = w->s2;
  b.out = (uint8_t*)out;
  b.out_stride = out_stride;
  a.part = b.part = plan->part;
  a.arrived = b.arrived = plan->arrived;
  a.exact = b.exact = (p.flags & BSG_F8_EXACT) != 0;
  hipError_t e = hipSuccess;
  if (tokens <= bsg::kF8OneTile) {  // both products quantise what they read
    a.x = (const uint8_t*)x;
    a.x_stride = 2 * x_stride;
    a.out = (uint8_t*)plan->h;
    e = bsg::f8_few_launch(a, src, true, plan->dtype, s);
    b.x = (const uint8_t*)plan->h;
    b.x_stride = 4 * p.inter;
    if (e == hipSuccess) e = bsg::f8_few_launch(b, bsg::Src::F32, false, plan->dtype, s);
    return launched(e, "bsg_f8_ffn_run");
  }
  e = bsg::f8_quantize_launch(src, tokens, p.hidden, x, x_stride, plan->x_codes, p.hidden, plan->x_scales, pad, s);
  a.out = plan->h_codes;
  a.so = plan->h_scales;
  if (e == hipSuccess) e = bsg::f8_tiled_launch(a, true, plan->dtype, plan->cus, s);
  if (e == hipSuccess) e = bsg::f8_tiled_launch(b, false, plan->dtype, plan->cus, s);
  return launched(e, "bsg_f8_ffn_run");
}

}  // extern "C"
