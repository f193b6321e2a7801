// C ABI of the mixture-of-experts layer (include/bsg_moe.h): plans, argument checks and launches.
#include <hip/hip_runtime.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <new>

#include "moe.h"
#include "plan.h"

struct bsg_moe_plan_s {
  uint32_t magic;
  bsg_moe_problem problem;
  bsg::MoeArgs args;  // template: shape and workspace; operands patched per call
  int device, format, dtype, log_level;
  void* workspace;
};

namespace {

using bsg::set_error;

constexpr uint32_t kMoeMagic = 0x4253474Du;  // "BSGM"

bsg_status validate(const bsg_moe_problem* p) {
  if (p->struct_size != sizeof(bsg_moe_problem)) {
    set_error("bsg_moe_problem.struct_size is %u, expected %zu", p->struct_size, sizeof(bsg_moe_problem));
    return BSG_ERR_ABI;
  }
  if (p->format != BSG_FMT_MXFP8 && p->format != BSG_FMT_NVFP4) {
    set_error("unknown format %d", p->format);
    return BSG_ERR_ABI;
  }
  if (p->dtype != BSG_OUT_BF16 && p->dtype != BSG_OUT_F16) {
    set_error("unsupported dtype %d (BF16 or F16 only)", p->dtype);
    return BSG_ERR_ABI;
  }
  if ((p->flags & ~(uint32_t)BSG_MOE_KEEP_PROBABILITIES) || p->reserved != 0) {
    set_error("unknown flag bits 0x%x, or reserved not 0", p->flags);
    return BSG_ERR_ABI;
  }
  if (p->experts < 1 || p->top_k < 1 || p->top_k > p->experts || p->hidden < 32 || p->inter < 32 || p->hidden % 32 ||
      p->inter % 32 || p->max_tokens < 1) {
    set_error("experts >= top_k >= 1, hidden and inter positive multiples of 32, max_tokens >= 1 (got %d, %d, %lld, "
              "%lld, %lld)", p->experts, p->top_k, (long long)p->hidden, (long long)p->inter, (long long)p->max_tokens);
    return BSG_ERR_SHAPE;
  }
  if (p->experts > BSG_MOE_MAX_EXPERTS || p->top_k > BSG_MOE_MAX_TOP_K || p->max_tokens > BSG_MOE_MAX_TOKENS ||
      p->hidden > 65536 || p->inter > 65536) {
    set_error("at most %d experts, top_k %d, %d tokens, hidden and inter 65536 (got %d, %d, %lld, %lld, %lld)",
              BSG_MOE_MAX_EXPERTS, BSG_MOE_MAX_TOP_K, BSG_MOE_MAX_TOKENS, p->experts, p->top_k,
              (long long)p->max_tokens, (long long)p->hidden, (long long)p->inter);
    return BSG_ERR_UNSUPPORTED;
  }
  return BSG_OK;
}

}  // namespace

extern "C" {

bsg_status bsg_moe_plan_create(const bsg_moe_problem* problem, bsg_moe_plan* out_plan) {
  if (!problem || !out_plan) {
    set_error("null problem or out_plan");
    return BSG_ERR_NULL;
  }
  *out_plan = nullptr;
  bsg_status st = validate(problem);
  if (st != BSG_OK) return st;
  int dev = -1, cus = 0;
  st = bsg::resolve_device(problem->device, &dev, &cus);
  if (st != BSG_OK) return st;
  bsg_moe_plan_s* plan = new (std::nothrow) bsg_moe_plan_s();
  if (!plan) {
    set_error("out of host memory");
    return BSG_ERR_ALLOC;
  }
  plan->magic = kMoeMagic;
  plan->problem = *problem;
  plan->problem.device = plan->device = dev;
  plan->format = problem->format == BSG_FMT_NVFP4;
  plan->dtype = problem->dtype == BSG_OUT_F16;
  bsg::MoeArgs& a = plan->args;
  a.experts = problem->experts;
  a.top_k = problem->top_k;
  a.hidden = (int)problem->hidden;
  a.inter = (int)problem->inter;
  a.keep = (problem->flags & BSG_MOE_KEEP_PROBABILITIES) ? 1 : 0;
  size_t counters_at = 0, counters = 0;
  const size_t bytes = bsg::moe_workspace(*problem, nullptr, &a, &counters_at, &counters);
  st = bsg::device_alloc(dev, bytes, &plan->workspace);
  if (st == BSG_OK) {
    bsg::moe_workspace(*problem, (uint8_t*)plan->workspace, &a, &counters_at, &counters);
    st = bsg::device_clear(dev, (uint8_t*)plan->workspace + counters_at, counters);
    if (st != BSG_OK) bsg::device_free(dev, plan->workspace);
  }
  if (st != BSG_OK) {
    delete plan;
    return st;
  }
  const char* log = getenv("BSG_LOG");
  plan->log_level = log ? atoi(log) : 0;
  if (plan->log_level >= 1)
    fprintf(stderr, "bsg: moe plan %s experts=%d top_k=%d hidden=%d inter=%d workspace %zu B on device %d\n",
            plan->format ? "nvfp4" : "mxfp8", a.experts, a.top_k, a.hidden, a.inter, bytes, dev);
  *out_plan = plan;
  return BSG_OK;
}

bsg_status bsg_moe_plan_destroy(bsg_moe_plan plan) {
  if (!plan) return BSG_OK;
  if (plan->magic != kMoeMagic) {
    set_error("invalid plan");
    return BSG_ERR_NULL;
  }
  plan->magic = 0;
  bsg::device_free(plan->device, plan->workspace);  // hipFree waits for work still using it
  delete plan;
  return BSG_OK;
}

bsg_status bsg_moe_run(bsg_moe_plan plan, int64_t tokens, const void* x, int64_t x_stride,
                       const bsg_moe_weights* w, void* out, int64_t out_stride, int32_t* ids, float* route_weights,
                       void* stream) {
  if (!plan || plan->magic != kMoeMagic) {
    set_error("invalid plan");
    return BSG_ERR_NULL;
  }
  if (tokens < 0 || tokens > plan->problem.max_tokens) {
    set_error("tokens must be in [0, max_tokens = %lld] (got %lld)", (long long)plan->problem.max_tokens,
              (long long)tokens);
    return BSG_ERR_SHAPE;
  }
  if (tokens == 0) return BSG_OK;
  if (!w) {
    set_error("null weights");
    return BSG_ERR_NULL;
  }
  if (w->struct_size != sizeof(bsg_moe_weights) || w->reserved != 0) {
    set_error("bsg_moe_weights.struct_size is %u, expected %zu (reserved 0)", w->struct_size, sizeof(bsg_moe_weights));
    return BSG_ERR_ABI;
  }
  if (!x || !out || !w->router || !w->w13 || !w->s13 || !w->w2 || !w->s2) {
    set_error("null operand pointer (x=%p out=%p router=%p w13=%p s13=%p w2=%p s2=%p)", x, out, w->router, w->w13, w->s13,
              w->w2, w->s2);
    return BSG_ERR_NULL;
  }
  if ((((uintptr_t)x | (uintptr_t)out | (uintptr_t)w->router | (uintptr_t)w->w13 | (uintptr_t)w->w2) & 15u) ||
      (((uintptr_t)w->s13 | (uintptr_t)w->s2 | (uintptr_t)w->alpha13 | (uintptr_t)w->alpha2 | (uintptr_t)ids |
        (uintptr_t)route_weights) & 3u)) {
    set_error("x, out, router, w13 and w2 must be 16-byte aligned; s13, s2, alphas, ids and weights 4-byte aligned");
    return BSG_ERR_ALIGN;
  }
  if ((x_stride | out_stride) & 7) {
    set_error("x_stride and out_stride must be multiples of 8 elements (got %lld, %lld)", (long long)x_stride,
              (long long)out_stride);
    return BSG_ERR_ALIGN;
  }
  const int64_t lim = (int64_t)1 << 31;
  if (x_stride < plan->problem.hidden || out_stride < plan->problem.hidden || x_stride >= lim || out_stride >= lim) {
    set_error("x_stride and out_stride must be in [hidden, 2^31) (got %lld, %lld)", (long long)x_stride,
              (long long)out_stride);
    return BSG_ERR_SHAPE;
  }
  bsg::MoeArgs a = plan->args;
  a.tokens = (int)tokens;
  a.x = (const uint16_t*)x;
  a.router = (const uint16_t*)w->router;
  a.w13 = (const uint8_t*)w->w13;
  a.s13 = (const uint8_t*)w->s13;
  a.w2 = (const uint8_t*)w->w2;
  a.s2 = (const uint8_t*)w->s2;
  a.alpha13 = w->alpha13;
  a.alpha2 = w->alpha2;
  a.out = (uint16_t*)out;
  a.ids = ids;
  a.weights = route_weights;
  a.x_stride = x_stride;
  a.out_stride = out_stride;
  if (plan->log_level >= 2)
    fprintf(stderr, "bsg: moe run tokens=%lld x=%p out=%p stream=%p\n", (long long)tokens, x, out, stream);
  const hipError_t e = bsg::moe_launch(a, plan->format, plan->dtype, (hipStream_t)stream);
  if (e != hipSuccess) {
    set_error("bsg_moe_run: launch failed: %s", hipGetErrorString(e));
    return BSG_ERR_HIP;
  }
  return BSG_OK;
}

}  // extern "C"
