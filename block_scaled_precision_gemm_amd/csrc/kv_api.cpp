// C ABI of the paged NVFP4 cache (include/bsg_kv.h): plans, argument checks and launches.
#include <hip/hip_runtime.h>
#include <math.h>
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include <new>

#include "kv.h"
#include "kv_split.h"
#include "plan.h"

struct bsg_kv_plan_s {
  uint32_t magic;
  bsg_kv_problem problem;
  bsg::KvArgs args;  // template: the plan's part; batch and operands patched per call
  int device, cus, dtype, log_level;
  void* workspace;
  uint64_t workspace_bytes;
};

namespace {

using bsg::set_error;

constexpr uint32_t kKvMagic = 0x4253474Bu;  // "BSGK"

bool geometry_ok(int kv_heads, int head_dim, int page_tokens) {
  return kv_heads >= 1 && kv_heads <= 1024 && (head_dim == 64 || head_dim == 128) && page_tokens >= 16 &&
         page_tokens <= 256 && (page_tokens & (page_tokens - 1)) == 0;
}

bool usable_scale(float s) { return isfinite(s) && s >= 0.0f && (s == 0.0f || isfinite(1.0f / s)); }

bsg_status validate(const bsg_kv_problem* p) {
  if (p->struct_size != sizeof(bsg_kv_problem)) {
    set_error("bsg_kv_problem.struct_size is %u, expected %zu", p->struct_size, sizeof(bsg_kv_problem));
    return BSG_ERR_ABI;
  }
  if (p->dtype != BSG_OUT_BF16 && p->dtype != BSG_OUT_F16) {
    set_error("unsupported dtype %d (BF16 or F16 only)", p->dtype);
    return BSG_ERR_ABI;
  }
  if (p->flags & ~(uint32_t)(BSG_KV_ROPE_INTERLEAVED | BSG_KV_NONCAUSAL)) {
    set_error("unknown flag bits 0x%x", p->flags);
    return BSG_ERR_ABI;
  }
  if (p->kv_heads < 1 || p->kv_heads > 1024 || p->q_heads < p->kv_heads || p->q_heads % p->kv_heads ||
      p->q_heads > 65535 - 2048) {
    set_error("q_heads must be a multiple of kv_heads, kv_heads in [1, 1024], q_heads < 63488 (got %d, %d)", p->q_heads,
              p->kv_heads);
    return BSG_ERR_SHAPE;
  }
  if (!geometry_ok(p->kv_heads, p->head_dim, p->page_tokens)) {
    set_error("head_dim must be 64 or 128 and page_tokens a power of two in [16, 256] (got %d, %d)", p->head_dim,
              p->page_tokens);
    return p->head_dim >= 1 && p->page_tokens >= 1 ? BSG_ERR_UNSUPPORTED : BSG_ERR_SHAPE;
  }
  if (p->num_pages < 1 || p->num_pages > 0x7FFFFFFF || p->max_tokens < 1 || p->max_tokens > (1 << 24) ||
      p->max_tokens * p->q_heads > ((int64_t)1 << 30)) {
    set_error("num_pages must be in [1, 2^31 - 1] and max_tokens in [1, 2^24] with max_tokens * q_heads <= 2^30 (got "
              "%lld, %lld)", (long long)p->num_pages, (long long)p->max_tokens);
    return BSG_ERR_SHAPE;
  }
  const int64_t packed = bsg_kv_page_bytes(p->kv_heads, p->head_dim, p->page_tokens);
  if (p->page_stride != 0 && (p->page_stride < packed || p->page_stride > ((int64_t)1 << 40))) {
    set_error("page_stride must be 0 or in [%lld, 2^40] (got %lld)", (long long)packed, (long long)p->page_stride);
    return BSG_ERR_SHAPE;
  }
  if (p->page_stride & 15) {
    set_error("page_stride must be a multiple of 16 (got %lld)", (long long)p->page_stride);
    return BSG_ERR_ALIGN;
  }
  if (p->rope_dim < 0 || p->rope_dim > p->head_dim || p->rope_dim % 16) {
    set_error("rope_dim must be a multiple of 16 in [0, head_dim] (got %d)", p->rope_dim);
    return BSG_ERR_SHAPE;
  }
  if (p->window < 0) {
    set_error("window must be >= 0 (got %d)", p->window);
    return BSG_ERR_SHAPE;
  }
  if (p->window > 0 && (p->flags & BSG_KV_NONCAUSAL)) {
    set_error("a window needs causal attention");
    return BSG_ERR_UNSUPPORTED;
  }
  if (!isfinite(p->scale) || !usable_scale(p->softcap) || !usable_scale(p->k_scale) || !usable_scale(p->v_scale)) {
    set_error("scale must be finite; softcap, k_scale and v_scale 0 or positive with a finite reciprocal (got %g, %g, "
              "%g, %g)", (double)p->scale, (double)p->softcap, (double)p->k_scale, (double)p->v_scale);
    return BSG_ERR_SHAPE;
  }
  return BSG_OK;
}

bsg_status check_plan(bsg_kv_plan plan) {
  if (!plan || plan->magic != kKvMagic) {
    set_error("invalid plan");
    return BSG_ERR_NULL;
  }
  return BSG_OK;
}

// Check the batch and copy it into `a`.  *empty: there is nothing to do.
bsg_status take_batch(bsg_kv_plan plan, const bsg_kv_batch* b, bsg::KvArgs* a, bool* empty) {
  if (!b) {
    set_error("null batch");
    return BSG_ERR_NULL;
  }
  if (b->struct_size != sizeof(bsg_kv_batch)) {
    set_error("bsg_kv_batch.struct_size is %u, expected %zu", b->struct_size, sizeof(bsg_kv_batch));
    return BSG_ERR_ABI;
  }
  const bsg_kv_problem& p = plan->problem;
  if (b->num_seqs < 0 || b->num_seqs > p.max_tokens || b->num_tokens < 0 || b->num_tokens > p.max_tokens) {
    set_error("num_seqs and num_tokens must be in [0, max_tokens = %lld] (got %d, %lld)", (long long)p.max_tokens,
              b->num_seqs, (long long)b->num_tokens);
    return BSG_ERR_SHAPE;
  }
  *empty = b->num_tokens == 0;
  if (*empty) return BSG_OK;
  if (b->num_seqs < 1 || b->max_q < 1 || b->max_kv < 1 || b->max_kv > (1 << 30) || b->max_q > b->num_tokens ||
      (int64_t)b->max_q * b->num_seqs < b->num_tokens) {
    set_error("a batch of %lld tokens needs num_seqs >= 1, max_q in [num_tokens / num_seqs, num_tokens] and max_kv in "
              "[1, 2^30] (got %d, %d, %d)", (long long)b->num_tokens, b->num_seqs, b->max_q, b->max_kv);
    return BSG_ERR_SHAPE;
  }
  if (!b->q_start || !b->kv_len || !b->pages) {
    set_error("null batch array");
    return BSG_ERR_NULL;
  }
  if (((uintptr_t)b->q_start | (uintptr_t)b->kv_len | (uintptr_t)b->pages) & 3u) {
    set_error("batch arrays must be 4-byte aligned");
    return BSG_ERR_ALIGN;
  }
  if (b->pages_stride < 1 || b->pages_stride > ((int64_t)1 << 31) || b->pages_stride * p.page_tokens < b->max_kv) {
    set_error("pages_stride * page_tokens must cover max_kv (got %lld * %d < %d)", (long long)b->pages_stride,
              p.page_tokens, b->max_kv);
    return BSG_ERR_SHAPE;
  }
  *a = plan->args;
  a->num_seqs = b->num_seqs;
  a->num_tokens = (int)b->num_tokens;
  a->max_q = b->max_q;
  a->max_kv = b->max_kv;
  a->one_each = b->max_q == 1 && b->num_tokens == b->num_seqs;
  a->q_start = b->q_start;
  a->kv_len = b->kv_len;
  a->pages = b->pages;
  a->pages_stride = b->pages_stride;
  return BSG_OK;
}

bsg_status take_heads(const bsg_heads* t, const char* name, bsg::HeadsArg* out) {
  if (!t || !t->ptr) {
    set_error("null %s", name);
    return BSG_ERR_NULL;
  }
  if ((uintptr_t)t->ptr & 15u) {
    set_error("%s must be 16-byte aligned (got %p)", name, t->ptr);
    return BSG_ERR_ALIGN;
  }
  if (((t->token_stride | t->head_stride) & 7)) {
    set_error("strides of %s must be multiples of 8 elements (got %lld, %lld)", name, (long long)t->token_stride,
              (long long)t->head_stride);
    return BSG_ERR_ALIGN;
  }
  const int64_t lim = (int64_t)1 << 31;
  if (t->token_stride <= -lim || t->token_stride >= lim || t->head_stride <= -lim || t->head_stride >= lim) {
    set_error("strides of %s must be below 2^31 elements", name);
    return BSG_ERR_SHAPE;
  }
  out->ptr = (uint8_t*)t->ptr;
  out->token_stride = t->token_stride;
  out->head_stride = t->head_stride;
  return BSG_OK;
}

bsg_status take_cache(const void* cache, bsg::KvArgs* a) {
  if (!cache) {
    set_error("null cache");
    return BSG_ERR_NULL;
  }
  if ((uintptr_t)cache & 15u) {
    set_error("cache must be 16-byte aligned (got %p)", cache);
    return BSG_ERR_ALIGN;
  }
  a->cache = (uint8_t*)cache;
  return BSG_OK;
}

bsg_status launched(hipError_t e, const char* what) {
  if (e == hipSuccess) return BSG_OK;
  set_error("%s: launch failed: %s", what, hipGetErrorString(e));
  return BSG_ERR_HIP;
}

}  // namespace

extern "C" {

int64_t bsg_kv_page_bytes(int32_t kv_heads, int32_t head_dim, int32_t page_tokens) {
  if (!geometry_ok(kv_heads, head_dim, page_tokens)) return 0;
  return (int64_t)kv_heads * page_tokens * head_dim * 9 / 8;
}

bsg_status bsg_kv_plan_create(const bsg_kv_problem* problem, bsg_kv_plan* out_plan) {
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
  bsg_kv_plan_s* plan = new (std::nothrow) bsg_kv_plan_s();
  if (!plan) {
    set_error("out of host memory");
    return BSG_ERR_ALLOC;
  }
  plan->magic = kKvMagic;
  plan->problem = *problem;
  bsg_kv_problem& p = plan->problem;
  p.device = plan->device = dev;
  plan->cus = cus;
  plan->dtype = p.dtype == BSG_OUT_F16;
  if (p.page_stride == 0) p.page_stride = bsg_kv_page_bytes(p.kv_heads, p.head_dim, p.page_tokens);
  if (p.scale == 0.0f) p.scale = 1.0f / sqrtf((float)p.head_dim);
  if (p.k_scale == 0.0f) p.k_scale = 1.0f;
  if (p.v_scale == 0.0f) p.v_scale = 1.0f;
  bsg::KvArgs& a = plan->args;
  a.q_heads = p.q_heads;
  a.kv_heads = p.kv_heads;
  a.group = p.q_heads / p.kv_heads;
  a.page_shift = __builtin_ctz((unsigned)p.page_tokens);
  a.num_pages = (int)p.num_pages;
  a.rope_half = p.rope_dim / 2;
  a.window = bsg::kept_window(p.window);
  a.flags = (int)p.flags;
  a.page_stride = p.page_stride;
  a.score_mul = p.scale * p.k_scale;
  a.cap = p.softcap * 1.44269504088896341f;
  a.cap_inv = p.softcap > 0.0f ? 1.0f / a.cap : 0.0f;
  a.k_scale = p.k_scale;
  a.v_scale = p.v_scale;
  a.k_inv = 1.0f / p.k_scale;
  a.v_inv = 1.0f / p.v_scale;
  size_t part = 0, counters = 0, groups = 0;
  bsg::kv_workspace(p, cus, &part, &counters, &groups);
  plan->workspace_bytes = (part + counters) * 4;
  st = bsg::device_alloc(dev, plan->workspace_bytes, &plan->workspace);
  if (st == BSG_OK) {
    a.part = (float*)plan->workspace;
    a.group_arrived = (int*)(a.part + part);
    a.arrived = a.group_arrived + groups;
    st = bsg::device_clear(dev, a.group_arrived, counters * 4);
    if (st != BSG_OK) bsg::device_free(dev, plan->workspace);
  }
  if (st != BSG_OK) {
    delete plan;
    return st;
  }
  const char* log = getenv("BSG_LOG");
  plan->log_level = log ? atoi(log) : 0;
  if (plan->log_level >= 1)
    fprintf(stderr, "bsg: kv plan q_heads=%d kv_heads=%d head_dim=%d page_tokens=%d pages=%lld workspace %llu B on device %d\n",
            p.q_heads, p.kv_heads, p.head_dim, p.page_tokens, (long long)p.num_pages,
            (unsigned long long)plan->workspace_bytes, dev);
  *out_plan = plan;
  return BSG_OK;
}

bsg_status bsg_kv_plan_destroy(bsg_kv_plan plan) {
  if (!plan) return BSG_OK;
  bsg_status st = check_plan(plan);
  if (st != BSG_OK) return st;
  plan->magic = 0;
  bsg::device_free(plan->device, plan->workspace);  // hipFree waits for work still using it
  delete plan;
  return BSG_OK;
}

bsg_status bsg_kv_plan_query(bsg_kv_plan plan, bsg_kv_plan_info* info) {
  bsg_status st = check_plan(plan);
  if (st != BSG_OK) return st;
  if (!info) {
    set_error("null info");
    return BSG_ERR_NULL;
  }
  if (info->struct_size != sizeof(bsg_kv_plan_info)) {
    set_error("bsg_kv_plan_info.struct_size is %u, expected %zu", info->struct_size, sizeof(bsg_kv_plan_info));
    return BSG_ERR_ABI;
  }
  const bsg_kv_problem& p = plan->problem;
  info->reserved = 0;
  info->page_bytes = bsg_kv_page_bytes(p.kv_heads, p.head_dim, p.page_tokens);
  info->page_stride = p.page_stride;
  info->workspace_bytes = plan->workspace_bytes;
  return BSG_OK;
}

bsg_status bsg_kv_append(bsg_kv_plan plan, const bsg_kv_batch* batch, const bsg_heads* q, const bsg_heads* k,
                         const bsg_heads* v, const bsg_heads* q_out, const float* rope, int64_t rope_rows,
                         void* cache, void* stream) {
  bsg_status st = check_plan(plan);
  if (st != BSG_OK) return st;
  bsg::KvArgs a;
  bool empty = false;
  st = take_batch(plan, batch, &a, &empty);
  if (st != BSG_OK || empty) return st;
  if (!!q != !!q_out) {
    set_error("q and q_out are given together or not at all");
    return BSG_ERR_NULL;
  }
  if ((st = take_heads(k, "k", &a.k)) != BSG_OK || (st = take_heads(v, "v", &a.v)) != BSG_OK) return st;
  if (q && ((st = take_heads(q, "q", &a.q)) != BSG_OK || (st = take_heads(q_out, "q_out", &a.out)) != BSG_OK)) return st;
  if ((st = take_cache(cache, &a)) != BSG_OK) return st;
  if (plan->problem.rope_dim > 0) {
    if (!rope) {
      set_error("null rope table (rope_dim %d)", plan->problem.rope_dim);
      return BSG_ERR_NULL;
    }
    if ((uintptr_t)rope & 15u) {
      set_error("the rope table must be 16-byte aligned (got %p)", (const void*)rope);
      return BSG_ERR_ALIGN;
    }
    if (rope_rows < batch->max_kv) {
      set_error("the rope table has %lld rows, max_kv is %d", (long long)rope_rows, batch->max_kv);
      return BSG_ERR_SHAPE;
    }
    a.rope = rope;
  }
  if (plan->log_level >= 2)
    fprintf(stderr, "bsg: kv append %d tokens of %d sequences stream=%p\n", a.num_tokens, a.num_seqs, stream);
  return launched(bsg::kv_append_launch(a, plan->dtype, plan->problem.head_dim, q != nullptr, (hipStream_t)stream),
                  "bsg_kv_append");
}

bsg_status bsg_kv_attend(bsg_kv_plan plan, const bsg_kv_batch* batch, const bsg_heads* q, const void* cache,
                         const bsg_heads* out, float* lse, void* stream) {
  bsg_status st = check_plan(plan);
  if (st != BSG_OK) return st;
  bsg::KvArgs a;
  bool empty = false;
  st = take_batch(plan, batch, &a, &empty);
  if (st != BSG_OK || empty) return st;
  if ((st = take_heads(q, "q", &a.q)) != BSG_OK || (st = take_heads(out, "out", &a.out)) != BSG_OK) return st;
  if ((st = take_cache(cache, &a)) != BSG_OK) return st;
  if ((uintptr_t)lse & 3u) {
    set_error("lse must be 4-byte aligned");
    return BSG_ERR_ALIGN;
  }
  a.lse = lse;
  if (!bsg::attend_fits(a.num_tokens, a.num_seqs, a.max_q, a.group, a.kv_heads,
                        bsg::context_positions(a.window, a.max_q, a.max_kv))) {
    set_error("%d tokens of %d sequences over contexts of up to %d positions are too many for one call", a.num_tokens,
              a.num_seqs, a.max_kv);
    return BSG_ERR_UNSUPPORTED;
  }
  if (plan->log_level >= 2)
    fprintf(stderr, "bsg: kv attend %d tokens of %d sequences, contexts up to %d, stream=%p\n", a.num_tokens, a.num_seqs,
            a.max_kv, stream);
  return launched(bsg::kv_attend_launch(a, plan->dtype, plan->problem.head_dim, plan->cus, (hipStream_t)stream),
                  "bsg_kv_attend");
}

bsg_status bsg_kv_read(bsg_kv_plan plan, const bsg_kv_batch* batch, const void* cache, const bsg_heads* k,
                       const bsg_heads* v, void* stream) {
  bsg_status st = check_plan(plan);
  if (st != BSG_OK) return st;
  bsg::KvArgs a;
  bool empty = false;
  st = take_batch(plan, batch, &a, &empty);
  if (st != BSG_OK || empty) return st;
  if ((st = take_heads(k, "k", &a.k)) != BSG_OK || (st = take_heads(v, "v", &a.v)) != BSG_OK) return st;
  if ((st = take_cache(cache, &a)) != BSG_OK) return st;
  if (plan->log_level >= 2)
    fprintf(stderr, "bsg: kv read %d tokens of %d sequences stream=%p\n", a.num_tokens, a.num_seqs, stream);
  return launched(bsg::kv_read_launch(a, plan->dtype, plan->problem.head_dim, (hipStream_t)stream), "bsg_kv_read");
}

}  // extern "C"
