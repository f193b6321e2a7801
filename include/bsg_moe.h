/*
 * bsg_moe.h -- mixture-of-experts layer for few tokens on AMD MI355X (gfx950), C ABI.
 *
 * For up to 64 tokens x (16-bit, [tokens][hidden]):
 *     logits = x router^T                     router 16-bit [experts][hidden]
 *     p = softmax(logits);  the top_k largest (ties: the lowest expert), weights w = their p divided by
 *     their sum (or the p themselves with BSG_MOE_KEEP_PROBABILITIES)
 *     gate, up = alpha13[e] (x w13[e]^T)      rows 0 .. inter-1 of w13[e] are gate's, the next inter up's
 *     y = alpha2[e] ((SiLU(gate) up) w2[e]^T)
 *     out = sum over the chosen experts of w y, in the order of their rank
 * with expert weights in the library's block-scaled operand formats (bsg.h; the B operand, row-major
 * scales): w13 [experts][2 inter][hidden], w2 [experts][hidden][inter], each expert's codes and scales
 * following the previous one's.  Sums are fp32; out is rounded once.  x enters its products as it is, except that
 * beside NVFP4 weights elements of a bf16 token below 2^-24 of its largest magnitude keep fewer than their 8 bits
 * (steps of 2^-31 of that magnitude).  SiLU(gate) up is held in two bf16 parts, 16 significant bits.
 *
 * Conventions are those of bsg.h: a plan made once, O(1) host work per call, no allocation or
 * synchronisation in a call (it can be captured into a HIP graph), bsg_status and bsg_last_error().
 * For more tokens, or a few experts with many tokens each, use the GEMM of bsg.h per expert.
 */
#ifndef BSG_MOE_H
#define BSG_MOE_H

#include "bsg.h"

#ifdef __cplusplus
extern "C" {
#endif

#define BSG_MOE_MAX_TOKENS 64
#define BSG_MOE_MAX_EXPERTS 512
#define BSG_MOE_MAX_TOP_K 16

enum { BSG_MOE_KEEP_PROBABILITIES = 1u << 0 /* weights are the softmax probabilities, not renormalised */ };

typedef struct bsg_moe_problem {
  uint32_t struct_size; /* = sizeof(bsg_moe_problem) */
  int32_t format;       /* bsg_format of w13 and w2 */
  int32_t dtype;        /* bsg_out_dtype of x, router and out */
  uint32_t flags;       /* BSG_MOE_* */
  int32_t experts;      /* 1 .. BSG_MOE_MAX_EXPERTS */
  int32_t top_k;        /* 1 .. min(experts, BSG_MOE_MAX_TOP_K) */
  int64_t hidden, inter; /* multiples of 32, up to 65536 */
  int64_t max_tokens;   /* 1 .. BSG_MOE_MAX_TOKENS */
  int32_t device;       /* HIP device ordinal; -1 = the current device at create time */
  int32_t reserved;     /* 0 */
} bsg_moe_problem;

typedef struct bsg_moe_weights { /* device pointers; codes 16-byte, scales and alphas 4-byte aligned */
  uint32_t struct_size;          /* = sizeof(bsg_moe_weights) */
  uint32_t reserved;             /* 0 */
  const void* router;            /* 16-byte aligned */
  const void *w13, *s13, *w2, *s2;
  const float *alpha13, *alpha2; /* [experts], or NULL for 1 */
} bsg_moe_weights;

typedef struct bsg_moe_plan_s* bsg_moe_plan; /* opaque, library-owned */

/* Validate and make a plan with its device workspace.  Calls on one plan must be ordered (one stream,
 * or events): they share the workspace.  One plan serves every layer of the same shape.
 * Errors: BSG_ERR_NULL, _ABI, _SHAPE, _UNSUPPORTED, _DEVICE, _HIP, _ALLOC. */
bsg_status bsg_moe_plan_create(const bsg_moe_problem* problem, bsg_moe_plan* out_plan);
bsg_status bsg_moe_plan_destroy(bsg_moe_plan plan); /* NULL is accepted */

/* One layer.  x, out: [tokens][hidden], rows x_stride and out_stride elements apart (multiples of 8,
 * at least hidden), 16-byte aligned; out must not overlap x.  ids (int32) and weights (float)
 * [tokens][top_k], each may be NULL: the chosen experts in the order of their rank, and their weights.
 * tokens 0 does nothing.  Errors: BSG_ERR_NULL, _ABI, _SHAPE, _ALIGN, _HIP. */
bsg_status bsg_moe_run(bsg_moe_plan plan, int64_t tokens, const void* x, int64_t x_stride,
                       const bsg_moe_weights* weights, void* out, int64_t out_stride, int32_t* ids,
                       float* route_weights, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BSG_MOE_H */
