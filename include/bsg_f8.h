/*
 * bsg_f8.h -- products in 8-bit floating point with a scale for each block of 128, and the gated
 * feed-forward block over them, on AMD MI355X (gfx950), C ABI.
 *
 * Elements are E4M3 codes (OCP 8-bit, as in bsg.h; 0x7F and 0xFF are NaN).  B(k) = ceil(k / 128) is the number
 * of blocks along k.  Two kinds of scales, both fp32:
 *   rows      one for each 128 consecutive elements of a row, block by block: the scale of row t, block b is
 *             scales[b * scale_stride + t], so that the scales which a product needs at a time are neighbours;
 *   weights   one for each 128 x 128 block, [B(n)][B(k)], row-major.
 * The last block of a row, and of the weights' rows, may be shorter.
 * Scales may have any values whose product, a row's scale times a weight's, is below 2^128: it is formed in fp32 and then
 * multiplied by the block's sum of codes.  Where it is larger it is infinite, also for a block whose sum is zero (NaN then).
 * Where it is below 2^-126 it is rounded to a multiple of 2^-149, which moves a block's part of an output by at most 2^-125.
 *
 * bsg_f8_quantize   codes and scales of 16-bit rows: of the elements x of a block, the scale is the least power of
 *                   two s >= 2^-126 with max|x| <= 448 s, and the codes are x / s rounded to nearest even (x / s is
 *                   exact, so no rounding comes before that one; scales that are powers of two lose no digits of
 *                   floating-point codes, and only elements below 2^-13 of a block's largest may have fewer than 4).  A
 *                   block with an infinity or a NaN becomes NaN.
 * bsg_f8_run        out[t][j] = sum_b sx[b][t] sw[j / 128][b] (sum of x[t][i] w[j][i] over i in block b) + bias[j]
 * bsg_f8_ffn_run    xq = quantize(x);  gate, up = xq w13^T;  hq = quantize(SiLU(gate) up);  out = hq w2^T
 *                   with quantize as above, the outer values in 16 bits and the inner ones in fp32 until they are codes.
 * Sums are fp32 and outputs are rounded once.  Products of up to 16 tokens, gate and up of up to 64, and all products of
 * plans with BSG_F8_EXACT are exact before they are summed.  The others are of matrix instructions that align the products of
 * every 8 elements to the largest and drop what lies 2^-13 below it.  That moves an output by at most 2^-10 of the sum of the
 * products' magnitudes; measured, 2e-6 of it for normally distributed elements (root mean square; 1.4e-5 of a sum of 128 of random
 * signs) and up to 2e-4 for codes of all sizes.  Sums that cancel keep the error of their magnitudes.  In bsg_f8_ffn_run of more
 * than 64 tokens it moves one inner value in 400 to a neighbouring code: outputs are off by 0.15% of their root mean square
 * (bsg_f8_ffn_run of 4095 tokens, fp16 outputs; 0.02% with BSG_F8_EXACT).  BSG_F8_EXACT takes 1.1 to 1.4 times as long for up
 * to some hundred tokens and 2.7 times for thousands.
 *
 * Conventions are those of bsg.h: a plan made once, O(1) host work per call on the caller's stream, no
 * allocation or synchronisation in a call (so calls can be captured into a HIP graph), bsg_status results and
 * bsg_last_error().  All pointers are device pointers, and no output may overlap an input.
 */
#ifndef BSG_F8_H
#define BSG_F8_H

#include "bsg.h"

#ifdef __cplusplus
extern "C" {
#endif

#define BSG_F8_BLOCK 128
#define BSG_F8_MAX_SIZE 262144     /* of n, k, hidden and inter */
#define BSG_F8_MAX_TOKENS 16777216

enum {
  BSG_F8_BIAS = 1u << 0, /* add bias[n] (not in bsg_f8_ffn_problem) */
  BSG_F8_EXACT = 1u << 2 /* products are exact before they are summed, however many tokens */
};

typedef struct bsg_f8_problem {
  uint32_t struct_size; /* = sizeof(bsg_f8_problem) */
  int32_t dtype;        /* bsg_out_dtype of out */
  uint32_t flags;       /* BSG_F8_* */
  int32_t device;       /* HIP device ordinal; -1 = the current device at create time */
  int64_t n, k;         /* outputs and inputs of a token: multiples of 16, up to BSG_F8_MAX_SIZE */
  int64_t max_tokens;   /* the most tokens of a call, 1 .. BSG_F8_MAX_TOKENS */
} bsg_f8_problem;

typedef struct bsg_f8_rows { /* quantised rows [tokens][k] */
  const void* codes;         /* 16-byte aligned */
  const float* scales;       /* 16-byte aligned, [B(k)][scale_stride] */
  int64_t stride;            /* bytes from row to row: a multiple of 16, at least k, below 2^22 */
  int64_t scale_stride;      /* a multiple of 4, at least the number of rows, below 2^25 */
} bsg_f8_rows;

typedef struct bsg_f8_plan_s* bsg_f8_plan; /* opaque, library-owned */

/* Codes and scales of x [rows][cols], 16-bit of `dtype` (bsg_out_dtype), rows x_stride elements apart (a multiple of
 * 8).  cols: a multiple of 16 up to BSG_F8_MAX_SIZE; codes rows codes_stride bytes apart, scales as bsg_f8_rows has
 * them; entries of scales from rows on are left as they were.  x and codes 16-byte, scales 4-byte aligned.  rows 0 does
 * nothing.  Needs no plan; runs on the current device.
 * Errors: BSG_ERR_NULL, _ABI (dtype), _SHAPE, _ALIGN, _HIP. */
bsg_status bsg_f8_quantize(int32_t dtype, int64_t rows, int64_t cols, const void* x, int64_t x_stride, void* codes,
                           int64_t codes_stride, float* scales, int64_t scale_stride, void* stream);

/* Validate and make a plan.  Calls on one plan must be ordered (one stream, or events) where workspace_bytes is not 0:
 * they share the workspace.  Errors: BSG_ERR_NULL, _ABI, _SHAPE, _DEVICE, _HIP, _ALLOC. */
bsg_status bsg_f8_plan_create(const bsg_f8_problem* problem, bsg_f8_plan* out_plan);
bsg_status bsg_f8_plan_destroy(bsg_f8_plan plan); /* NULL is accepted */
bsg_status bsg_f8_plan_workspace(bsg_f8_plan plan, uint64_t* bytes);

/* One product.  w: [n][k] codes, 16-byte aligned, sw its scales; bias: float [n], required iff the plan has BSG_F8_BIAS
 * (ignored otherwise); out: rows of n 16-bit values, out_stride elements apart (a multiple of 8, at least n, below 2^22),
 * 16-byte aligned.  tokens 0 does nothing.  Errors: BSG_ERR_NULL, _SHAPE, _ALIGN, _HIP. */
bsg_status bsg_f8_run(bsg_f8_plan plan, int64_t tokens, const bsg_f8_rows* x, const void* w, const float* sw,
                      const float* bias, void* out, int64_t out_stride, void* stream);

typedef struct bsg_f8_ffn_problem {
  uint32_t struct_size;  /* = sizeof(bsg_f8_ffn_problem) */
  int32_t dtype;         /* bsg_out_dtype of x and out */
  uint32_t flags;        /* 0 or BSG_F8_EXACT */
  int32_t device;        /* HIP device ordinal; -1 = the current device at create time */
  int64_t hidden, inter; /* multiples of 16, up to BSG_F8_MAX_SIZE */
  int64_t max_tokens;    /* the most tokens of a call, 1 .. BSG_F8_MAX_TOKENS */
} bsg_f8_ffn_problem;

typedef struct bsg_f8_ffn_weights { /* codes 16-byte, scales 4-byte aligned */
  uint32_t struct_size;             /* = sizeof(bsg_f8_ffn_weights) */
  uint32_t reserved;                /* 0 */
  const void* w13;                  /* [2 inter][hidden]: gate's rows, then up's */
  const float* s13;                 /* [2][B(inter)][B(hidden)]: gate's blocks, then up's */
  const void* w2;                   /* [hidden][inter] */
  const float* s2;                  /* [B(hidden)][B(inter)] */
} bsg_f8_ffn_weights;

typedef struct bsg_f8_ffn_plan_s* bsg_f8_ffn_plan; /* opaque, library-owned */

/* Validate and make a plan with its device workspace (x and SiLU(gate) up between the kernels).  Calls on one plan must be
 * ordered: they share the workspace.  One plan serves every layer of the same shape.
 * Errors: BSG_ERR_NULL, _ABI, _SHAPE, _DEVICE, _HIP, _ALLOC. */
bsg_status bsg_f8_ffn_plan_create(const bsg_f8_ffn_problem* problem, bsg_f8_ffn_plan* out_plan);
bsg_status bsg_f8_ffn_plan_destroy(bsg_f8_ffn_plan plan); /* NULL is accepted */
bsg_status bsg_f8_ffn_plan_workspace(bsg_f8_ffn_plan plan, uint64_t* bytes);

/* One block.  x, out: [tokens][hidden], rows x_stride and out_stride elements apart (multiples of 8, at least hidden,
 * below 2^22), 16-byte aligned.  tokens 0 does nothing.  Errors: BSG_ERR_NULL, _ABI, _SHAPE, _ALIGN, _HIP. */
bsg_status bsg_f8_ffn_run(bsg_f8_ffn_plan plan, int64_t tokens, const void* x, int64_t x_stride,
                          const bsg_f8_ffn_weights* weights, void* out, int64_t out_stride, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BSG_F8_H */
