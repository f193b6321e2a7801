/*
 * bsg_kv.h -- paged NVFP4 key/value cache and attention for AMD MI355X (gfx950), C ABI.
 *
 * The part of a decode layer between its block-scaled projections (bsg.h): new keys and values are
 * rotated by their positions and stored as NVFP4 blocks in a paged cache, and queries attend to that
 * cache.  Conventions are those of bsg.h: a plan made once, O(1) host work per call on the caller's
 * stream, no allocation or synchronisation in a call (so calls can be captured into a HIP graph),
 * bsg_status results and bsg_last_error().
 *
 * Cache layout.  Page p starts at cache + p * page_stride and holds page_tokens positions of every
 * key/value head.  Head h of a page is one contiguous chunk of page_tokens * head_dim * 9/8 bytes at
 * byte h * that size (P = page_tokens, D = head_dim):
 *     bytes [0, P*D/2)             key codes    [P][D/2]   packed E2M1, element 2t in the low nibble
 *     bytes [P*D/2, P*D)           value codes  [P][D/2]
 *     bytes [P*D, P*D + P*D/16)    key scales   [P][D/16]  E4M3, one per 16 consecutive dims
 *     bytes [P*D + P*D/16, P*D*9/8) value scales [D/16][P] E4M3 (position fastest)
 * Scale codes are non-negative (0x00..0x7E), or 0x7F for a block that reads as NaN.
 *
 * Stored values.  Of 16 consecutive dims x (after rotation, in fp32) with the plan's scale g (k_scale
 * or v_scale): y = x * (1/g), s = E4M3 rounding of min(max|y| * (1/6), 448), q = E2M1 rounding of y / s
 * (0 where s = 0), both to nearest even; the cache then stands for q * s * g.  Values beyond 2688 g
 * saturate; a NaN makes its block NaN.
 *
 * Batch.  Sequence b of a batch has the new tokens [q_start[b], q_start[b+1]) of the token tensors and a
 * context of kv_len[b] positions that includes them: its new token i is at position
 * kv_len[b] - (q_start[b+1] - q_start[b]) + i.  Position p of sequence b lives in page
 * pages[b * pages_stride + p / page_tokens] at slot p % page_tokens.  The three arrays are device
 * memory, read by the kernels; values that point outside the cache are never dereferenced (see each
 * call).
 *
 * Rotary positions (rope_dim R > 0): the first R dims of each key and query head are rotated in pairs
 * by a table of fp32 [rows][2][R/2] -- row p: R/2 cosines, then R/2 sines of position p -- which the
 * caller makes once for its base frequency and context scaling.  Pairs are (i, i + R/2), or
 * (2i, 2i + 1) with BSG_KV_ROPE_INTERLEAVED: (x1, x2) -> (x1 c - x2 s, x2 c + x1 s) in fp32.
 */
#ifndef BSG_KV_H
#define BSG_KV_H

#include "bsg.h"

#ifdef __cplusplus
extern "C" {
#endif

enum {
  BSG_KV_ROPE_INTERLEAVED = 1u << 0, /* rotate neighbouring dims instead of the two halves */
  BSG_KV_NONCAUSAL = 1u << 1         /* every query sees the whole context (default: positions <= its own) */
};

typedef struct bsg_kv_problem {
  uint32_t struct_size; /* = sizeof(bsg_kv_problem) */
  int32_t dtype;        /* bsg_out_dtype of q, k, v and the outputs */
  int32_t q_heads;      /* a multiple of kv_heads; query head j reads key/value head j / (q_heads / kv_heads) */
  int32_t kv_heads;     /* 1 .. 1024 */
  int32_t head_dim;     /* 64 or 128 */
  int32_t page_tokens;  /* 16, 32, 64, 128 or 256 */
  int64_t num_pages;    /* pages in the cache, 1 .. 2^31 - 1 */
  int64_t page_stride;  /* bytes from page to page, a multiple of 16; 0 = packed */
  int64_t max_tokens;   /* the most new tokens, and the most sequences, of a call */
  uint32_t flags;       /* BSG_KV_* */
  int32_t rope_dim;     /* rotated dims, 0 or a multiple of 16 up to head_dim */
  int32_t window;       /* > 0: a query at position p sees positions (p - window, p]; 0 (or 2^30 and more) = all */
  float scale;          /* of the scores; 0 = 1 / sqrt(head_dim) */
  float softcap;        /* > 0: scores become softcap * tanh(score / softcap), within 2^-16 or 2^-19 of that; 0 = none */
  float k_scale, v_scale; /* global scales of stored keys and values; 0 = 1 */
  int32_t device;       /* HIP device ordinal; -1 = the current device at create time */
} bsg_kv_problem;

typedef struct bsg_kv_batch {
  uint32_t struct_size; /* = sizeof(bsg_kv_batch) */
  int32_t num_seqs;     /* 0 .. max_tokens */
  int64_t num_tokens;   /* new tokens of all sequences = q_start[num_seqs], 0 .. max_tokens */
  int32_t max_q;        /* no sequence has more new tokens than this; in [num_tokens / num_seqs, num_tokens] */
  int32_t max_kv;       /* no kv_len is larger than this (bsg_kv_attend reads larger ones as this; bsg_kv_append and
                         * bsg_kv_read take positions from kv_len as it is and leave out those from max_kv on) */
  const int32_t* q_start; /* device [num_seqs + 1], ascending from 0 */
  const int32_t* kv_len;  /* device [num_seqs] */
  const int32_t* pages;   /* device [num_seqs][pages_stride] */
  int64_t pages_stride;   /* entries per sequence; pages_stride * page_tokens >= max_kv */
} bsg_kv_batch;

/* A tensor [tokens][heads][head_dim] of 16-bit values: head_dim contiguous, strides in elements,
 * multiples of 8; the pointer 16-byte aligned. */
typedef struct bsg_heads {
  void* ptr;
  int64_t token_stride, head_stride;
} bsg_heads;

typedef struct bsg_kv_plan_s* bsg_kv_plan; /* opaque, library-owned */

typedef struct bsg_kv_plan_info {
  uint32_t struct_size; /* = sizeof(bsg_kv_plan_info), set by the caller */
  int32_t reserved;
  int64_t page_bytes;      /* bytes of a packed page */
  int64_t page_stride;     /* bytes from page to page of this plan */
  uint64_t workspace_bytes;
} bsg_kv_plan_info;

/* Validate and make a plan with its device workspace (partial results of contexts that are split
 * over workgroups, and their arrival counters).  Calls on one plan must be ordered (one stream, or
 * events): they share the workspace.  One plan serves every layer of the same geometry.
 * Errors: BSG_ERR_NULL, _ABI, _SHAPE, _UNSUPPORTED, _ALIGN, _DEVICE, _HIP, _ALLOC. */
bsg_status bsg_kv_plan_create(const bsg_kv_problem* problem, bsg_kv_plan* out_plan);
bsg_status bsg_kv_plan_destroy(bsg_kv_plan plan); /* NULL is accepted */
bsg_status bsg_kv_plan_query(bsg_kv_plan plan, bsg_kv_plan_info* info);

/* Bytes of one packed page (0 for a geometry that bsg_kv_plan_create refuses). */
int64_t bsg_kv_page_bytes(int32_t kv_heads, int32_t head_dim, int32_t page_tokens);

/* Store the batch's new keys and values at their positions, keys rotated; with q, also write the
 * rotated queries to q_out (which may be q itself).  k, v: [num_tokens][kv_heads][head_dim]; q, q_out:
 * [num_tokens][q_heads][head_dim], both or neither.  rope: the table, required iff rope_dim > 0, 16-byte
 * aligned, with rope_rows >= max_kv rows.  A token whose position is negative or not below max_kv, or
 * whose page number is not in [0, num_pages), is not stored.  Distinct tokens of a call must have
 * distinct slots.  Errors: BSG_ERR_NULL, _ABI, _SHAPE, _ALIGN, _HIP. */
bsg_status bsg_kv_append(bsg_kv_plan plan, const bsg_kv_batch* batch, const bsg_heads* q, const bsg_heads* k,
                         const bsg_heads* v, const bsg_heads* q_out, const float* rope, int64_t rope_rows,
                         void* cache, void* stream);

/* out = softmax(scale * k_scale * q . K) V * v_scale over each query's visible positions; a query that
 * sees none gives zeros.  lse (or NULL): float [num_tokens][q_heads], the natural logarithm of the sum
 * of the exponentials of the scores (-inf where none is visible).  Cache slots that no query sees are
 * never used as numbers.  Page numbers outside [0, num_pages) are read as the nearest valid page.  Scores,
 * their statistics and all sums are fp32; the weights are rounded to fp16 for their products with V (2^-11 of
 * themselves; those below 2^-34 of a row's largest may count as zero), and the output is rounded once.
 * Errors: as bsg_kv_append, and BSG_ERR_UNSUPPORTED for more work than one call can count: about 2^31 tiles of 64
 * positions over all sequences, heads and blocks of 16 rows, or 2^32 threads of the many-row kernel. */
bsg_status bsg_kv_attend(bsg_kv_plan plan, const bsg_kv_batch* batch, const bsg_heads* q, const void* cache,
                         const bsg_heads* out, float* lse, void* stream);

/* The values that the cache holds at the positions of the batch's new tokens: k, v
 * [num_tokens][kv_heads][head_dim] (rounded to the plan's dtype; exact while k_scale and v_scale are
 * powers of two that keep them in its range).  Tokens that bsg_kv_append would not store read as zeros.
 * Errors: as bsg_kv_append. */
bsg_status bsg_kv_read(bsg_kv_plan plan, const bsg_kv_batch* batch, const void* cache, const bsg_heads* k,
                       const bsg_heads* v, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* BSG_KV_H */
