// Shared definitions of the mixture-of-experts kernels (include/bsg_moe.h).
#pragma once

#include "bsg_moe.h"
#include "common.h"

namespace bsg {

struct MoeArgs {
  // plan
  int experts, top_k, hidden, inter, keep;
  // call
  int tokens;
  const uint16_t* x;
  const uint16_t* router;
  const uint8_t *w13, *s13, *w2, *s2;
  const float *alpha13, *alpha2;
  uint16_t* out;
  int* ids;
  float* weights;
  int64_t x_stride, out_stride;
  // workspace
  int router_parts;  // of the logits' sums over hidden
  float* logits;     // [router_parts][tokens][experts]
  uint16_t* xs;      // x as the first product takes it: [tokens][hidden], or [2][tokens][hidden] bf16 parts of it
  int* x_exp;        // [tokens] powers of two of scaled rows
  uint16_t* h;       // [2][tokens * top_k][inter] bf16 parts of SiLU(gate) up, rows grouped by expert
  float* y;          // [tokens * top_k][hidden] weighted outputs, rows grouped by expert
  int* active;       // number of slots
  int4* slots;       // (expert, first row, rows, 0): up to 16 rows of one expert
  int* row_token;    // [tokens * top_k]
  float* row_weight; // [tokens * top_k]
  int* row_of;       // [tokens][top_k] row of a token's choice
  int* arrived;      // [1 + hidden / 64 rounded up] arrival counters, zero between calls
};

// Bytes of the workspace, and `a`'s pointers into it (base may be null to ask for the size).
size_t moe_workspace(const bsg_moe_problem& p, uint8_t* base, MoeArgs* a, size_t* counters_at, size_t* counters_bytes);

// The kernels of one layer, in order.  format: 0 MXFP8, 1 NVFP4; dtype: 0 bf16, 1 f16.
hipError_t moe_launch(const MoeArgs& a, int format, int dtype, hipStream_t stream);

}  // namespace bsg
