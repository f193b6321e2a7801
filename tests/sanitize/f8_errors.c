/* Drives the host-side paths of bsg_f8.h that need no GPU: every field's validation with extreme values, handles that are
 * no plans, a launch that fails, and the forced-architecture refusal. */
#include <limits.h>
#include <stdio.h>
#include <string.h>

#include "bsg_f8.h"

static int failures = 0;

static void expect(const char* what, bsg_status got, bsg_status want) {
  if (got != want || !bsg_last_error() || strlen(bsg_last_error()) >= 512) {
    printf("FAIL %s: got %s want %s (%s)\n", what, bsg_status_string(got), bsg_status_string(want), bsg_last_error());
    ++failures;
  }
}

static bsg_f8_problem product(void) {
  bsg_f8_problem p;
  memset(&p, 0, sizeof(p));
  p.struct_size = sizeof(p);
  p.dtype = BSG_OUT_BF16;
  p.n = p.k = 64;
  p.max_tokens = 4;
  p.device = -1;
  return p;
}

/* The same change to a product's problem and to a feed-forward block's. */
static void plan_case(const char* what, bsg_f8_problem p, bsg_status want) {
  bsg_f8_ffn_problem f;
  bsg_f8_plan plan = (bsg_f8_plan)0x1;
  bsg_f8_ffn_plan ffn = (bsg_f8_ffn_plan)0x1;
  memset(&f, 0, sizeof(f));
  f.struct_size = p.struct_size == sizeof(p) ? sizeof(f) : p.struct_size;
  f.dtype = p.dtype;
  f.flags = p.flags;
  f.device = p.device;
  f.hidden = p.n;
  f.inter = p.k;
  f.max_tokens = p.max_tokens;
  expect(what, bsg_f8_plan_create(&p, &plan), want);
  expect(what, bsg_f8_ffn_plan_create(&f, &ffn), want);
  if (plan || ffn) { printf("FAIL %s: handle not cleared\n", what); ++failures; }
}

static void quantize_case(const char* what, int64_t rows, int64_t cols, int64_t xs, int64_t cs, int64_t ss, bsg_status want) {
  static uint64_t mem[64] __attribute__((aligned(16)));
  expect(what, bsg_f8_quantize(BSG_OUT_F16, rows, cols, mem, xs, mem, cs, (float*)mem, ss, NULL), want);
}

int main(void) {
  const int64_t huge[] = {LLONG_MIN, -1, 0, 8, BSG_F8_MAX_SIZE + 16, LLONG_MAX, LLONG_MAX - 15};
  const size_t n_huge = sizeof(huge) / sizeof(huge[0]);
  bsg_f8_problem p;
  for (size_t i = 0; i < n_huge; ++i) {
    p = product(); p.n = huge[i]; plan_case("n", p, BSG_ERR_SHAPE);
    p = product(); p.k = huge[i]; plan_case("k", p, BSG_ERR_SHAPE);
    if (huge[i] < 1 || huge[i] > BSG_F8_MAX_TOKENS) {
      p = product(); p.max_tokens = huge[i]; plan_case("max_tokens", p, BSG_ERR_SHAPE);
      quantize_case("rows", huge[i] ? huge[i] : -1, 64, 64, 64, 4, BSG_ERR_SHAPE);
    }
    quantize_case("cols", 1, huge[i], 64, 64, 4, BSG_ERR_SHAPE);
    if (huge[i]) {
      const bsg_status st = huge[i] % 16 ? BSG_ERR_ALIGN : BSG_ERR_SHAPE;
      if (huge[i] != BSG_F8_MAX_SIZE + 16) { /* a good stride */
        quantize_case("x_stride", 1, 64, huge[i], 64, 4, huge[i] % 8 ? BSG_ERR_ALIGN : BSG_ERR_SHAPE);
        quantize_case("codes_stride", 1, 64, 64, huge[i], 4, st);
        if (huge[i] != 8) quantize_case("scale_stride", 1, 64, 64, 64, huge[i], huge[i] % 4 ? BSG_ERR_ALIGN : BSG_ERR_SHAPE);
      }
    }
  }
  p = product(); p.dtype = INT_MAX; plan_case("dtype", p, BSG_ERR_ABI);
  p = product(); p.flags = UINT_MAX; plan_case("flags", p, BSG_ERR_ABI);
  p = product(); p.struct_size = 0; plan_case("struct_size", p, BSG_ERR_ABI);
  plan_case("architecture", product(), BSG_ERR_DEVICE);
  quantize_case("a launch that fails", 1, 64, 64, 64, 4, BSG_ERR_HIP);
  quantize_case("no rows", 0, 64, 64, 64, 4, BSG_OK);

  static uint64_t block[1024];
  uint64_t bytes = 0;
  expect("null plan", bsg_f8_run(NULL, 1, NULL, NULL, NULL, NULL, NULL, 0, NULL), BSG_ERR_NULL);
  expect("no plan", bsg_f8_run((bsg_f8_plan)block, LLONG_MIN, NULL, NULL, NULL, NULL, NULL, 0, NULL), BSG_ERR_NULL);
  expect("no ffn plan", bsg_f8_ffn_run((bsg_f8_ffn_plan)block, 1, NULL, 0, NULL, NULL, 0, NULL), BSG_ERR_NULL);
  expect("workspace", bsg_f8_plan_workspace((bsg_f8_plan)block, &bytes), BSG_ERR_NULL);
  expect("ffn workspace", bsg_f8_ffn_plan_workspace(NULL, &bytes), BSG_ERR_NULL);
  expect("destroy", bsg_f8_plan_destroy((bsg_f8_plan)block), BSG_ERR_NULL);
  expect("ffn destroy", bsg_f8_ffn_plan_destroy((bsg_f8_ffn_plan)block), BSG_ERR_NULL);
  expect("destroy null", bsg_f8_plan_destroy(NULL), BSG_OK);
  expect("ffn destroy null", bsg_f8_ffn_plan_destroy(NULL), BSG_OK);
  expect("null problem", bsg_f8_plan_create(NULL, NULL), BSG_ERR_NULL);
  expect("null ffn problem", bsg_f8_ffn_plan_create(NULL, NULL), BSG_ERR_NULL);
  printf("%s: %d failures\n", failures ? "failed" : "ok", failures);
  return failures != 0;
}
