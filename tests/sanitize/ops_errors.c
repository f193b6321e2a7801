/* Drives the host-side paths of bsg_kv.h and bsg_moe.h that need no GPU: every field's validation with
 * extreme values, handles that are no plans, and the forced-architecture refusal. */
#include <limits.h>
#include <math.h>
#include <stdio.h>
#include <string.h>

#include "bsg_kv.h"
#include "bsg_moe.h"

static int failures = 0;

static void expect(const char* what, bsg_status got, bsg_status want) {
  if (got != want || !bsg_last_error() || strlen(bsg_last_error()) >= 512) {
    printf("FAIL %s: got %s want %s (%s)\n", what, bsg_status_string(got), bsg_status_string(want), bsg_last_error());
    ++failures;
  }
}

static bsg_kv_problem kv(void) {
  bsg_kv_problem p;
  memset(&p, 0, sizeof(p));
  p.struct_size = sizeof(p);
  p.dtype = BSG_OUT_BF16;
  p.q_heads = 8;
  p.kv_heads = 2;
  p.head_dim = 64;
  p.page_tokens = 16;
  p.num_pages = 4;
  p.max_tokens = 8;
  p.device = -1;
  return p;
}

static bsg_moe_problem moe(void) {
  bsg_moe_problem p;
  memset(&p, 0, sizeof(p));
  p.struct_size = sizeof(p);
  p.format = BSG_FMT_NVFP4;
  p.dtype = BSG_OUT_BF16;
  p.experts = 8;
  p.top_k = 2;
  p.hidden = p.inter = 64;
  p.max_tokens = 4;
  p.device = -1;
  return p;
}

static void kv_case(const char* what, bsg_kv_problem p, bsg_status want) {
  bsg_kv_plan plan = (bsg_kv_plan)0x1;
  expect(what, bsg_kv_plan_create(&p, &plan), want);
  if (plan) { printf("FAIL %s: handle not cleared\n", what); ++failures; }
}

static void moe_case(const char* what, bsg_moe_problem p, bsg_status want) {
  bsg_moe_plan plan = (bsg_moe_plan)0x1;
  expect(what, bsg_moe_plan_create(&p, &plan), want);
  if (plan) { printf("FAIL %s: handle not cleared\n", what); ++failures; }
}

int main(void) {
  static unsigned char fake[8192];
  bsg_kv_problem p;
  bsg_moe_problem m;
  expect("kv null", bsg_kv_plan_create(NULL, NULL), BSG_ERR_NULL);
  p = kv(); p.struct_size = 0;             kv_case("kv size", p, BSG_ERR_ABI);
  p = kv(); p.dtype = INT_MIN;             kv_case("kv dtype", p, BSG_ERR_ABI);
  p = kv(); p.flags = 1u << 31;            kv_case("kv flags", p, BSG_ERR_ABI);
  p = kv(); p.q_heads = INT_MAX;           kv_case("kv q_heads", p, BSG_ERR_SHAPE);
  p = kv(); p.kv_heads = INT_MIN;          kv_case("kv kv_heads", p, BSG_ERR_SHAPE);
  p = kv(); p.head_dim = INT_MAX;          kv_case("kv head_dim", p, BSG_ERR_UNSUPPORTED);
  p = kv(); p.page_tokens = INT_MIN;       kv_case("kv page_tokens", p, BSG_ERR_SHAPE);
  p = kv(); p.num_pages = INT64_MAX;       kv_case("kv num_pages", p, BSG_ERR_SHAPE);
  p = kv(); p.max_tokens = INT64_MAX;      kv_case("kv max_tokens", p, BSG_ERR_SHAPE);
  p = kv(); p.page_stride = INT64_MIN;     kv_case("kv page_stride low", p, BSG_ERR_SHAPE);
  p = kv(); p.page_stride = INT64_MAX;     kv_case("kv page_stride high", p, BSG_ERR_SHAPE);
  p = kv(); p.rope_dim = INT_MIN;          kv_case("kv rope_dim", p, BSG_ERR_SHAPE);
  p = kv(); p.window = INT_MIN;            kv_case("kv window", p, BSG_ERR_SHAPE);
  p = kv(); p.window = 5; p.flags = BSG_KV_NONCAUSAL; kv_case("kv window without causal", p, BSG_ERR_UNSUPPORTED);
  p = kv(); p.scale = NAN;                 kv_case("kv scale", p, BSG_ERR_SHAPE);
  p = kv(); p.k_scale = 1e-45f;            kv_case("kv k_scale", p, BSG_ERR_SHAPE);
  p = kv(); p.softcap = -0.5f;             kv_case("kv softcap", p, BSG_ERR_SHAPE);
  p = kv();                                kv_case("kv valid", p, BSG_ERR_DEVICE);
  if (!strstr(bsg_last_error(), "BSG_FORCE_ARCH")) { printf("FAIL forced-arch message\n"); ++failures; }
  if (bsg_kv_page_bytes(INT_MAX, INT_MAX, INT_MAX) || bsg_kv_page_bytes(INT_MIN, 64, 16) ||
      bsg_kv_page_bytes(1024, 128, 256) != (int64_t)1024 * 256 * 144) { printf("FAIL page bytes\n"); ++failures; }
  {
    bsg_kv_plan plans[2];
    int i;
    plans[0] = NULL;
    plans[1] = (bsg_kv_plan)fake;
    for (i = 0; i < 2; ++i) {
      expect("append", bsg_kv_append(plans[i], NULL, NULL, NULL, NULL, NULL, NULL, 0, NULL, NULL), BSG_ERR_NULL);
      expect("attend", bsg_kv_attend(plans[i], NULL, NULL, NULL, NULL, NULL, NULL), BSG_ERR_NULL);
      expect("read", bsg_kv_read(plans[i], NULL, NULL, NULL, NULL, NULL), BSG_ERR_NULL);
      expect("query", bsg_kv_plan_query(plans[i], NULL), BSG_ERR_NULL);
      expect("destroy", bsg_kv_plan_destroy(plans[i]), i ? BSG_ERR_NULL : BSG_OK);
      expect("run", bsg_moe_run((bsg_moe_plan)plans[i], 1, NULL, 0, NULL, NULL, 0, NULL, NULL, NULL), BSG_ERR_NULL);
      expect("destroy moe", bsg_moe_plan_destroy((bsg_moe_plan)plans[i]), i ? BSG_ERR_NULL : BSG_OK);
    }
  }
  expect("moe null", bsg_moe_plan_create(NULL, NULL), BSG_ERR_NULL);
  m = moe(); m.struct_size = 0;            moe_case("moe size", m, BSG_ERR_ABI);
  m = moe(); m.format = INT_MIN;           moe_case("moe format", m, BSG_ERR_ABI);
  m = moe(); m.flags = ~0u;                moe_case("moe flags", m, BSG_ERR_ABI);
  m = moe(); m.reserved = -1;              moe_case("moe reserved", m, BSG_ERR_ABI);
  m = moe(); m.experts = INT_MAX;          moe_case("moe experts", m, BSG_ERR_UNSUPPORTED);
  m = moe(); m.top_k = INT_MAX;            moe_case("moe top_k", m, BSG_ERR_SHAPE);
  m = moe(); m.hidden = INT64_MIN;         moe_case("moe hidden", m, BSG_ERR_SHAPE);
  m = moe(); m.inter = INT64_MAX - 31;     moe_case("moe inter", m, BSG_ERR_UNSUPPORTED);
  m = moe(); m.max_tokens = INT64_MAX;     moe_case("moe max_tokens", m, BSG_ERR_UNSUPPORTED);
  m = moe();                               moe_case("moe valid", m, BSG_ERR_DEVICE);
  printf("%s: %d failures\n", failures ? "FAIL" : "ok", failures);
  return failures != 0;
}
