// Shared definitions of the paged NVFP4 key/value cache kernels (include/bsg_kv.h): arguments, the
// page layout, and which position of which sequence a new token has.
#pragma once

#include "bsg_kv.h"
#include "codec.h"
#include "common.h"

namespace bsg {

struct HeadsArg {  // a bsg_heads, patched per call
  uint8_t* ptr;
  int64_t token_stride, head_stride;  // elements
};

constexpr int kForceShared = 1 << 30;  // in flags, beside BSG_KV_*: shared positions are read once wherever that can be

// Kernel arguments: the plan's part is filled at plan creation, the rest per call.
struct KvArgs {
  // plan
  int q_heads, kv_heads, group, page_shift;  // group = q_heads / kv_heads; page_tokens = 1 << page_shift
  int num_pages, rope_half, window, flags;
  int64_t page_stride;
  float score_mul;   // scale * k_scale: score = score_mul * q . (stored k)
  float cap, cap_inv;  // the soft cap in base 2, and its reciprocal; 0: none
  float k_inv, v_inv, v_scale, k_scale;
  // batch
  int num_seqs, num_tokens, max_q, max_kv;
  int mixed;         // attention: 1: sequences of up to kFewRows rows are the few-row kernel's, others the many-row kernel's
  int one_each;      // 1: every sequence has exactly one new token (token t is sequence t)
  const int* q_start;
  const int* kv_len;
  const int* pages;
  int64_t pages_stride;
  // operands
  HeadsArg q, k, v, out;
  const float* rope;
  uint8_t* cache;
  float* lse;
  // workspace of the attention kernels
  float* part;       // partial outputs and their softmax statistics
  int* group_arrived;  // arrival counters of groups of parts, and of units; zero between calls
  int* arrived;
  int splits;        // position splits of the many-row kernel
  int row_groups, row_width, row_listed;  // its workgroups (kv_split.h)
  // positions below `shared` lie in the same pages for all sequences; where they are read once for all, by the many-row
  // kernel, it leaves parts for the few-row kernel, which reads what lies behind them
  int shared;
  float* shared_part;
  int shared_rows, shared_width, shared_splits;  // rows of its blocks, blocks of a head, parts of a block; 0: none
};

// Byte offsets inside the chunk of one head of a page (P = page tokens, D = head dim).
template <int D>
struct PageLayout {
  static constexpr int kRow = D / 2;      // code bytes of one position
  static constexpr int kBlocks = D / 16;  // scale codes of one position
  __host__ __device__ static constexpr int chunk(int P) { return P * D + P * D / 8; }
  __host__ __device__ static constexpr int v_codes(int P) { return P * (D / 2); }
  __host__ __device__ static constexpr int k_scales(int P) { return P * D; }
  __host__ __device__ static constexpr int v_scales(int P) { return P * D + P * (D / 16); }
};

// q_start and kv_len as the kernels use them: clamped to what the host was told, so that no index
// formed from them leaves a buffer.
__device__ __forceinline__ int seq_start(const KvArgs& p, int b) {
  return min(max(p.q_start[b], 0), p.num_tokens);
}
__device__ __forceinline__ int seq_len(const KvArgs& p, int b) { return min(max(p.kv_len[b], 0), p.max_kv); }

__device__ __forceinline__ int clamp_page(const KvArgs& p, int page) { return min(max(page, 0), p.num_pages - 1); }

// dtype: 0 bf16, 1 f16.  Each returns the launch status; D is 64 or 128.
hipError_t kv_append_launch(const KvArgs& a, int dtype, int head_dim, bool with_q, hipStream_t stream);
hipError_t kv_read_launch(const KvArgs& a, int dtype, int head_dim, hipStream_t stream);
// (a.shared: what the caller says that all sequences share, whether or not that is made use of)
hipError_t kv_attend_launch(const KvArgs& a, int dtype, int head_dim, int cus, hipStream_t stream);

// Workspace of the attention kernels for calls of up to max_tokens tokens: floats of partials, then
// counters, the first of them those of groups.
void kv_workspace(const bsg_kv_problem& p, int cus, size_t* part_floats, size_t* counters, size_t* group_counters);

}  // namespace bsg
