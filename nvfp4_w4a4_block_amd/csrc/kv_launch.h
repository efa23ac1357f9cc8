// Host-side launchers of the paged FP8 KV cache (internal to the library; the
// public C ABI is include/nvfp4.h).  Arguments are already validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace nvfp4 {

// Paged FP8 KV cache: the K and V pages (k + layer * layer_stride + page *
// page_stride bytes: one page of [heads][1 << page_shift][dim] E4M3 bytes), the
// table [seqs][width] of page ids and the committed lengths lens [seqs].
struct KvCache {
  uint8_t* k = nullptr;
  uint8_t* v = nullptr;
  int64_t layer_stride = 0, page_stride = 0;
  int layers = 1, pages = 0, heads = 0, page_shift = 0, dim = 0;
  const int32_t* table = nullptr;
  const int32_t* lens = nullptr;
  int seqs = 0, width = 0;
};

struct KvAppendArgs {
  KvCache c;
  int nodes;
  const void *x_k, *x_v;  // rows of heads * dim values, row b * nodes + v
  int64_t k_stride, v_stride;  // values from a row to the next
  bool bf16;
  const float *k_scale, *v_scale;
  const int32_t* counts;  // optional [seqs]
};

struct KvCompactArgs {
  KvCache c;
  int nodes;
  const int32_t* result;  // [seqs][3 + nodes]
  int32_t* new_lens;      // [seqs]
};

// Rows of queries over the cache (kv_attention.hip).
struct KvAttentionArgs {
  KvCache c;
  int nodes, group;  // query heads = heads * group
  const void* q;
  int64_t q_stride;  // values from a row to the next
  bool bf16;
  float sm_scale;
  const float *k_scale, *v_scale;
  const int32_t* parent;  // optional [seqs][nodes]
  const int32_t* counts;  // optional [seqs]
  void* out;              // [seqs][nodes][heads * group][dim]
  float* lse;             // optional [seqs][nodes][heads * group]
  void* workspace;
  int64_t workspace_bytes;
};

// Page table, holder counts and free list (kv_pool.hip).
struct KvPoolArgs {
  int n, seqs, width, pages, page_shift;
  int32_t *table, *held, *refs, *free_list, *shortage;
  const int32_t *src, *dst, *tokens;  // resize: dst names the sequences
  int32_t* moves;                     // fork: [n][3] page to copy, to, used slots (-1: none)
};

hipError_t launch_kv_append(const KvAppendArgs& a, hipStream_t stream);
hipError_t launch_kv_compact(const KvCompactArgs& a, hipStream_t stream);
bool kv_attention_supported(const KvAttentionArgs& a);  // one launch holds its items
int64_t kv_attention_workspace_bytes(const KvAttentionArgs& a);
hipError_t launch_kv_attention(const KvAttentionArgs& a, hipStream_t stream);
hipError_t launch_kv_resize(const KvPoolArgs& a, hipStream_t stream);
hipError_t launch_kv_fork(const KvPoolArgs& a, const KvCache& c, hipStream_t stream);

}  // namespace nvfp4
