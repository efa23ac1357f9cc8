// Host-side launchers of the gated delta rule, the rotary append and the token
// log probabilities (internal to the library; the public C ABI is
// include/nvfp4.h).  Arguments are already validated.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kv_launch.h"

namespace nvfp4 {

struct KvRopeArgs {
  KvAppendArgs append;  // keys, values, cache, lengths
  const void* q;        // rows of q_heads * dim values
  int64_t q_stride;
  int q_heads;
  int rotary;  // values of a head that turn
  bool interleaved;
  const double* inv_freq;  // [rotary / 2] radians per position
  double rope_scale;
  const int32_t* parent;  // optional [seqs][nodes]
  void* q_out;            // [seqs][nodes][q_heads][dim]
};

// A chain or trees of tokens through the gated delta rule (delta*.hip).
struct DeltaArgs {
  int seqs, nodes, key_heads, heads, dk, dv, slots;
  const void *q, *k, *v;
  int64_t q_stride, k_stride, v_stride;  // values from a row to the next
  bool bf16;
  const float *g, *beta;  // [seqs * nodes][heads]
  float scale, norm_eps;  // norm_eps negative: q and k as they are
  float* states;          // [slots][heads][dv][dk]
  const int32_t *src, *dst;
  const int32_t* parent;  // trees: [seqs][nodes]
  const int32_t* counts;  // optional [seqs]
  void* out;              // [seqs][nodes][heads][dv]
  float *keys, *updates;  // trees: [seqs][nodes][key_heads][dk], [seqs][nodes][heads][dv]
  void* workspace;
  int64_t workspace_bytes;
};

struct DeltaCommitArgs {
  int layers, seqs, nodes, key_heads, heads, dk, dv, slots;
  float* states;                      // [layers][slots][heads][dv][dk]
  const float *keys, *updates, *g;    // [layers][seqs][nodes] rows
  const int32_t *result, *src, *dst;  // [seqs][3 + nodes], [seqs], [seqs]
  const int32_t* counts;              // optional [seqs]
};

struct LogprobArgs {
  int rows, vocab, top;
  const void* logits;
  int64_t stride;
  bool bf16;
  const int32_t* tokens;
  float *logprobs, *entropy, *top_logprobs;
  int32_t* top_tokens;
  void* workspace;
};

hipError_t launch_kv_append_rope(const KvRopeArgs& a, hipStream_t stream);
int64_t delta_rule_workspace_bytes(const DeltaArgs& a);
hipError_t launch_delta_rule(const DeltaArgs& a, hipStream_t stream);
hipError_t launch_delta_tree(const DeltaArgs& a, hipStream_t stream);
hipError_t launch_delta_commit(const DeltaCommitArgs& a, hipStream_t stream);
int64_t token_logprobs_workspace_bytes(const LogprobArgs& a);
hipError_t launch_token_logprobs(const LogprobArgs& a, hipStream_t stream);

}  // namespace nvfp4
