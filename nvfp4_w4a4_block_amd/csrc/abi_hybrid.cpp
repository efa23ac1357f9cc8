// C ABI of the gated delta rule, the rotary append and the token log
// probabilities (declared in include/nvfp4.h): argument validation on the host,
// then dispatch, as in abi.cpp.
#include "nvfp4.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "hybrid_launch.h"

namespace {

constexpr int64_t kMaxInt = (int64_t)1 << 31;     // exclusive
constexpr int64_t kMaxTokens = (int64_t)1 << 30;  // tokens a table row covers
constexpr int64_t kMaxTable = (int64_t)1 << 29;   // entries of a page table
constexpr int64_t kMaxRows = (int64_t)1 << 24;    // rows of one call
constexpr int64_t kMaxHeads = 1024;
constexpr int64_t kMaxGroup = 256;                // query heads of a KV head

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
bool dtype_ok(int dt) { return dt == NVFP4_F32 || dt == NVFP4_BF16; }
nvfp4_status from_hip(hipError_t e) { return e == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP; }
bool dim_ok(int64_t d) { return d == 64 || d == 128 || d == 256; }
bool is_finite(double x) { return x > -__builtin_inf() && x < __builtin_inf(); }
int64_t size_of(nvfp4_dtype dt) { return dt == NVFP4_BF16 ? 2 : 4; }

bool rows_ok(int64_t B, int64_t M) {
  return B >= 0 && B <= 65535 && M >= 0 && M <= 65535 && (M == 0 || B <= kMaxRows / M);
}

// Values from a row to the next: at least a row, and 16-byte aligned rows.
bool stride_ok(int64_t stride, int64_t row, nvfp4_dtype dt) {
  return stride >= row && stride < kMaxInt && stride * size_of(dt) % 16 == 0;
}

// Whether rows (n of them, `row` values, `stride` apart) and out's bytes share any.
bool overlap(const void* rows, int64_t n, int64_t row, int64_t stride, nvfp4_dtype dt, const void* out,
             int64_t out_bytes) {
  const uintptr_t r0 = (uintptr_t)rows, o0 = (uintptr_t)out;
  return r0 < o0 + out_bytes && o0 < r0 + ((n - 1) * stride + row) * size_of(dt);
}

bool delta_shape_ok(int64_t B, int64_t M, int64_t Hk, int64_t H, int64_t Dk, int64_t Dv, int64_t S) {
  return rows_ok(B, M) && H >= 1 && H <= kMaxHeads && Hk >= 1 && H % Hk == 0 && dim_ok(Dk) && dim_ok(Dv) && S >= 1 &&
         S < kMaxInt;
}

nvfp4::DeltaArgs delta_of(int64_t B, int64_t M, int64_t Hk, int64_t H, int64_t Dk, int64_t Dv, int64_t S,
                          nvfp4_dtype dt) {
  nvfp4::DeltaArgs a = {};
  a.seqs = (int)B;
  a.nodes = (int)M;
  a.key_heads = (int)Hk;
  a.heads = (int)H;
  a.dk = (int)Dk;
  a.dv = (int)Dv;
  a.slots = (int)S;
  a.bf16 = dt == NVFP4_BF16;
  return a;
}

// Whether an output's bytes are some of q's, k's, v's or the states': several
// workgroups read a row or state that one of them would write.
bool shared(const nvfp4::DeltaArgs& a, nvfp4_dtype dt, const void* out, int64_t bytes) {
  const int64_t n = (int64_t)a.seqs * a.nodes, key_row = (int64_t)a.key_heads * a.dk, row = (int64_t)a.heads * a.dv;
  return overlap(a.q, n, key_row, a.q_stride, dt, out, bytes) || overlap(a.k, n, key_row, a.k_stride, dt, out, bytes) ||
         overlap(a.v, n, row, a.v_stride, dt, out, bytes) ||
         overlap(a.states, a.slots, row * a.dk, row * a.dk, NVFP4_F32, out, bytes);
}

// The rows that a chain and a tree have in common; M == 0 needs none of them.
nvfp4_status delta_rows(nvfp4::DeltaArgs& a, nvfp4_dtype dt, const void* q, const void* k, const void* v,
                        int64_t q_stride, int64_t k_stride, int64_t v_stride, const float* g, const float* beta,
                        float scale, float norm_eps, const float* states, const int32_t* src, const int32_t* counts,
                        void* out) {
  const bool rows = a.nodes > 0;
  if (!states || !src || (rows && (!q || !k || !v || !g || !beta || !out))) return NVFP4_ERR_NULL;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(out, 16) || !aligned(states, 16) ||
      !aligned(g, 4) || !aligned(beta, 4) || !aligned(src, 4) || !aligned(counts, 4))
    return NVFP4_ERR_ALIGN;
  a.q = q;
  a.k = k;
  a.v = v;
  a.q_stride = q_stride;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.g = g;
  a.beta = beta;
  a.scale = scale;
  a.norm_eps = norm_eps;
  a.states = const_cast<float*>(states);
  a.src = src;
  a.counts = counts;
  a.out = out;
  if (rows && shared(a, dt, out, (int64_t)a.seqs * a.nodes * a.heads * a.dv * size_of(dt))) return NVFP4_ERR_SHAPE;
  return NVFP4_OK;
}

bool delta_values_ok(int64_t Hk, int64_t H, int64_t Dk, int64_t Dv, nvfp4_dtype dt, int64_t q_stride,
                     int64_t k_stride, int64_t v_stride, float scale, float norm_eps) {
  return stride_ok(q_stride, Hk * Dk, dt) && stride_ok(k_stride, Hk * Dk, dt) && stride_ok(v_stride, H * Dv, dt) &&
         is_finite(scale) && is_finite(norm_eps);
}

}  // namespace

extern "C" {

nvfp4_status nvfp4_kv_append_rope(int64_t B, int64_t M, int64_t Hq, int64_t H, int64_t D, int64_t R,
                                  int64_t page_size, int64_t P, int64_t W, const void* q, const void* k,
                                  const void* v, nvfp4_dtype dt, int64_t q_stride, int64_t k_stride,
                                  int64_t v_stride, const double* inv_freq, double rope_scale, int interleaved,
                                  const float* k_scale, const float* v_scale, uint8_t* k_pages, uint8_t* v_pages,
                                  int64_t page_stride, const int32_t* table, const int32_t* lens,
                                  const int32_t* parent, const int32_t* counts, void* q_out, void* stream) {
  if (!dtype_ok(dt)) return NVFP4_ERR_DTYPE;
  if (!rows_ok(B, M) || H < 1 || H > kMaxHeads || Hq < 1 || Hq > kMaxHeads * kMaxGroup || !dim_ok(D) || R < 16 ||
      R > D || R % 16 != 0 || page_size < 16 || page_size > 1024 || (page_size & (page_size - 1)) != 0 || P < 1 ||
      P >= kMaxInt || W < 1 || W > kMaxTokens / page_size || (B > 0 && W > kMaxTable / B) ||
      page_stride < H * page_size * D || page_stride >= kMaxInt || page_stride % 16 != 0 ||
      !stride_ok(q_stride, Hq * D, dt) || !stride_ok(k_stride, H * D, dt) || !stride_ok(v_stride, H * D, dt) ||
      !is_finite(rope_scale) || (parent && M > 64))
    return NVFP4_ERR_SHAPE;
  if (B == 0 || M == 0) return NVFP4_OK;
  if (!q || !k || !v || !inv_freq || !k_scale || !v_scale || !k_pages || !v_pages || !table || !lens || !q_out)
    return NVFP4_ERR_NULL;
  if (!aligned(q, 16) || !aligned(k, 16) || !aligned(v, 16) || !aligned(q_out, 16) || !aligned(k_pages, 16) ||
      !aligned(v_pages, 16) || !aligned(inv_freq, 8) || !aligned(k_scale, 4) || !aligned(v_scale, 4) ||
      !aligned(table, 4) || !aligned(lens, 4) || !aligned(parent, 4) || !aligned(counts, 4))
    return NVFP4_ERR_ALIGN;
  if (k_pages == v_pages) return NVFP4_ERR_SHAPE;  // two writers of a row
  const int64_t n = B * M, bytes = n * Hq * D * size_of(dt);
  const bool in_place = q_out == q && q_stride == Hq * D;  // each value is read and written by one thread
  if ((!in_place && overlap(q, n, Hq * D, q_stride, dt, q_out, bytes)) ||
      overlap(k, n, H * D, k_stride, dt, q_out, bytes) || overlap(v, n, H * D, v_stride, dt, q_out, bytes))
    return NVFP4_ERR_SHAPE;
  nvfp4::KvRopeArgs a = {};
  nvfp4::KvCache& c = a.append.c;
  c.k = k_pages;
  c.v = v_pages;
  c.page_stride = page_stride;
  c.pages = (int)P;
  c.heads = (int)H;
  c.page_shift = __builtin_ctzll((unsigned long long)page_size);
  c.dim = (int)D;
  c.table = table;
  c.lens = lens;
  c.seqs = (int)B;
  c.width = (int)W;
  a.append.nodes = (int)M;
  a.append.x_k = k;
  a.append.x_v = v;
  a.append.k_stride = k_stride;
  a.append.v_stride = v_stride;
  a.append.bf16 = dt == NVFP4_BF16;
  a.append.k_scale = k_scale;
  a.append.v_scale = v_scale;
  a.append.counts = counts;
  a.q = q;
  a.q_stride = q_stride;
  a.q_heads = (int)Hq;
  a.rotary = (int)R;
  a.interleaved = interleaved != 0;
  a.inv_freq = inv_freq;
  a.rope_scale = rope_scale;
  a.parent = parent;
  a.q_out = q_out;
  return from_hip(nvfp4::launch_kv_append_rope(a, static_cast<hipStream_t>(stream)));
}

int64_t nvfp4_delta_rule_workspace_bytes(int64_t B, int64_t M, int64_t Hk, int64_t H, int64_t Dk, int64_t Dv,
                                         nvfp4_dtype dt) {
  if (!dtype_ok(dt) || !delta_shape_ok(B, M, Hk, H, Dk, Dv, 1) || B == 0 || M == 0) return 0;
  return nvfp4::delta_rule_workspace_bytes(delta_of(B, M, Hk, H, Dk, Dv, 1, dt));
}

nvfp4_status nvfp4_delta_rule(int64_t B, int64_t M, int64_t Hk, int64_t H, int64_t Dk, int64_t Dv, int64_t S,
                              const void* q, const void* k, const void* v, nvfp4_dtype dt, int64_t q_stride,
                              int64_t k_stride, int64_t v_stride, const float* g, const float* beta, float scale,
                              float norm_eps, float* states, const int32_t* src, const int32_t* dst,
                              const int32_t* counts, void* out, void* workspace, int64_t workspace_bytes,
                              void* stream) {
  if (!dtype_ok(dt)) return NVFP4_ERR_DTYPE;
  if (!delta_shape_ok(B, M, Hk, H, Dk, Dv, S) || workspace_bytes < 0 ||
      !delta_values_ok(Hk, H, Dk, Dv, dt, q_stride, k_stride, v_stride, scale, norm_eps))
    return NVFP4_ERR_SHAPE;
  if (B == 0) return NVFP4_OK;
  if (!dst || (workspace_bytes > 0 && !workspace)) return NVFP4_ERR_NULL;
  nvfp4::DeltaArgs a = delta_of(B, M, Hk, H, Dk, Dv, S, dt);
  const nvfp4_status st = delta_rows(a, dt, q, k, v, q_stride, k_stride, v_stride, g, beta, scale, norm_eps, states,
                                     src, counts, out);
  if (st != NVFP4_OK) return st;
  if (!aligned(dst, 4) || !aligned(workspace, 16)) return NVFP4_ERR_ALIGN;
  a.dst = dst;
  a.workspace = workspace;
  a.workspace_bytes = workspace_bytes;
  return from_hip(nvfp4::launch_delta_rule(a, static_cast<hipStream_t>(stream)));
}

nvfp4_status nvfp4_delta_tree(int64_t B, int64_t M, int64_t Hk, int64_t H, int64_t Dk, int64_t Dv, int64_t S,
                              const void* q, const void* k, const void* v, nvfp4_dtype dt, int64_t q_stride,
                              int64_t k_stride, int64_t v_stride, const float* g, const float* beta, float scale,
                              float norm_eps, const float* states, const int32_t* src, const int32_t* parent,
                              const int32_t* counts, void* out, float* keys, float* updates, void* stream) {
  if (!dtype_ok(dt)) return NVFP4_ERR_DTYPE;
  if (!delta_shape_ok(B, M, Hk, H, Dk, Dv, S) || M > 64 ||
      !delta_values_ok(Hk, H, Dk, Dv, dt, q_stride, k_stride, v_stride, scale, norm_eps))
    return NVFP4_ERR_SHAPE;
  if (B == 0 || M == 0) return NVFP4_OK;
  if (!parent || !keys || !updates) return NVFP4_ERR_NULL;
  nvfp4::DeltaArgs a = delta_of(B, M, Hk, H, Dk, Dv, S, dt);
  const nvfp4_status st = delta_rows(a, dt, q, k, v, q_stride, k_stride, v_stride, g, beta, scale, norm_eps, states,
                                     src, counts, out);
  if (st != NVFP4_OK) return st;
  if (!aligned(parent, 4) || !aligned(keys, 16) || !aligned(updates, 16)) return NVFP4_ERR_ALIGN;
  const int64_t n = B * M, key_bytes = n * Hk * Dk * 4, update_bytes = n * H * Dv * 4;
  if (shared(a, dt, keys, key_bytes) || shared(a, dt, updates, update_bytes) ||
      overlap(out, n, H * Dv, H * Dv, dt, keys, key_bytes) || overlap(out, n, H * Dv, H * Dv, dt, updates, update_bytes) ||
      overlap(keys, n, Hk * Dk, Hk * Dk, NVFP4_F32, updates, update_bytes))
    return NVFP4_ERR_SHAPE;
  a.parent = parent;
  a.keys = keys;
  a.updates = updates;
  return from_hip(nvfp4::launch_delta_tree(a, static_cast<hipStream_t>(stream)));
}

nvfp4_status nvfp4_delta_commit(int64_t L, int64_t B, int64_t M, int64_t Hk, int64_t H, int64_t Dk, int64_t Dv,
                                int64_t S, float* states, const float* keys, const float* updates, const float* g,
                                const int32_t* result, const int32_t* src, const int32_t* dst, void* stream) {
  return nvfp4_delta_commit_counts(L, B, M, Hk, H, Dk, Dv, S, states, keys, updates, g, result, src, dst, nullptr,
                                   stream);
}

nvfp4_status nvfp4_delta_commit_counts(int64_t L, int64_t B, int64_t M, int64_t Hk, int64_t H, int64_t Dk,
                                       int64_t Dv, int64_t S, float* states, const float* keys,
                                       const float* updates, const float* g, const int32_t* result,
                                       const int32_t* src, const int32_t* dst, const int32_t* counts,
                                       void* stream) {
  if (!delta_shape_ok(B, M, Hk, H, Dk, Dv, S) || M < 1 || M > 64 || L < 0 || L > 4096)
    return NVFP4_ERR_SHAPE;
  if (L == 0 || B == 0) return NVFP4_OK;
  if (!states || !keys || !updates || !g || !result || !src || !dst) return NVFP4_ERR_NULL;
  if (!aligned(states, 16) || !aligned(keys, 16) || !aligned(updates, 16) || !aligned(g, 4) || !aligned(result, 4) ||
      !aligned(src, 4) || !aligned(dst, 4) || !aligned(counts, 4))
    return NVFP4_ERR_ALIGN;
  nvfp4::DeltaCommitArgs a;
  a.layers = (int)L;
  a.seqs = (int)B;
  a.nodes = (int)M;
  a.key_heads = (int)Hk;
  a.heads = (int)H;
  a.dk = (int)Dk;
  a.dv = (int)Dv;
  a.slots = (int)S;
  a.states = states;
  a.keys = keys;
  a.updates = updates;
  a.g = g;
  a.result = result;
  a.src = src;
  a.dst = dst;
  a.counts = counts;
  return from_hip(nvfp4::launch_delta_commit(a, static_cast<hipStream_t>(stream)));
}

int64_t nvfp4_token_logprobs_workspace_bytes(int64_t M, int64_t N, int64_t top, nvfp4_dtype dt) {
  if (!dtype_ok(dt) || M < 1 || M > 65535 || N < 1 || N >= kMaxRows || top < 0 || top > 64 || top > N) return 0;
  nvfp4::LogprobArgs a = {};
  a.rows = (int)M;
  a.vocab = (int)N;
  a.top = (int)top;
  a.bf16 = dt == NVFP4_BF16;
  return nvfp4::token_logprobs_workspace_bytes(a);
}

nvfp4_status nvfp4_token_logprobs(int64_t M, int64_t N, int64_t top, const void* logits, nvfp4_dtype dt,
                                  int64_t stride, const int32_t* tokens, float* logprobs, float* entropy,
                                  float* top_logprobs, int32_t* top_tokens, void* workspace,
                                  int64_t workspace_bytes, void* stream) {
  if (!dtype_ok(dt)) return NVFP4_ERR_DTYPE;
  if (M < 0 || M > 65535 || N < 1 || N >= kMaxRows || top < 0 || top > 64 || top > N || stride < N ||
      stride >= kMaxInt)
    return NVFP4_ERR_SHAPE;
  if (M == 0) return NVFP4_OK;
  if (!logits || !tokens || !logprobs || !entropy || !workspace || (top > 0 && (!top_logprobs || !top_tokens)))
    return NVFP4_ERR_NULL;
  if (!aligned(logits, size_of(dt)) || !aligned(workspace, 16) || !aligned(tokens, 4) || !aligned(logprobs, 4) ||
      !aligned(entropy, 4) || !aligned(top_logprobs, 4) || !aligned(top_tokens, 4))
    return NVFP4_ERR_ALIGN;
  nvfp4::LogprobArgs a = {};
  a.rows = (int)M;
  a.vocab = (int)N;
  a.top = (int)top;
  a.logits = logits;
  a.stride = stride;
  a.bf16 = dt == NVFP4_BF16;
  a.tokens = tokens;
  a.logprobs = logprobs;
  a.entropy = entropy;
  a.top_logprobs = top_logprobs;
  a.top_tokens = top_tokens;
  a.workspace = workspace;
  if (workspace_bytes < nvfp4::token_logprobs_workspace_bytes(a)) return NVFP4_ERR_SHAPE;
  return from_hip(nvfp4::launch_token_logprobs(a, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
