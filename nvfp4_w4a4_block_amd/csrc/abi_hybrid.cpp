// C ABI of the gated delta rule, the rotary append and the token log
// probabilities (declared in include/nvfp4.h): argument validation on the host,
// then dispatch, as in abi.cpp.
#include "nvfp4.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

#include <initializer_list>

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

// Bytes of an array; none of a NULL one.
struct Span {
  uintptr_t begin;
  int64_t bytes;
};

Span span(const void* p, __int128 bytes) {
  const __int128 most = (int64_t)1 << 62;  // past any address
  return {(uintptr_t)p, p == nullptr || bytes <= 0 ? 0 : (int64_t)(bytes < most ? bytes : most)};
}

// n rows of `row` values, `stride` apart.
Span rows_span(const void* p, int64_t n, int64_t row, int64_t stride, int64_t size) {
  return span(p, n > 0 ? ((__int128)(n - 1) * stride + row) * size : 0);
}

bool apart(const Span& x, const Span& y) {
  return x.bytes == 0 || y.bytes == 0 || x.begin + x.bytes <= y.begin || y.begin + y.bytes <= x.begin;
}

// Whether outputs share no bytes with each other or with what is read: several
// workgroups read what one of them would write.
bool apart(std::initializer_list<Span> outs, std::initializer_list<Span> read) {
  for (const Span* x = outs.begin(); x != outs.end(); ++x) {
    for (const Span* y = outs.begin(); y != x; ++y)
      if (!apart(*x, *y)) return false;
    for (const Span& y : read)
      if (!apart(*x, y)) return false;
  }
  return true;
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

// Whether the outputs of a chain or tree share no bytes with each other or with its rows,
// states and numbers.
bool delta_apart(const nvfp4::DeltaArgs& a, std::initializer_list<Span> outs) {
  const int64_t n = (int64_t)a.seqs * a.nodes, key_row = (int64_t)a.key_heads * a.dk, row = (int64_t)a.heads * a.dv;
  const int64_t size = a.bf16 ? 2 : 4;
  return apart(outs, {rows_span(a.q, n, key_row, a.q_stride, size), rows_span(a.k, n, key_row, a.k_stride, size),
                      rows_span(a.v, n, row, a.v_stride, size), span(a.g, 4 * n * a.heads), span(a.beta, 4 * n * a.heads),
                      span(a.states, (__int128)4 * a.slots * row * a.dk), span(a.src, 4 * a.seqs),
                      span(a.dst, 4 * a.seqs), span(a.parent, 4 * n), span(a.counts, 4 * a.seqs)});
}

Span delta_out(const nvfp4::DeltaArgs& a) {
  return span(a.out, (__int128)a.seqs * a.nodes * a.heads * a.dv * (a.bf16 ? 2 : 4));
}

// The rows that a chain and a tree have in common; M == 0 needs none of them.
nvfp4_status delta_rows(nvfp4::DeltaArgs& a, const void* q, const void* k, const void* v,
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
  const int64_t n = B * M, size = size_of(dt);
  const Span out = span(q_out, n * Hq * D * size);
  const int64_t page_bytes = (P - 1) * page_stride + H * page_size * D;
  const bool in_place = q_out == q && q_stride == Hq * D;  // each value is read and written by one thread
  if (!apart({out}, {rows_span(in_place ? nullptr : q, n, Hq * D, q_stride, size),
                     rows_span(k, n, H * D, k_stride, size), rows_span(v, n, H * D, v_stride, size),
                     span(inv_freq, 4 * R), span(k_scale, 4), span(v_scale, 4), span(k_pages, page_bytes),
                     span(v_pages, page_bytes), span(table, 4 * B * W), span(lens, 4 * B), span(parent, 4 * n),
                     span(counts, 4 * B)}))
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
  const nvfp4_status st = delta_rows(a, q, k, v, q_stride, k_stride, v_stride, g, beta, scale, norm_eps, states,
                                     src, counts, out);
  if (st != NVFP4_OK) return st;
  if (!aligned(dst, 4) || !aligned(workspace, 16)) return NVFP4_ERR_ALIGN;
  a.dst = dst;
  a.workspace = workspace;
  a.workspace_bytes = workspace_bytes;
  if (!delta_apart(a, {delta_out(a), span(workspace, workspace_bytes)}))
    return NVFP4_ERR_SHAPE;
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
  const nvfp4_status st = delta_rows(a, q, k, v, q_stride, k_stride, v_stride, g, beta, scale, norm_eps, states,
                                     src, counts, out);
  if (st != NVFP4_OK) return st;
  if (!aligned(parent, 4) || !aligned(keys, 16) || !aligned(updates, 16)) return NVFP4_ERR_ALIGN;
  a.parent = parent;
  a.keys = keys;
  a.updates = updates;
  const int64_t n = B * M;
  if (!delta_apart(a, {delta_out(a), span(keys, 4 * n * Hk * Dk), span(updates, 4 * n * H * Dv)}))
    return NVFP4_ERR_SHAPE;
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
  const __int128 n = (__int128)L * B * M;
  if (!apart({span(states, (__int128)4 * L * S * H * Dv * Dk)},
             {span(keys, 4 * n * Hk * Dk), span(updates, 4 * n * H * Dv), span(g, 4 * n * H),
              span(result, 4 * B * (3 + M)), span(src, 4 * B), span(dst, 4 * B), span(counts, 4 * B)}))
    return NVFP4_ERR_SHAPE;
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
  if (!apart({span(logprobs, 4 * M), span(entropy, 4 * M), span(top > 0 ? top_logprobs : nullptr, 4 * M * top),
              span(top > 0 ? top_tokens : nullptr, 4 * M * top), span(workspace, workspace_bytes)},
             {rows_span(logits, M, N, stride, size_of(dt)), span(tokens, 4 * M)}))
    return NVFP4_ERR_SHAPE;
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
