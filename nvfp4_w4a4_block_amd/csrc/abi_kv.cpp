// C ABI of the paged FP8 KV cache (declared in include/nvfp4.h): argument
// validation on the host, then dispatch, as in abi.cpp.
#include "nvfp4.h"

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "kv_launch.h"

namespace {

constexpr int64_t kMaxInt = (int64_t)1 << 31;      // exclusive
constexpr int64_t kMaxTokens = (int64_t)1 << 30;   // tokens a table row covers
constexpr int64_t kMaxTable = (int64_t)1 << 29;    // entries of a page table
constexpr int64_t kMaxRows = (int64_t)1 << 24;     // query or key rows of one call
constexpr int64_t kMaxHeads = 1024;
constexpr int64_t kMaxGroup = 256;                 // query heads of a KV head
constexpr int64_t kMaxEntries = 1024;              // sequences of one fork or resize

bool aligned(const void* p, uintptr_t n) { return ((uintptr_t)p & (n - 1)) == 0; }
bool dtype_ok(int dt) { return dt == NVFP4_F32 || dt == NVFP4_BF16; }
nvfp4_status from_hip(hipError_t e) { return e == hipSuccess ? NVFP4_OK : NVFP4_ERR_HIP; }

bool page_size_ok(int64_t n) { return n >= 16 && n <= 1024 && (n & (n - 1)) == 0; }

int shift_of(int64_t n) {
  int s = 0;
  while (((int64_t)1 << s) < n) ++s;
  return s;
}

// The cache's geometry: heads, page size, head dimension, pages, strides (bytes).
// Layers lie behind each other, or side by side within the pages' stride.
bool pages_ok(int64_t L, int64_t P, int64_t H, int64_t page_size, int64_t D, int64_t layer_stride,
              int64_t page_stride) {
  if (L < 0 || L > 4096 || P < 1 || P >= kMaxInt || H < 1 || H > kMaxHeads) return false;
  if (!page_size_ok(page_size) || (D != 64 && D != 128 && D != 256)) return false;
  if (page_stride < H * page_size * D || page_stride >= kMaxInt || page_stride % 16 != 0) return false;
  if (layer_stride < 0 || layer_stride >= ((int64_t)1 << 46) || layer_stride % 16 != 0) return false;
  const int64_t bytes = H * page_size * D;
  return L <= 1 || layer_stride >= (P - 1) * page_stride + bytes ||
         (layer_stride >= bytes && page_stride >= (L - 1) * layer_stride + bytes);
}

bool table_ok(int64_t B, int64_t W, int64_t page_size) {
  if (B < 0 || B > 65535 || W < 1) return false;
  return W <= kMaxTokens / page_size && (B == 0 || W <= kMaxTable / B);
}

bool nodes_ok(int64_t B, int64_t M) { return M >= 0 && M <= 65535 && (M == 0 || B <= kMaxRows / M); }

nvfp4::KvCache cache_of(int64_t L, int64_t P, int64_t H, int64_t page_size, int64_t D, uint8_t* k, uint8_t* v,
                        int64_t layer_stride, int64_t page_stride, int64_t B, int64_t W, const int32_t* table,
                        const int32_t* lens) {
  nvfp4::KvCache c;
  c.k = k;
  c.v = v;
  c.layer_stride = layer_stride;
  c.page_stride = page_stride;
  c.layers = (int)L;
  c.pages = (int)P;
  c.heads = (int)H;
  c.page_shift = shift_of(page_size);
  c.dim = (int)D;
  c.table = table;
  c.lens = lens;
  c.seqs = (int)B;
  c.width = (int)W;
  return c;
}

// Values from a row to the next: at least a row, and 16-byte aligned rows.
bool stride_ok(int64_t stride, int64_t row, nvfp4_dtype dt) {
  return stride >= row && stride < ((int64_t)1 << 31) && stride % (dt == NVFP4_BF16 ? 8 : 4) == 0;
}

bool attention_shape_ok(int64_t B, int64_t M, int64_t Hq, int64_t H, int64_t D, int64_t page_size, int64_t W) {
  if (H < 1 || H > kMaxHeads || Hq < 1 || Hq % H != 0 || Hq / H > kMaxGroup) return false;
  if (!page_size_ok(page_size) || (D != 64 && D != 128 && D != 256)) return false;
  return table_ok(B, W, page_size) && nodes_ok(B, M);
}

bool pool_ok(int64_t n, int64_t S, int64_t W, int64_t P, int64_t page_size) {
  return n >= 0 && n <= kMaxEntries && S >= 1 && page_size_ok(page_size) && table_ok(S, W, page_size) && P >= 1 && P < kMaxInt - 1;
}

}  // namespace

extern "C" {

nvfp4_status nvfp4_kv_append(int64_t B, int64_t M, int64_t H, int64_t D, int64_t page_size, int64_t P, int64_t W,
                             const void* k, const void* v, nvfp4_dtype dt, int64_t k_stride, int64_t v_stride,
                             const float* k_scale, const float* v_scale, uint8_t* k_pages, uint8_t* v_pages,
                             int64_t page_stride, const int32_t* table, const int32_t* lens, const int32_t* counts,
                             void* stream) {
  if (!dtype_ok(dt)) return NVFP4_ERR_DTYPE;
  if (!pages_ok(1, P, H, page_size, D, 0, page_stride) || !table_ok(B, W, page_size) || !nodes_ok(B, M) ||
      !stride_ok(k_stride, H * D, dt) || !stride_ok(v_stride, H * D, dt) || B * M * (H * D / 16) >= kMaxInt)
    return NVFP4_ERR_SHAPE;
  if (B == 0 || M == 0) return NVFP4_OK;
  if (!k || !v || !k_scale || !v_scale || !k_pages || !v_pages || !table || !lens) return NVFP4_ERR_NULL;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(k_scale, 4) ||
      !aligned(v_scale, 4) || !aligned(table, 4) || !aligned(lens, 4) || !aligned(counts, 4))
    return NVFP4_ERR_ALIGN;
  if (k_pages == v_pages) return NVFP4_ERR_SHAPE;  // two writers of a row
  nvfp4::KvAppendArgs a;
  a.c = cache_of(1, P, H, page_size, D, k_pages, v_pages, 0, page_stride, B, W, table, lens);
  a.nodes = (int)M;
  a.x_k = k;
  a.x_v = v;
  a.k_stride = k_stride;
  a.v_stride = v_stride;
  a.bf16 = dt == NVFP4_BF16;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.counts = counts;
  return from_hip(nvfp4::launch_kv_append(a, static_cast<hipStream_t>(stream)));
}

int64_t nvfp4_kv_attention_workspace_bytes(int64_t B, int64_t M, int64_t Hq, int64_t H, int64_t D, int64_t page_size,
                                           int64_t W, nvfp4_dtype dt) {
  if (!dtype_ok(dt) || !attention_shape_ok(B, M, Hq, H, D, page_size, W) || B == 0 || M == 0) return 0;
  nvfp4::KvAttentionArgs a = {};
  a.c = cache_of(1, 1, H, page_size, D, nullptr, nullptr, 0, 0, B, W, nullptr, nullptr);
  a.nodes = (int)M;
  a.group = (int)(Hq / H);
  a.bf16 = dt == NVFP4_BF16;
  return nvfp4::kv_attention_supported(a) ? nvfp4::kv_attention_workspace_bytes(a) : 0;
}

nvfp4_status nvfp4_kv_attention(int64_t B, int64_t M, int64_t Hq, int64_t H, int64_t D, int64_t page_size, int64_t P,
                                int64_t W, const void* q, nvfp4_dtype dt, int64_t q_stride, float sm_scale,
                                const float* k_scale, const float* v_scale, const uint8_t* k_pages,
                                const uint8_t* v_pages, int64_t page_stride, const int32_t* table,
                                const int32_t* lens, const int32_t* parent, const int32_t* counts, void* out,
                                float* lse, void* workspace, int64_t workspace_bytes, void* stream) {
  if (!dtype_ok(dt)) return NVFP4_ERR_DTYPE;
  if (!attention_shape_ok(B, M, Hq, H, D, page_size, W) || !pages_ok(1, P, H, page_size, D, 0, page_stride) ||
      !stride_ok(q_stride, Hq * D, dt) || workspace_bytes < 0 || (parent && M > 64) ||
      !(sm_scale > -__builtin_inff() && sm_scale < __builtin_inff()))
    return NVFP4_ERR_SHAPE;
  if (B == 0 || M == 0) return NVFP4_OK;
  if (!q || !k_scale || !v_scale || !k_pages || !v_pages || !table || !lens || !out ||
      (workspace_bytes > 0 && !workspace))
    return NVFP4_ERR_NULL;
  if (!aligned(q, 16) || !aligned(out, 16) || !aligned(k_pages, 16) || !aligned(v_pages, 16) ||
      !aligned(workspace, 16) || !aligned(k_scale, 4) || !aligned(v_scale, 4) || !aligned(table, 4) ||
      !aligned(lens, 4) || !aligned(parent, 4) || !aligned(counts, 4) || !aligned(lse, 4))
    return NVFP4_ERR_ALIGN;
  nvfp4::KvAttentionArgs a = {};
  a.c = cache_of(1, P, H, page_size, D, const_cast<uint8_t*>(k_pages), const_cast<uint8_t*>(v_pages), 0, page_stride,
                 B, W, table, lens);
  a.nodes = (int)M;
  a.group = (int)(Hq / H);
  a.q = q;
  a.q_stride = q_stride;
  a.bf16 = dt == NVFP4_BF16;
  a.sm_scale = sm_scale;
  a.k_scale = k_scale;
  a.v_scale = v_scale;
  a.parent = parent;
  a.counts = counts;
  a.out = out;
  a.lse = lse;
  a.workspace = workspace;
  a.workspace_bytes = workspace_bytes;
  if (!nvfp4::kv_attention_supported(a)) return NVFP4_ERR_SHAPE;
  // several workgroups read a row of q that one of them writes
  const uintptr_t size = a.bf16 ? 2 : 4, q0 = (uintptr_t)q, o0 = (uintptr_t)out;
  const uintptr_t q1 = q0 + ((B * M - 1) * q_stride + Hq * D) * size, o1 = o0 + B * M * Hq * D * size;
  if (q0 < o1 && o0 < q1) return NVFP4_ERR_SHAPE;
  return from_hip(nvfp4::launch_kv_attention(a, static_cast<hipStream_t>(stream)));
}

nvfp4_status nvfp4_kv_compact(int64_t L, int64_t B, int64_t M, int64_t H, int64_t D, int64_t page_size, int64_t P,
                              int64_t W, uint8_t* k_pages, uint8_t* v_pages, int64_t layer_stride,
                              int64_t page_stride, const int32_t* table, const int32_t* lens, const int32_t* result,
                              int32_t* new_lens, void* stream) {
  if (!pages_ok(L, P, H, page_size, D, layer_stride, page_stride) || L < 1 || !table_ok(B, W, page_size) || M < 1 ||
      M > 64 || B * L * H >= kMaxInt / 128)
    return NVFP4_ERR_SHAPE;
  if (B == 0) return NVFP4_OK;
  if (!k_pages || !v_pages || !table || !lens || !result || !new_lens) return NVFP4_ERR_NULL;
  if (!aligned(k_pages, 16) || !aligned(v_pages, 16) || !aligned(table, 4) || !aligned(lens, 4) ||
      !aligned(result, 4) || !aligned(new_lens, 4))
    return NVFP4_ERR_ALIGN;
  if (lens < new_lens + B && new_lens < lens + B) return NVFP4_ERR_SHAPE;  // every workgroup reads lens
  if (k_pages == v_pages) return NVFP4_ERR_SHAPE;  // two waves would move a row
  nvfp4::KvCompactArgs a;
  a.c = cache_of(L, P, H, page_size, D, k_pages, v_pages, layer_stride, page_stride, B, W, table, lens);
  a.nodes = (int)M;
  a.result = result;
  a.new_lens = new_lens;
  return from_hip(nvfp4::launch_kv_compact(a, static_cast<hipStream_t>(stream)));
}

nvfp4_status nvfp4_kv_resize(int64_t n, int64_t S, int64_t W, int64_t P, int64_t page_size, int32_t* table,
                             int32_t* held, int32_t* refs, int32_t* free_list, const int32_t* seqs,
                             const int32_t* tokens, int32_t* shortage, void* stream) {
  if (!pool_ok(n, S, W, P, page_size)) return NVFP4_ERR_SHAPE;
  if (!table || !held || !refs || !free_list || !shortage || (n > 0 && (!seqs || !tokens))) return NVFP4_ERR_NULL;
  if (!aligned(table, 4) || !aligned(held, 4) || !aligned(refs, 4) || !aligned(free_list, 4) ||
      !aligned(shortage, 4) || !aligned(seqs, 4) || !aligned(tokens, 4))
    return NVFP4_ERR_ALIGN;
  nvfp4::KvPoolArgs a = {};
  a.n = (int)n;
  a.seqs = (int)S;
  a.width = (int)W;
  a.pages = (int)P;
  a.page_shift = shift_of(page_size);
  a.table = table;
  a.held = held;
  a.refs = refs;
  a.free_list = free_list;
  a.shortage = shortage;
  a.dst = seqs;
  a.tokens = tokens;
  return from_hip(nvfp4::launch_kv_resize(a, static_cast<hipStream_t>(stream)));
}

nvfp4_status nvfp4_kv_fork(int64_t n, int64_t S, int64_t W, int64_t P, int64_t page_size, int32_t* table,
                           int32_t* held, int32_t* refs, int32_t* free_list, const int32_t* src, const int32_t* dst,
                           const int32_t* tokens, int32_t* shortage, int32_t* moves, int64_t L, int64_t H, int64_t D,
                           uint8_t* k_pages, uint8_t* v_pages, int64_t layer_stride, int64_t page_stride,
                           void* stream) {
  if (!pool_ok(n, S, W, P, page_size) || !pages_ok(L, P, H, page_size, D, layer_stride, page_stride))
    return NVFP4_ERR_SHAPE;
  if (!table || !held || !refs || !free_list || !shortage || (n > 0 && (!src || !dst || !tokens || !moves)) ||
      (n > 0 && L > 0 && (!k_pages || !v_pages)))
    return NVFP4_ERR_NULL;
  if (!aligned(table, 4) || !aligned(held, 4) || !aligned(refs, 4) || !aligned(free_list, 4) ||
      !aligned(shortage, 4) || !aligned(src, 4) || !aligned(dst, 4) || !aligned(tokens, 4) || !aligned(moves, 4) ||
      !aligned(k_pages, 16) || !aligned(v_pages, 16))
    return NVFP4_ERR_ALIGN;
  nvfp4::KvPoolArgs a = {};
  a.n = (int)n;
  a.seqs = (int)S;
  a.width = (int)W;
  a.pages = (int)P;
  a.page_shift = shift_of(page_size);
  a.table = table;
  a.held = held;
  a.refs = refs;
  a.free_list = free_list;
  a.shortage = shortage;
  a.src = src;
  a.dst = dst;
  a.tokens = tokens;
  a.moves = moves;
  const nvfp4::KvCache c = cache_of(L, P, H, page_size, D, k_pages, v_pages, layer_stride, page_stride, S, W, table,
                                    nullptr);
  return from_hip(nvfp4::launch_kv_fork(a, c, static_cast<hipStream_t>(stream)));
}

}  // extern "C"
