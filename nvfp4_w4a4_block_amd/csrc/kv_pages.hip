// Writing and compacting the paged FP8 KV cache.
//
// The page "TensorRT Edge-LLM Completes the MLPerf Edge Agentic Benchmark
// 6.4x Faster on Jetson AGX Thor" keeps the KV cache in FP8 (section "Using
// NVFP4 quantization to accelerate Qwen3.6-27B inference") and verifies a tree
// of drafted tokens in one pass (section "Using tree-based multi-token
// prediction to accelerate LLM inference").  A step writes the keys and values
// of every node behind the committed tokens (kv_append_kernel), and once the
// path is accepted moves the path's tokens to the front (kv_compact_kernel).
#pragma clang fp contract(off)
#include "device_common.h"
#include "kv_codec.h"
#include "kv_launch.h"

namespace nvfp4 {
namespace {

constexpr int kMaxTokens = 1 << 30;  // no table covers more

// Address of a token's row of one head, or NULL when the position lies outside
// the table or its page id outside the cache.
__device__ __forceinline__ uint8_t* token_row(uint8_t* base, const KvCache& c, int seq, int head, int pos) {
  const int at = pos >> c.page_shift;
  if (pos < 0 || at >= c.width) return nullptr;
  const int page = c.table[(int64_t)seq * c.width + at];
  if (page < 0 || page >= c.pages) return nullptr;
  const int slot = pos & ((1 << c.page_shift) - 1);
  return base + page * c.page_stride + (((int64_t)head << c.page_shift) + slot) * c.dim;
}

// q = E4M3(x * (1 / s)) of every node's keys and values, 16 elements per
// thread (one 16-byte store; a row never crosses a page), written to the node's
// slot.  Each element is read and written once: bound by memory for prompts (8188
// fp32 rows of 8 x 128, K and V, 84 MB: 14.3 us, 5.9 TB/s, part of it from the
// Infinity Cache), by the launch for a tree (16 bf16 nodes: 3.2 us).
template <bool BF16>
__global__ __launch_bounds__(256) void kv_append_kernel(KvAppendArgs a, uint32_t chunks) {
  const KvCache& c = a.c;
  const uint32_t per_row = (uint32_t)(c.heads * c.dim) >> 4;
  const uint32_t i = blockIdx.x * 256u + threadIdx.x;
  if (i >= chunks) return;
  const bool is_v = blockIdx.y != 0;
  const uint32_t row = i / per_row, chunk = i - row * per_row;
  const int b = (int)(row / (uint32_t)a.nodes), v = (int)(row - (uint32_t)b * a.nodes);
  const int len = c.lens[b];
  const int count = a.counts ? a.counts[b] : a.nodes;
  if (len < 0 || len > kMaxTokens || v >= count) return;
  const int e = (int)chunk << 4, head = e >> (31 - __clz(c.dim)), d = e & (c.dim - 1);
  uint8_t* to = token_row(is_v ? c.v : c.k, c, b, head, len + v);
  if (!to) return;
  const float s = is_v ? *a.v_scale : *a.k_scale;
  const float inv = s == 0.0f ? 0.0f : 1.0f / s;
  const int64_t from = (int64_t)row * (is_v ? a.v_stride : a.k_stride) + e;
  float x[16];
  if constexpr (BF16) {
    const u4_t* p = reinterpret_cast<const u4_t*>(static_cast<const uint16_t*>(is_v ? a.x_v : a.x_k) + from);
    const u4_t lo = p[0], hi = p[1];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[2 * j] = __uint_as_float(lo[j] << 16);
      x[2 * j + 1] = __uint_as_float(lo[j] & 0xFFFF0000u);
      x[8 + 2 * j] = __uint_as_float(hi[j] << 16);
      x[9 + 2 * j] = __uint_as_float(hi[j] & 0xFFFF0000u);
    }
  } else {
    const f4_t* p = reinterpret_cast<const f4_t*>(static_cast<const float*>(is_v ? a.x_v : a.x_k) + from);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const f4_t w = p[j];
#pragma unroll
      for (int u = 0; u < 4; ++u) x[4 * j + u] = w[u];
    }
  }
  u4_t w;
#pragma unroll
  for (int j = 0; j < 4; ++j)
    w[j] = e4m3x4(x[4 * j] * inv, x[4 * j + 1] * inv, x[4 * j + 2] * inv, x[4 * j + 3] * inv);
  *reinterpret_cast<u4_t*>(to + d) = w;
}

// One wave moves the accepted path's rows of one (sequence, layer, K or V,
// head): row len + path[i] -> row len + 1 + i, 64 chunks of 16 bytes per round.
// The path ascends, so path[i] >= i + 1: a round's destinations lie before
// every later round's sources, and within a round the wave has loaded all its
// chunks before it stores one.  Bound by its chain of loads (length, path, two
// table entries, row) and the launch: one tree of 16 in 16 layers 3.2 us, 32 trees
// of 33 in 24 layers of 4 x 256 9.3 us (about 21 MB read and written).
__global__ __launch_bounds__(256) void kv_compact_kernel(KvCompactArgs a, uint32_t waves) {
  const KvCache& c = a.c;
  const uint32_t w = blockIdx.x * 4u + (threadIdx.x >> 6);
  if (w >= waves) return;
  const int lane = threadIdx.x & 63;
  const uint32_t heads2 = 2u * c.heads, per_seq = heads2 * c.layers;
  const int b = (int)(w / per_seq);
  const uint32_t x = w - (uint32_t)b * per_seq;
  const int layer = (int)(x / heads2), hv = (int)(x - (uint32_t)layer * heads2), head = hv >> 1;
  const int32_t* res = a.result + (int64_t)b * (3 + a.nodes);
  const int len = c.lens[b];
  int moves = res[1];
  moves = moves < 0 ? 0 : moves < a.nodes ? moves : a.nodes - 1;
  if (x == 0 && lane == 0) a.new_lens[b] = len < 0 || len > kMaxTokens ? len : len + 1 + moves;
  if (len < 0 || len > kMaxTokens) return;
  uint8_t* base = ((hv & 1) ? c.v : c.k) + layer * c.layer_stride;
  const int per = c.dim >> 4;  // 16-byte chunks of a row
  for (int r = 0; r < moves * per; r += 64) {
    const int i = (r + lane) / per, part = (r + lane) - i * per;
    const uint8_t* from = nullptr;
    uint8_t* to = nullptr;
    if (i < moves) {
      const int node = res[3 + i];
      if (node >= 0 && node < a.nodes && node != i + 1) {
        from = token_row(base, c, b, head, len + node);
        to = token_row(base, c, b, head, len + 1 + i);
      }
    }
    if (from && to) {
      const u4_t d = reinterpret_cast<const u4_t*>(from)[part];
      reinterpret_cast<u4_t*>(to)[part] = d;
    }
  }
}

}  // namespace

hipError_t launch_kv_append(const KvAppendArgs& a, hipStream_t stream) {
  const uint32_t chunks = (uint32_t)a.c.seqs * a.nodes * ((uint32_t)(a.c.heads * a.c.dim) >> 4);
  const dim3 grid((chunks + 255) / 256, 2);
  if (a.bf16) kv_append_kernel<true><<<grid, 256, 0, stream>>>(a, chunks);
  else kv_append_kernel<false><<<grid, 256, 0, stream>>>(a, chunks);
  return hipGetLastError();
}

hipError_t launch_kv_compact(const KvCompactArgs& a, hipStream_t stream) {
  const uint32_t waves = (uint32_t)a.c.seqs * a.c.layers * a.c.heads * 2u;
  kv_compact_kernel<<<(waves + 3) / 4, 256, 0, stream>>>(a, waves);
  return hipGetLastError();
}

}  // namespace nvfp4
