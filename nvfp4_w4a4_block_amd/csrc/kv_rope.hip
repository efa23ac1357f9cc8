// Rotary positions on the way into the paged FP8 KV cache: one launch turns a
// step's queries, writes its keys turned and its values as they are.
//
// The page "TensorRT Edge-LLM Completes the MLPerf Edge Agentic Benchmark 6.4x
// Faster on Jetson AGX Thor" verifies a tree of drafted tokens in one pass
// (section "Using tree-based multi-token prediction to accelerate LLM inference"):
// its nodes at one depth share a position, while each has a place of its own in
// the cache.
//
// Mathematics.  Pair (x, y) at position p: (x c - y s, y c + x s), c and s the
// scaled cosine and sine of p * inv_freq.  The angle in turns, p * inv_freq / 2 pi,
// is a product of 64 bits whose whole part is dropped there: at position 2^30 it is
// off by 2^-24 turns at most, where 32 bits would keep nothing of it.  What is
// left goes to sine and cosine in 64 bits, too (14 multiply-adds), which are rounded
// to fp32 once, with the factor in them.
//
// Bounds.  Every value is read and written once: memory for prompts, the launch
// for a tree.  A workgroup takes the tokens of one sequence from `first` on, works
// out their sines and cosines once, for all heads, in LDS, and then gives each
// thread 16 values of a head at a time: 8 pairs, or 16 values that do not turn.
#include "hybrid_launch.h"
#include "kv_codec.h"
#include "kv_tree.h"

namespace nvfp4 {
namespace {

constexpr int kMaxTokens = 1 << 30;  // no table covers more
constexpr int kSpan = 8;             // tokens of a workgroup, at most

template <bool BF16>
__device__ __forceinline__ void load8(const void* rows, int64_t at, float (&x)[8]) {
  if constexpr (BF16) {
    const u4_t w = *reinterpret_cast<const u4_t*>(static_cast<const uint16_t*>(rows) + at);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    const f4_t* p = reinterpret_cast<const f4_t*>(static_cast<const float*>(rows) + at);
    const f4_t lo = p[0], hi = p[1];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[i] = lo[i];
      x[4 + i] = hi[i];
    }
  }
}

template <bool BF16>
__device__ __forceinline__ void store8(void* rows, int64_t at, const float (&x)[8]) {
  if constexpr (BF16) {
    typedef __bf16 bf8_t __attribute__((ext_vector_type(8)));
    bf8_t w;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = (__bf16)x[i];
    *reinterpret_cast<bf8_t*>(static_cast<__bf16*>(rows) + at) = w;
  } else {
    f4_t* p = reinterpret_cast<f4_t*>(static_cast<float*>(rows) + at);
    p[0] = f4_t{x[0], x[1], x[2], x[3]};
    p[1] = f4_t{x[4], x[5], x[6], x[7]};
  }
}

// Eight values to their E4M3 bytes.
__device__ __forceinline__ u2_t codes8(const float (&x)[8], float inv) {
  return u2_t{e4m3x4(x[0] * inv, x[1] * inv, x[2] * inv, x[3] * inv),
              e4m3x4(x[4] * inv, x[5] * inv, x[6] * inv, x[7] * inv)};
}

// Cosine and sine of x turns, |x| <= 1/2: the series of both within an eighth of a
// turn (what is left out is below 7e-12), exchanged and signed by the quarter.
__device__ __forceinline__ void turn(double x, double& c, double& s) {
  const double quarter = __builtin_rint(4.0 * x);
  const double r = (x - 0.25 * quarter) * 6.283185307179586477, z = r * r;
  double si = -1.0 / 39916800.0, co = 1.0 / 479001600.0;
  si = __builtin_fma(si, z, 1.0 / 362880.0);
  si = __builtin_fma(si, z, -1.0 / 5040.0);
  si = __builtin_fma(si, z, 1.0 / 120.0);
  si = __builtin_fma(si, z, -1.0 / 6.0);
  si = __builtin_fma(si * z, r, r);
  co = __builtin_fma(co, z, -1.0 / 3628800.0);
  co = __builtin_fma(co, z, 1.0 / 40320.0);
  co = __builtin_fma(co, z, -1.0 / 720.0);
  co = __builtin_fma(co, z, 1.0 / 24.0);
  co = __builtin_fma(co, z, -0.5);
  co = __builtin_fma(co, z, 1.0);
  const int k = (int)quarter & 3;
  const double a = (k & 1) ? si : co, b = (k & 1) ? co : si;
  c = (k == 1 || k == 2) ? -a : a;
  s = (k & 2) ? -b : b;
}

// grid (ceil(nodes / span), seqs, parts): part p of the parts takes every
// parts-th of the tokens' units of 16 values.
template <bool BF16, bool INTERLEAVED>
__global__ __launch_bounds__(256) void kv_append_rope_kernel(KvRopeArgs a, int span) {
  __shared__ float cs[kSpan][2][128];  // cosine, sine of each pair
  __shared__ int64_t row_of[kSpan];    // byte offset of the token's row of head 0, -1: none
  const KvAppendArgs& ap = a.append;
  const KvCache& c = ap.c;
  const int b = blockIdx.y, first = blockIdx.x * span, half = a.rotary >> 1;
  const int len = c.lens[b];
  int count = ap.counts ? ap.counts[b] : ap.nodes;
  count = count < ap.nodes ? count : ap.nodes;
  if (len < 0 || len > kMaxTokens) count = 0;
  const int last = first + span < ap.nodes ? first + span : ap.nodes;
  const int live = (count < last ? count : last) - first;  // tokens here, the others are no tokens
  int depth = 0;  // of node threadIdx.x, in the first wave
  __shared__ int depths[64];
  if (a.parent && threadIdx.x < 64) {
    const int lane = threadIdx.x;
    depth = __popcll(ancestors_of_wave(lane < ap.nodes ? a.parent[(int64_t)b * ap.nodes + lane] : -1)) - 1;
    depths[lane] = depth;
  }
  if ((int)threadIdx.x >= 64 && (int)threadIdx.x - 64 < live) {
    const int t = threadIdx.x - 64, pos = len + first + t, at = pos >> c.page_shift;
    int64_t row = -1;
    if (at < c.width) {
      const int page = c.table[(int64_t)b * c.width + at];
      if (page >= 0 && page < c.pages)
        row = page * c.page_stride + (int64_t)(pos & ((1 << c.page_shift) - 1)) * c.dim;
    }
    row_of[t] = row;
  }
  if (a.parent) __syncthreads();
  for (int i = threadIdx.x; i < live * half; i += 256) {
    const int t = i / half, j = i - t * half;
    const int64_t pos = (int64_t)len + (a.parent ? depths[first + t] : first + t);
    const double turns = (double)pos * (a.inv_freq[j] * 0.15915494309189533577);
    double co, si;
    turn(turns - __builtin_rint(turns), co, si);
    cs[t][0][j] = (float)(co * a.rope_scale);
    cs[t][1][j] = (float)(si * a.rope_scale);
  }
  __syncthreads();
  const int per = c.dim >> 4, heads = a.q_heads + 2 * c.heads, turning = a.rotary >> 4;
  const float ks = *ap.k_scale, vs = *ap.v_scale;
  const float k_inv = ks == 0.0f ? 0.0f : 1.0f / ks, v_inv = vs == 0.0f ? 0.0f : 1.0f / vs;
  const int units = (last - first) * heads * per;
  for (int i = blockIdx.z * 256 + threadIdx.x; i < units; i += 256 * gridDim.z) {
    const int hi = i / per, part = i - hi * per, t = hi / heads, head = hi - t * heads;
    const int64_t row = (int64_t)b * ap.nodes + first + t;
    const bool is_q = head < a.q_heads, is_v = head >= a.q_heads + c.heads;
    const int h = is_q ? head : is_v ? head - a.q_heads - c.heads : head - a.q_heads;
    const bool turns = part < turning && !is_v;
    // where the two eights of values stand in the head
    const int d0 = turns && !INTERLEAVED ? 8 * part : 16 * part;
    const int d1 = turns && !INTERLEAVED ? 8 * part + half : 16 * part + 8;
    const int64_t out = (row * a.q_heads + h) * c.dim;
    float x[8], y[8];
    if (t >= live) {
      if (!is_q) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = 0.0f;
      store8<BF16>(a.q_out, out + d0, x);
      store8<BF16>(a.q_out, out + d1, x);
      continue;
    }
    const void* rows = is_q ? a.q : is_v ? ap.x_v : ap.x_k;
    const int64_t at = row * (is_q ? a.q_stride : is_v ? ap.v_stride : ap.k_stride) + (int64_t)h * c.dim;
    load8<BF16>(rows, at + d0, x);
    load8<BF16>(rows, at + d1, y);
    if (turns) {
      float co[8], si[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        co[e] = cs[t][0][8 * part + e];
        si[e] = cs[t][1][8 * part + e];
      }
      if constexpr (INTERLEAVED) {
        // pairs (x0, x1) .. (y6, y7)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const float p0 = x[2 * e], p1 = x[2 * e + 1], r0 = y[2 * e], r1 = y[2 * e + 1];
          x[2 * e] = p0 * co[e] - p1 * si[e];
          x[2 * e + 1] = p1 * co[e] + p0 * si[e];
          y[2 * e] = r0 * co[4 + e] - r1 * si[4 + e];
          y[2 * e + 1] = r1 * co[4 + e] + r0 * si[4 + e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const float p = x[e], r = y[e];
          x[e] = p * co[e] - r * si[e];
          y[e] = r * co[e] + p * si[e];
        }
      }
    }
    if (is_q) {
      store8<BF16>(a.q_out, out + d0, x);
      store8<BF16>(a.q_out, out + d1, y);
    } else if (row_of[t] >= 0) {
      uint8_t* to = (is_v ? c.v : c.k) + row_of[t] + ((int64_t)h << c.page_shift) * c.dim;
      const float inv = is_v ? v_inv : k_inv;
      const u2_t lo = codes8(x, inv), hi8 = codes8(y, inv);
      if (d1 == d0 + 8) {
        *reinterpret_cast<u4_t*>(to + d0) = u4_t{lo.x, lo.y, hi8.x, hi8.y};
      } else {
        *reinterpret_cast<u2_t*>(to + d0) = lo;
        *reinterpret_cast<u2_t*>(to + d1) = hi8;
      }
    }
  }
}

}  // namespace

hipError_t launch_kv_append_rope(const KvRopeArgs& a, hipStream_t stream) {
  const int span = 1;
  const dim3 grid((a.append.nodes + span - 1) / span, a.append.c.seqs, 1);
  if (a.append.bf16) {
    if (a.interleaved) kv_append_rope_kernel<true, true><<<grid, 256, 0, stream>>>(a, span);
    else kv_append_rope_kernel<true, false><<<grid, 256, 0, stream>>>(a, span);
  } else {
    if (a.interleaved) kv_append_rope_kernel<false, true><<<grid, 256, 0, stream>>>(a, span);
    else kv_append_rope_kernel<false, false><<<grid, 256, 0, stream>>>(a, span);
  }
  return hipGetLastError();
}

}  // namespace nvfp4
