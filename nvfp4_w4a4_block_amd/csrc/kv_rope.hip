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
// left goes to sine and cosine in 64 bits, too (14 multiply-adds).  So do the turns:
// fp32 ones move an E4M3 code where a value is next to the middle of two, about one
// in a million, and the time is memory's either way.
//
// Bounds.  Every value is read and written once: memory for prompts, the launch
// for a tree.  A workgroup takes a token, works out its sines and cosines once, for
// all heads, in LDS, and then gives each thread 16 values of a head at a time: 8
// pairs, or 16 values that do not turn.  Four prompts of 2,047 tokens, 16 heads of
// queries and 2 x 8 of keys and values of 128, fp32: 43.6 us, 5.0 TB/s of 218 MB; in bf16,
// half the bytes for the same turns, 24.2, 4.8 TB/s of 117 MB.  A tree of 16 bf16 nodes:
// 4.9 us.
#include "hybrid_launch.h"
#include "kv_codec.h"
#include "kv_tree.h"

namespace nvfp4 {
namespace {

constexpr int kMaxTokens = 1 << 30;  // no table covers more

template <bool BF16>
__device__ __forceinline__ void load8(const void* rows, int64_t at, double (&x)[8]) {
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
__device__ __forceinline__ void store8(void* rows, int64_t at, const double (&x)[8]) {
  if constexpr (BF16) {
    typedef __bf16 bf8_t __attribute__((ext_vector_type(8)));
    bf8_t w;
#pragma unroll
    for (int i = 0; i < 8; ++i) w[i] = (__bf16)(float)x[i];
    *reinterpret_cast<bf8_t*>(static_cast<__bf16*>(rows) + at) = w;
  } else {
    f4_t lo, hi;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      lo[i] = (float)x[i];
      hi[i] = (float)x[4 + i];
    }
    f4_t* p = reinterpret_cast<f4_t*>(static_cast<float*>(rows) + at);
    p[0] = lo;
    p[1] = hi;
  }
}

// x in fp32's 24 bits, the last of them set where anything is cut off: rounding that
// to fewer bits is rounding x.
__device__ __forceinline__ float cut(double x) {
  uint64_t b = __double_as_longlong(x);
  const uint32_t lo = (uint32_t)b;
  b = (b & ~(uint64_t)0xFFFFFFFF) | (lo & 0xE0000000u) | ((lo & 0x1FFFFFFFu) ? 0x20000000u : 0u);
  return (float)__longlong_as_double(b);
}

// Eight values to their E4M3 bytes.  Values that were turned are rounded once; those
// that were not, as an append without turning rounds them: value / scale to fp32 first.
__device__ __forceinline__ u2_t codes8(const double (&x)[8], double inv, bool turned) {
  float y[8];
#pragma unroll
  for (int e = 0; e < 8; ++e) {
    const double z = x[e] * inv;
    y[e] = turned ? cut(z) : (float)z;
  }
  return u2_t{e4m3x4(y[0], y[1], y[2], y[3]), e4m3x4(y[4], y[5], y[6], y[7])};
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

// grid (nodes, seqs).
template <bool BF16, bool INTERLEAVED>
__global__ __launch_bounds__(256) void kv_append_rope_kernel(KvRopeArgs a) {
  __shared__ double cs[2][128];  // cosine, sine of each pair
  __shared__ int64_t row;       // byte offset of the token's row of head 0, -1: none
  __shared__ int depth;         // of the tree's node
  const KvAppendArgs& ap = a.append;
  const KvCache& c = ap.c;
  const int b = blockIdx.y, t = blockIdx.x, half = a.rotary >> 1;
  const int len = c.lens[b];
  int count = ap.counts ? ap.counts[b] : ap.nodes;
  count = count < ap.nodes ? count : ap.nodes;
  if (len < 0 || len > kMaxTokens) count = 0;
  const bool live = t < count;
  if (a.parent && threadIdx.x < 64) {
    const int lane = threadIdx.x;
    const uint64_t line = ancestors_of_wave(lane < ap.nodes ? a.parent[(int64_t)b * ap.nodes + lane] : -1);
    if (lane == t) depth = __popcll(line) - 1;
  }
  if (threadIdx.x == 64 && live) {
    const int pos = len + t, at = pos >> c.page_shift;
    int64_t to = -1;
    if (at < c.width) {
      const int page = c.table[(int64_t)b * c.width + at];
      if (page >= 0 && page < c.pages)
        to = page * c.page_stride + (int64_t)(pos & ((1 << c.page_shift) - 1)) * c.dim;
    }
    row = to;
  }
  if (a.parent) __syncthreads();
  if (live && (int)threadIdx.x < half) {
    const int j = threadIdx.x;
    const int64_t pos = (int64_t)len + (a.parent ? depth : t);
    const double turns = (double)pos * (a.inv_freq[j] * 0.15915494309189533577);
    double co, si;
    turn(turns - __builtin_rint(turns), co, si);
    cs[0][j] = co * a.rope_scale;
    cs[1][j] = si * a.rope_scale;
  }
  __syncthreads();
  const int per = c.dim >> 4, heads = a.q_heads + 2 * c.heads, turning = a.rotary >> 4;
  const float ks = *ap.k_scale, vs = *ap.v_scale;
  const float k_inv = ks == 0.0f ? 0.0f : 1.0f / ks, v_inv = vs == 0.0f ? 0.0f : 1.0f / vs;
  const int64_t from = (int64_t)b * ap.nodes + t;
  for (int i = threadIdx.x; i < heads * per; i += 256) {
    const int head = i / per, part = i - head * per;
    const bool is_q = head < a.q_heads, is_v = head >= a.q_heads + c.heads;
    const int h = is_q ? head : is_v ? head - a.q_heads - c.heads : head - a.q_heads;
    const bool turns = part < turning && !is_v;
    // where the two eights of values stand in the head
    const int d0 = turns && !INTERLEAVED ? 8 * part : 16 * part;
    const int d1 = turns && !INTERLEAVED ? 8 * part + half : 16 * part + 8;
    const int64_t out = (from * a.q_heads + h) * c.dim;
    double x[8], y[8];
    if (!live) {
      if (!is_q) continue;
#pragma unroll
      for (int e = 0; e < 8; ++e) x[e] = 0.0;
      store8<BF16>(a.q_out, out + d0, x);
      store8<BF16>(a.q_out, out + d1, x);
      continue;
    }
    const void* rows = is_q ? a.q : is_v ? ap.x_v : ap.x_k;
    const int64_t at = from * (is_q ? a.q_stride : is_v ? ap.v_stride : ap.k_stride) + (int64_t)h * c.dim;
    load8<BF16>(rows, at + d0, x);
    load8<BF16>(rows, at + d1, y);
    if (turns) {
      double co[8], si[8];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        co[e] = cs[0][8 * part + e];
        si[e] = cs[1][8 * part + e];
      }
      if constexpr (INTERLEAVED) {
        // pairs (x0, x1) .. (y6, y7)
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const double p0 = x[2 * e], p1 = x[2 * e + 1], r0 = y[2 * e], r1 = y[2 * e + 1];
          x[2 * e] = p0 * co[e] - p1 * si[e];
          x[2 * e + 1] = p1 * co[e] + p0 * si[e];
          y[2 * e] = r0 * co[4 + e] - r1 * si[4 + e];
          y[2 * e + 1] = r1 * co[4 + e] + r0 * si[4 + e];
        }
      } else {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          const double p = x[e], r = y[e];
          x[e] = p * co[e] - r * si[e];
          y[e] = r * co[e] + p * si[e];
        }
      }
    }
    if (is_q) {
      store8<BF16>(a.q_out, out + d0, x);
      store8<BF16>(a.q_out, out + d1, y);
    } else if (row >= 0) {
      uint8_t* to = (is_v ? c.v : c.k) + row + ((int64_t)h << c.page_shift) * c.dim;
      const double inv = is_v ? v_inv : k_inv;
      const u2_t lo = codes8(x, inv, turns), hi8 = codes8(y, inv, turns);
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
  const dim3 grid(a.append.nodes, a.append.c.seqs);
  if (a.append.bf16) {
    if (a.interleaved) kv_append_rope_kernel<true, true><<<grid, 256, 0, stream>>>(a);
    else kv_append_rope_kernel<true, false><<<grid, 256, 0, stream>>>(a);
  } else {
    if (a.interleaved) kv_append_rope_kernel<false, true><<<grid, 256, 0, stream>>>(a);
    else kv_append_rope_kernel<false, false><<<grid, 256, 0, stream>>>(a);
  }
  return hipGetLastError();
}

}  // namespace nvfp4
