// Log probabilities of given tokens under rows of logits, entropies and the most
// probable tokens.
//
// The logits are those of the LM head, which the page "TensorRT Edge-LLM Completes
// the MLPerf Edge Agentic Benchmark 6.4x Faster on Jetson AGX Thor" keeps in NVFP4
// as well (section "Using NVFP4 quantization to accelerate Qwen3.6-27B inference").
//
// Mathematics.  Over a part of a row: m its maximum, a = sum e^(z - m) - 1 (the
// maximum's own 1 left out, so that a row that is sure of one token keeps the
// rest's digits), t = sum e^(z - m) (z - m).  Two parts join as m = max, with f =
// e^(m2 - m1) of the lower one: a = a1 + f (1 + a2), t = t1 + f (t2 + (1 + a2) (m2 -
// m1)).  An empty part has a = -1; a NaN or +infinity makes a NaN, which joins keep.
// Then log sum e^z = m + log1p(a), entropy = log1p(a) - t / (1 + a).
//
// Order.  A logit's key is its bits as an ordered number above the complement of
// its column, so keys are unique and descend by value, then column.  What is not in
// the first `top` of a part is not in the row's.
#include "device_common.h"
#include "hybrid_launch.h"

namespace nvfp4 {
namespace {

constexpr int kWaves = 4;
constexpr int kBatch = 16;  // logits of a lane at a time
constexpr int kPart = 64 * kWaves * kBatch;

struct Stat {
  float m, a, t;
};

__device__ __forceinline__ Stat join(const Stat& x, const Stat& y) {
  const bool first = x.m >= y.m;
  const Stat hi = first ? x : y, lo = first ? y : x;
  if (lo.a == -1.0f) return hi;  // nothing there
  const float d = lo.m - hi.m, f = expf(d), w = 1.0f + lo.a;
  if (f == 0.0f && w == w) return hi;  // d may be so low that a product with it overflows
  return {hi.m, hi.a + f * w, hi.t + f * (lo.t + w * d)};
}

__device__ __forceinline__ uint32_t ordered(float v) {
  const uint32_t b = __float_as_uint(v);
  return (b & 0x80000000u) ? ~b : (b | 0x80000000u);
}

__device__ __forceinline__ float from_ordered(uint32_t o) {
  return __uint_as_float((o & 0x80000000u) ? (o & 0x7FFFFFFFu) : ~o);
}

// Part of a row: its numbers and its first keys.
struct Plan {
  int parts;       // of a row
  Stat* stats;     // [rows][parts]
  uint64_t* keys;  // [rows][parts][top], 0 behind the last
};

// The first `top` of the keys that the workgroup's threads hold, into best in
// descending order: one after the other.
template <int N>
__device__ __forceinline__ void select(uint64_t (&key)[N], int top, uint64_t* best, uint64_t* shared) {
  for (int i = 0; i < top; ++i) {
    uint64_t k = 0;
#pragma unroll
    for (int e = 0; e < N; ++e) k = key[e] > k ? key[e] : k;
    for (int off = 32; off > 0; off >>= 1) {
      const uint64_t o = __shfl_xor(k, off);
      k = o > k ? o : k;
    }
    __syncthreads();
    if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = k;
    __syncthreads();
    k = 0;
    for (int w = 0; w < kWaves; ++w) k = shared[w] > k ? shared[w] : k;
#pragma unroll
    for (int e = 0; e < N; ++e) key[e] = key[e] == k ? 0 : key[e];
    if (threadIdx.x == 0) best[i] = k;
  }
}

__device__ __forceinline__ Stat join_all(Stat s, Stat* shared) {
  for (int off = 32; off > 0; off >>= 1) s = join(s, Stat{__shfl_xor(s.m, off), __shfl_xor(s.a, off), __shfl_xor(s.t, off)});
  if ((threadIdx.x & 63) == 0) shared[threadIdx.x >> 6] = s;
  __syncthreads();
  s = shared[0];
  for (int w = 1; w < kWaves; ++w) s = join(s, shared[w]);
  return s;
}

// grid (parts, rows).
template <bool BF16>
__global__ __launch_bounds__(64 * kWaves) void logprob_part_kernel(LogprobArgs a, Plan p) {
  __shared__ Stat stats[kWaves];
  __shared__ uint64_t tops[kWaves];
  const int64_t row = blockIdx.y;
  uint64_t key[kBatch];
  Stat s = {-__builtin_inff(), -1.0f, 0.0f};
#pragma unroll
  for (int e = 0; e < kBatch; ++e) {
    const int n = blockIdx.x * kPart + e * 64 * kWaves + threadIdx.x;
    key[e] = 0;
    if (n < a.vocab) {
      float z;
      if constexpr (BF16) z = __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.logits)[row * a.stride + n] << 16);
      else z = static_cast<const float*>(a.logits)[row * a.stride + n];
      key[e] = ((uint64_t)ordered(z) << 32) | (0xFFFFFFFFu - (uint32_t)n);
      if (!(z < __builtin_inff())) s.a = __builtin_nanf("");
      else if (z > -__builtin_inff()) s = join(s, Stat{z, 0.0f, 0.0f});
    }
  }
  s = join_all(s, stats);
  const int64_t at = row * p.parts + blockIdx.x;
  if (threadIdx.x == 0) p.stats[at] = s;
  select(key, a.top, p.keys + at * a.top, tops);
}

// grid (rows).
template <bool BF16>
__global__ __launch_bounds__(64 * kWaves) void logprob_row_kernel(LogprobArgs a, Plan p) {
  __shared__ Stat stats[kWaves];
  __shared__ uint64_t tops[kWaves];
  __shared__ uint64_t best[64];
  const int64_t row = blockIdx.x;
  Stat s = {-__builtin_inff(), -1.0f, 0.0f};
  for (int i = threadIdx.x; i < p.parts; i += 64 * kWaves) s = join(s, p.stats[row * p.parts + i]);
  s = join_all(s, stats);
  const bool none = !(s.m > -__builtin_inff()) || s.a != s.a;
  const float nan = __builtin_nanf(""), l = log1pf(s.a);
  if (threadIdx.x == 0) {
    const int token = a.tokens[row];
    float z = nan;
    if (token >= 0 && token < a.vocab) {
      if constexpr (BF16) z = __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.logits)[row * a.stride + token] << 16);
      else z = static_cast<const float*>(a.logits)[row * a.stride + token];
    }
    a.logprobs[row] = none ? nan : (z - s.m) - l;
    a.entropy[row] = none ? nan : l - s.t / (1.0f + s.a);
  }
  if (a.top == 0) return;
  for (int i = threadIdx.x; i < 64; i += 64 * kWaves) best[i] = 0;
  const int n = p.parts * a.top;
  for (int i0 = 0; i0 < n; i0 += 8 * 64 * kWaves) {
    uint64_t key[9];
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const int i = i0 + e * 64 * kWaves + threadIdx.x;
      key[e] = i < n ? p.keys[row * n + i] : 0;
    }
    __syncthreads();
    key[8] = threadIdx.x < 64 ? best[threadIdx.x] : 0;
    __syncthreads();
    select(key, a.top, best, tops);
  }
  __syncthreads();
  if ((int)threadIdx.x < a.top) {
    const uint64_t k = best[threadIdx.x];
    const float z = from_ordered((uint32_t)(k >> 32));
    a.top_logprobs[row * a.top + threadIdx.x] = none ? nan : (z - s.m) - l;
    a.top_tokens[row * a.top + threadIdx.x] = none ? -1 : (int32_t)(0xFFFFFFFFu - (uint32_t)k);
  }
}

int parts_of(const LogprobArgs& a) { return (a.vocab + kPart - 1) / kPart; }

}  // namespace

int64_t token_logprobs_workspace_bytes(const LogprobArgs& a) {
  const int64_t n = (int64_t)a.rows * parts_of(a);
  return (n * (int64_t)sizeof(Stat) + 15) / 16 * 16 + n * a.top * 8;
}

hipError_t launch_token_logprobs(const LogprobArgs& a, hipStream_t stream) {
  Plan p;
  p.parts = parts_of(a);
  p.stats = static_cast<Stat*>(a.workspace);
  p.keys = reinterpret_cast<uint64_t*>(static_cast<char*>(a.workspace) +
                                       ((int64_t)a.rows * p.parts * (int64_t)sizeof(Stat) + 15) / 16 * 16);
  const dim3 grid(p.parts, a.rows);
  if (a.bf16) {
    logprob_part_kernel<true><<<grid, 64 * kWaves, 0, stream>>>(a, p);
    logprob_row_kernel<true><<<a.rows, 64 * kWaves, 0, stream>>>(a, p);
  } else {
    logprob_part_kernel<false><<<grid, 64 * kWaves, 0, stream>>>(a, p);
    logprob_row_kernel<false><<<a.rows, 64 * kWaves, 0, stream>>>(a, p);
  }
  return hipGetLastError();
}

}  // namespace nvfp4
