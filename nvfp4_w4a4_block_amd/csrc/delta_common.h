// Device-side helpers of the gated delta rule's kernels.
#pragma once

#include "device_common.h"
#include "hybrid_launch.h"

namespace nvfp4 {

// Chains block by block, given their workspace (delta_chunk.hip).
int64_t delta_chunk_workspace_bytes(const DeltaArgs& a);
void launch_delta_chunks(const DeltaArgs& a, hipStream_t stream);

// Trees (with parents) and chains of one block (delta_single.hip).
constexpr int kChunk = 64;  // tokens of a block
void launch_delta_block(const DeltaArgs& a, hipStream_t stream);

// Four values of a row of q, k or v from value `at` on, at a multiple of four.
template <bool BF16>
__device__ __forceinline__ f4_t load4(const void* rows, int64_t at) {
  if constexpr (BF16) {
    const u2_t w = *reinterpret_cast<const u2_t*>(static_cast<const uint16_t*>(rows) + at);
    return f4_t{__uint_as_float(w.x << 16), __uint_as_float(w.x & 0xFFFF0000u), __uint_as_float(w.y << 16),
                __uint_as_float(w.y & 0xFFFF0000u)};
  } else {
    return *reinterpret_cast<const f4_t*>(static_cast<const float*>(rows) + at);
  }
}

// One value to out, rounded to nearest even; NaN stays NaN.
template <bool BF16>
__device__ __forceinline__ void store1(void* out, int64_t at, float x) {
  if constexpr (BF16) static_cast<__bf16*>(out)[at] = (__bf16)x;
  else static_cast<float*>(out)[at] = x;
}

// The wave's own LDS stores before its loads: no other wave has part in them.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

__device__ __forceinline__ f4_t scale4(f4_t x, int e) {
  return f4_t{__builtin_amdgcn_ldexpf(x[0], e), __builtin_amdgcn_ldexpf(x[1], e), __builtin_amdgcn_ldexpf(x[2], e),
              __builtin_amdgcn_ldexpf(x[3], e)};
}

__device__ __forceinline__ float max4(float m, f4_t x) {
  m = fmaxf(fmaxf(m, fabsf(x[0])), fabsf(x[1]));
  return fmaxf(fmaxf(m, fabsf(x[2])), fabsf(x[3]));
}

// floor(log2 x) of x > 0; 0 of 0.
__device__ __forceinline__ int exponent_of(float x) {
  return x > 0.0f ? (int)((__float_as_uint(x) >> 23) & 255) - 127 : 0;
}

__device__ __forceinline__ float max_of_wave(float x) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) x = fmaxf(x, __shfl_xor(x, off));
  return x;
}

__device__ __forceinline__ float sum_of_wave(float x) {
#pragma unroll
  for (int off = 32; off > 0; off >>= 1) x += __shfl_xor(x, off);
  return x;
}

// Sum over the four 16-lane groups of a wave, in all of them.
__device__ __forceinline__ float sum_of_groups(float x) {
  x += __shfl_xor(x, 16);
  return x + __shfl_xor(x, 32);
}

__device__ __forceinline__ bool delta_used(int src, int slots) { return src >= -1 && src < slots; }

// Tokens of a sequence in use.
__device__ __forceinline__ int delta_count(const int32_t* counts, int nodes, int b) {
  const int n = counts ? counts[b] : nodes;
  return n < 0 ? 0 : n < nodes ? n : nodes;
}

// The slot that sequence b's state goes to, -1: none.  It must be in range, the
// src of no other sequence in use and the dst of no earlier one.  Every lane of
// the wave calls it.
__device__ __forceinline__ int delta_dst(const int32_t* src, const int32_t* dst, int seqs, int slots, int b) {
  const int to = dst[b];
  if (to < 0 || to >= slots) return -1;
  bool taken = false;
  for (int i = threadIdx.x & 63; i < seqs; i += 64) {
    const int s = src[i];
    taken |= i != b && delta_used(s, slots) && (s == to || (i < b && dst[i] == to));
  }
  return __any(taken) ? -1 : to;
}

// A wave's share of a state: 16 * COLS of its dv rows, all DK of their values.
// Lane j + 16 g holds values 16 t + 4 g .. + 3 of row 16 c + j, which is also how
// a 16x16 matrix product leaves its result (row index 16 t + 4 g + e, column j).
template <int DK, int COLS>
struct StateTile {
  f4_t s[COLS][DK / 16];
};

template <int DK, int COLS>
__device__ __forceinline__ void load_state(const float* state, StateTile<DK, COLS>& x) {
  const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
#pragma unroll
  for (int c = 0; c < COLS; ++c)
#pragma unroll
    for (int t = 0; t < DK / 16; ++t)
      x.s[c][t] = *reinterpret_cast<const f4_t*>(state + (16 * c + j) * DK + 16 * t + 4 * g);
}

template <int DK, int COLS>
__device__ __forceinline__ void store_state(float* state, const StateTile<DK, COLS>& x) {
  const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
#pragma unroll
  for (int c = 0; c < COLS; ++c)
#pragma unroll
    for (int t = 0; t < DK / 16; ++t)
      *reinterpret_cast<f4_t*>(state + (16 * c + j) * DK + 16 * t + 4 * g) = x.s[c][t];
}

template <int DK, int COLS>
__device__ __forceinline__ void zero_state(StateTile<DK, COLS>& x) {
#pragma unroll
  for (int c = 0; c < COLS; ++c)
#pragma unroll
    for (int t = 0; t < DK / 16; ++t) x.s[c][t] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
}

}  // namespace nvfp4
