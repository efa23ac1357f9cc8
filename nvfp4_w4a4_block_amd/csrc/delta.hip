// Gated delta rule, token by token: decoding steps, and the accepted path of a tree put
// into the states.
//
// The model of the page "TensorRT Edge-LLM Completes the MLPerf Edge Agentic
// Benchmark 6.4x Faster on Jetson AGX Thor" is a hybrid whose recurrent states are
// kept and restored with the cached attention pages (section "Reusing KV cache
// across agent turns").
//
// Mathematics.  Per value head, S [dv][dk] in fp32: S <- e^g S, u = beta (v - S k),
// S <- S + u k^T, o = scale S q.  Rows of S are independent of each other, so a
// wave that holds some of them whole needs nothing from any other.
#include "delta_common.h"

namespace nvfp4 {
namespace {

constexpr int kWaves = 4;
constexpr int kTile = 8;  // tokens whose q and k stand in LDS

__device__ __forceinline__ float sum_of_squares(f4_t x) {
  return sum_of_wave(x[0] * x[0] + x[1] * x[1] + x[2] * x[2] + x[3] * x[3]);
}

// One row of q or k (DK values) as used, by a whole wave: normalised, times scale.
template <int DK, bool BF16>
__device__ __forceinline__ void stage_row(const void* rows, int64_t at, float eps, float scale, float* to) {
  const int lane = threadIdx.x & 63;
  f4_t x = {0.0f, 0.0f, 0.0f, 0.0f};
  if (lane < DK / 4) x = load4<BF16>(rows, at + 4 * lane);
  if (eps >= 0.0f) {
    float square = sum_of_squares(x) + eps;
    if (!(square > 0x1p-100f && square < 0x1p126f)) {
      // past what fp32's squares hold: of the row over a power of two.  Where eps, scaled
      // alike, is past fp32 it is all
      const int e = exponent_of(max_of_wave(max4(0.0f, x)));
      const float small = __builtin_amdgcn_ldexpf(eps, -2 * e);
      const bool all = small > 1e38f;
      if (!all) x = scale4(x, -e);
      square = all ? eps : sum_of_squares(x) + small;
    }
    scale *= 1.0f / __builtin_sqrtf(square);
  }
  if (lane < DK / 4) *reinterpret_cast<f4_t*>(to + 4 * lane) = x * scale;
}

// Each of a wave's 16 rows of the state with one row of q or k.
template <int DK>
__device__ __forceinline__ float dot(const StateTile<DK, 1>& x, const float* row) {
  const int g = (threadIdx.x & 63) >> 4;
  f4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int t = 0; t < DK / 16; ++t) acc += x.s[0][t] * *reinterpret_cast<const f4_t*>(row + 16 * t + 4 * g);
  return sum_of_groups((acc[0] + acc[1]) + (acc[2] + acc[3]));
}

// A chain, one token after the other.  Bound by reading and writing the states once:
// one token of 64 sequences, 48 heads of 128 x 128, 82 us, 4.9 TB/s of the 403 MB; of
// one sequence 5.9 us, of which its 6.3 MB are 1.3.  grid (dv / 64, heads, seqs).
template <int DK, bool BF16>
__global__ __launch_bounds__(64 * kWaves) void delta_step_kernel(DeltaArgs a) {
  __shared__ float rows[2][kTile][DK];  // k, q
  const int b = blockIdx.z, h = blockIdx.y, wave = threadIdx.x >> 6, lane = threadIdx.x & 63, j = lane & 15;
  const int kh = h / (a.heads / a.key_heads), row0 = (blockIdx.x * kWaves + wave) * 16;
  const int src = a.src[b];
  const bool used = delta_used(src, a.slots);
  const int count = used ? delta_count(a.counts, a.nodes, b) : 0;
  const int64_t state_size = (int64_t)a.dv * DK;
  StateTile<DK, 1> x;
  if (used && src >= 0) load_state<DK, 1>(a.states + ((int64_t)src * a.heads + h) * state_size + row0 * DK, x);
  else zero_state<DK, 1>(x);
  const int64_t first = (int64_t)b * a.nodes;
  for (int t0 = 0; t0 < count; t0 += kTile) {
    const int n = count - t0 < kTile ? count - t0 : kTile;
    __syncthreads();
    for (int i = wave; i < 2 * n; i += kWaves) {
      const int t = i >> 1;
      if (i & 1) stage_row<DK, BF16>(a.q, (first + t0 + t) * a.q_stride + kh * DK, a.norm_eps, a.scale, rows[1][t]);
      else stage_row<DK, BF16>(a.k, (first + t0 + t) * a.k_stride + kh * DK, a.norm_eps, 1.0f, rows[0][t]);
    }
    __syncthreads();
    for (int t = 0; t < n; ++t) {
      const int64_t r = first + t0 + t;
      const float decay = expf(a.g[r * a.heads + h]), beta = a.beta[r * a.heads + h];
      float v;
      const int64_t at = r * a.v_stride + h * a.dv + row0 + j;
      if constexpr (BF16) v = __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.v)[at] << 16);
      else v = static_cast<const float*>(a.v)[at];
#pragma unroll
      for (int e = 0; e < DK / 16; ++e) x.s[0][e] *= decay;
      const float u = beta * (v - dot<DK>(x, rows[0][t]));
#pragma unroll
      for (int e = 0; e < DK / 16; ++e)
        x.s[0][e] += u * *reinterpret_cast<const f4_t*>(&rows[0][t][16 * e + 4 * (lane >> 4)]);
      const float o = dot<DK>(x, rows[1][t]);
      if (lane < 16) store1<BF16>(a.out, (r * a.heads + h) * a.dv + row0 + j, o);
    }
  }
  for (int t = count; t < a.nodes; ++t)
    if (lane < 16) store1<BF16>(a.out, ((first + t) * a.heads + h) * a.dv + row0 + j, 0.0f);
  if (!used) return;
  const int to = delta_dst(a.src, a.dst, a.seqs, a.slots, b);
  if (to >= 0) store_state<DK, 1>(a.states + ((int64_t)to * a.heads + h) * state_size + row0 * DK, x);
}

// The accepted path of a tree into one state: e^G_end S + sum_i e^(G_end - G_i)
// u_i k_i^T over the root and the path, the sums of the decays behind each node in
// 64 bits.  A wave holds 16 rows of the state and takes the keys from LDS.  Bound by
// reading and writing the states once: 48 layers of one sequence, 48 heads of 128 x
// 128, a path of four: 62 us, 4.9 TB/s of the 302 MB; 5 layers of 24 sequences, 8 heads
// of 64 x 128, where a tile's latencies count as much: 18.8.  32 rows a wave halve the
// LDS reads of a key, but also the waves: 64.9 and 18.0.
// grid (layers * dv / 64, heads, seqs).
template <int DK>
__global__ __launch_bounds__(64 * kWaves) void delta_commit_kernel(DeltaCommitArgs a) {
  __shared__ float keys[kTile][DK];
  const int b = blockIdx.z, h = blockIdx.y, parts = a.dv / 64, layer = blockIdx.x / parts;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
  const int src = a.src[b];
  if (!delta_used(src, a.slots)) return;
  const int to = delta_dst(a.src, a.dst, a.seqs, a.slots, b);
  if (to < 0) return;
  const int kh = h / (a.heads / a.key_heads);
  const int row0 = ((blockIdx.x - layer * parts) * kWaves + wave) * 16;
  const int64_t state_size = (int64_t)a.dv * DK;
  float* states = a.states + (int64_t)layer * a.slots * a.heads * state_size;
  StateTile<DK, 1> x;
  if (src >= 0) load_state<DK, 1>(states + ((int64_t)src * a.heads + h) * state_size + row0 * DK, x);
  else zero_state<DK, 1>(x);
  // lane i: node i of the path (the root first), its decay and what follows it
  const int32_t* res = a.result + (int64_t)b * (3 + a.nodes);
  int n = res[1];
  n = 1 + (n < 0 ? 0 : n < a.nodes ? n : a.nodes - 1);
  int node = lane == 0 ? 0 : lane < n ? res[2 + lane] : -1;
  if (node >= delta_count(a.counts, a.nodes, b)) node = -1;
  const int64_t first = ((int64_t)layer * a.seqs + b) * a.nodes;
  const double decay = node >= 0 ? (double)a.g[(first + node) * a.heads + h] : 0.0;
  double after = 0.0;  // sum of the decays behind this node
  {
    double s = decay;
    for (int off = 1; off < 64; off <<= 1) {
      const double o = __shfl_down(s, off);
      s += lane + off < 64 ? o : 0.0;
    }
    const double all = __shfl(s, 0);
    const double o = __shfl_down(s, 1);
    after = lane < 63 ? o : 0.0;
    const float f = expf((float)all);
#pragma unroll
    for (int t = 0; t < DK / 16; ++t) x.s[0][t] *= f;
  }
  const float weight = node >= 0 ? expf((float)after) : 0.0f;
  for (int t0 = 0; t0 < n; t0 += kTile) {
    // a tile's u at once, one latency for all; a place without a node adds 0 times 0
    float u[kTile];
#pragma unroll
    for (int i = 0; i < kTile; ++i) {
      const int v = __builtin_amdgcn_readlane(node, t0 + i);
      const float w = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(weight), t0 + i));
      const float y = a.updates[((first + (v < 0 ? 0 : v)) * a.heads + h) * a.dv + row0 + j];
      u[i] = v < 0 ? 0.0f : w * y;
    }
    __syncthreads();
    for (int i = wave; i < kTile; i += kWaves) {
      const int v = __builtin_amdgcn_readlane(node, t0 + i);
      if (lane < DK / 4)
        *reinterpret_cast<f4_t*>(&keys[i][4 * lane]) =
            v < 0 ? f4_t{0.0f, 0.0f, 0.0f, 0.0f} : load4<false>(a.keys, ((first + v) * a.key_heads + kh) * DK + 4 * lane);
    }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kTile; ++i) {
      if (t0 + i >= n) break;
#pragma unroll
      for (int t = 0; t < DK / 16; ++t) x.s[0][t] += u[i] * *reinterpret_cast<const f4_t*>(&keys[i][16 * t + 4 * g]);
    }
  }
  store_state<DK, 1>(states + ((int64_t)to * a.heads + h) * state_size + row0 * DK, x);
}

template <int DK, bool BF16>
void step(const DeltaArgs& a, hipStream_t stream) {
  delta_step_kernel<DK, BF16><<<dim3(a.dv / 64, a.heads, a.seqs), 64 * kWaves, 0, stream>>>(a);
}

template <int DK>
void commit(const DeltaCommitArgs& a, hipStream_t stream) {
  delta_commit_kernel<DK><<<dim3(a.layers * (a.dv / 64), a.heads, a.seqs), 64 * kWaves, 0, stream>>>(a);
}

}  // namespace

// Up to four tokens go one after the other, up to 64 as one block, more block by
// block.  us a call in steps and as one block, 16 key and 48 value heads of 128, of 1, 8
// and 64 sequences: 4 bf16 tokens 10.3, 16.1, 101 and 10.3, 15.4, 93, 4 fp32 ones 10.4,
// 16.2, 107 and 10.4, 20.8, 122; 2 bf16 ones 10.6, 13.5, 86 and 10.5, 15.0, 91; 16 bf16
// ones 19.8, 31.6, 214 and 10.6, 15.7, 101.
constexpr int kFewTokens = 4;

int64_t delta_rule_workspace_bytes(const DeltaArgs& a) {
  return a.nodes <= kChunk ? 0 : delta_chunk_workspace_bytes(a);
}

hipError_t launch_delta_rule(const DeltaArgs& a, hipStream_t stream) {
  if (a.nodes > kFewTokens && a.nodes <= kChunk) {
    launch_delta_block(a, stream);
    return hipGetLastError();
  }
  if (a.nodes > kChunk && a.workspace_bytes >= delta_chunk_workspace_bytes(a)) {
    launch_delta_chunks(a, stream);
    return hipGetLastError();
  }
  if (a.dk == 64) a.bf16 ? step<64, true>(a, stream) : step<64, false>(a, stream);
  else if (a.dk == 128) a.bf16 ? step<128, true>(a, stream) : step<128, false>(a, stream);
  else a.bf16 ? step<256, true>(a, stream) : step<256, false>(a, stream);
  return hipGetLastError();
}

hipError_t launch_delta_tree(const DeltaArgs& a, hipStream_t stream) {
  launch_delta_block(a, stream);
  return hipGetLastError();
}

hipError_t launch_delta_commit(const DeltaCommitArgs& a, hipStream_t stream) {
  if (a.dk == 64) commit<64>(a, stream);
  else if (a.dk == 128) commit<128>(a, stream);
  else commit<256>(a, stream);
  return hipGetLastError();
}

}  // namespace nvfp4
