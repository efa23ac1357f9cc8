// Attention of a step's nodes over the paged FP8 KV cache.
//
// Simple form: one workgroup per (sequence, node, query head); 256 keys per
// pass, one key per thread, running maximum and sum.
#include "device_common.h"
#include "launch.h"

namespace nvfp4 {
namespace {

// Ancestor-or-self bits of node v of a tree of at most 64 nodes, lane = node:
// parent pointers doubled six times.  A parent outside [0, v) makes v a root.
__device__ __forceinline__ uint64_t ancestors_of_wave(int par) {
  const int lane = threadIdx.x & 63;
  uint64_t mask = 1ull << lane;
  int p = par >= 0 && par < lane ? par : -1;
  for (int s = 0; s < 6; ++s) {
    const int at = p < 0 ? lane : p;
    const uint64_t up = __shfl(mask, at);
    const int pp = __shfl(p, at);
    if (p >= 0) {
      mask |= up;
      p = pp;
    }
  }
  return mask;
}

template <bool BF16>
__global__ __launch_bounds__(256) void kv_attention_simple_kernel(KvAttentionArgs a) {
  __shared__ float qs[256], ps[256], red[4];
  __shared__ int64_t rows[256];
  __shared__ uint64_t line;
  const KvCache& c = a.c;
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const int hq = blockIdx.x, v = blockIdx.y, b = blockIdx.z;
  const int heads_q = c.heads * a.group, h = hq / a.group, D = c.dim;
  const int64_t row = (int64_t)b * a.nodes + v;
  const int64_t out_at = (row * heads_q + hq) * D;
  const int len = c.lens[b];
  int count = a.counts ? a.counts[b] : a.nodes;
  count = count < a.nodes ? count : a.nodes;
  const bool here = len >= 0 && v < count;
  if (!here) {
    if (t < D) {
      if (BF16) static_cast<uint16_t*>(a.out)[out_at + t] = 0;
      else static_cast<float*>(a.out)[out_at + t] = 0.0f;
    }
    if (t == 0 && a.lse) a.lse[row * heads_q + hq] = -__builtin_inff();
    return;
  }
  if (wave == 0) {
    const int par = a.parent && lane < a.nodes ? a.parent[(int64_t)b * a.nodes + lane] : -1;
    const uint64_t m = ancestors_of_wave(par);
    if (lane == (v & 63)) line = m;
  }
  if (t < D) {
    const int64_t at = row * a.q_stride + (int64_t)hq * D + t;
    qs[t] = BF16 ? __uint_as_float((uint32_t)static_cast<const uint16_t*>(a.q)[at] << 16)
                 : static_cast<const float*>(a.q)[at];
  }
  __syncthreads();
  const float ks = *a.k_scale * a.sm_scale, vs = *a.v_scale;
  const int end = len + (a.parent ? count : v + 1);
  float m = -__builtin_inff(), l = 0.0f, acc = 0.0f;
  for (int k0 = 0; k0 < end; k0 += 256) {
    const int pos = k0 + t;
    float s = -__builtin_inff();
    rows[t] = -1;
    if (pos < end && (pos < len || !a.parent || ((line >> (pos - len)) & 1))) {
      const int at = pos >> c.page_shift;
      const int page = at < c.width ? c.table[(int64_t)b * c.width + at] : -1;
      if (page >= 0 && page < c.pages) {
        const int64_t off =
            page * c.page_stride + (((int64_t)h << c.page_shift) + (pos & ((1 << c.page_shift) - 1))) * D;
        rows[t] = off;
        float dot = 0.0f;
        for (int d = 0; d < D; ++d) dot += qs[d] * e4m3_to_f32(c.k[off + d]);
        s = dot * ks;
      }
    }
    float top = s;
    for (int off = 32; off > 0; off >>= 1) top = __builtin_fmaxf(top, __shfl_xor(top, off));
    if (lane == 0) red[wave] = top;
    __syncthreads();
    top = __builtin_fmaxf(__builtin_fmaxf(red[0], red[1]), __builtin_fmaxf(red[2], red[3]));
    const float mn = __builtin_fmaxf(m, top);
    const float p = s == -__builtin_inff() ? 0.0f : expf(s - mn);
    const float f = m == -__builtin_inff() ? 0.0f : expf(m - mn);
    ps[t] = p;
    float sum = p;
    for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
    __syncthreads();
    if (lane == 0) red[wave] = sum;
    __syncthreads();
    l = l * f + (red[0] + red[1] + red[2] + red[3]);
    m = mn;
    if (t < D) {
      acc *= f;
      for (int j = 0; j < 256; ++j)
        if (rows[j] >= 0) acc += ps[j] * e4m3_to_f32(c.v[rows[j] + t]);
    }
    __syncthreads();
  }
  if (t < D) {
    const float o = l > 0.0f ? acc / l * vs : 0.0f;
    if (BF16) static_cast<uint16_t*>(a.out)[out_at + t] = f32_to_bf16_rne(o);
    else static_cast<float*>(a.out)[out_at + t] = o;
  }
  if (t == 0 && a.lse) a.lse[row * heads_q + hq] = l > 0.0f ? m + logf(l) : -__builtin_inff();
}

}  // namespace

int64_t kv_attention_workspace_bytes(const KvAttentionArgs&) { return 0; }

hipError_t launch_kv_attention(const KvAttentionArgs& a, hipStream_t stream) {
  const dim3 grid(a.c.heads * a.group, a.nodes, a.c.seqs);
  if (a.bf16) kv_attention_simple_kernel<true><<<grid, 256, 0, stream>>>(a);
  else kv_attention_simple_kernel<false><<<grid, 256, 0, stream>>>(a);
  return hipGetLastError();
}

}  // namespace nvfp4
