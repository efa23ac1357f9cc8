// Gated delta rule over drafted trees and chains of at most 64 tokens, in one launch.
//
// The page "TensorRT Edge-LLM Completes the MLPerf Edge Agentic Benchmark 6.4x
// Faster on Jetson AGX Thor" verifies a tree of drafted tokens in one pass (section
// "Using tree-based multi-token prediction to accelerate LLM inference").  A tree is a
// block of delta_block.h whose tokens see their ancestors: one reading of the state
// serves all nodes, where a state per node would be written and read again.  A short
// chain is a block that writes the state that follows.
//
// A workgroup has 64 columns of one head's state, a wave 16 of them; its first waves
// prepare the block (the other workgroups of the head do the same), while all of them
// wait for their columns.
//
// Bounds.  Latency: one load, the block's inverse and the products behind it.  A tree
// of 16 nodes, 16 key and 48 value heads of 128, bf16: 7.2 us on the device, of which
// its 4.5 MB are 0.9; 16 trees of up to 33 fp32 nodes, 4 and 8 heads of 64: 10.1; one of
// 64 fp32 nodes, 4 and 8 heads of 256, whose block takes a CU's whole LDS: 20.8.
#include "delta_block.h"

namespace nvfp4 {
namespace {

// grid (heads, dv / 64, seqs).
template <int DK, bool BF16, int NT, bool TREE>
__global__ __launch_bounds__(256) void delta_block_kernel(DeltaArgs a) {
  typedef BlockOps<DK, BF16, NT> Ops;
  constexpr int P = Ops::kParts, KT = DK / 16;
  __shared__ BlockShared<DK, BF16, NT, true> sh;
  const int h = blockIdx.x, b = blockIdx.z, lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
  const int group = a.heads / a.key_heads, kh = h / group, col0 = (blockIdx.y * 4 + (threadIdx.x >> 6)) * 16;
  const int64_t first = (int64_t)b * a.nodes, value_at = (int64_t)h * a.dv + col0 + j, row = (int64_t)a.heads * a.dv;
  BlockRows<DK, BF16> rows;
  load_block_rows<DK, BF16, NT, TREE>(a, first, a.nodes, h, kh, rows);
  const int src = a.src[b];
  const bool used = delta_used(src, a.slots);
  const int n = used ? delta_count(a.counts, a.nodes, b) : 0;
  StateTile<DK, 1> st;
  if (used && src >= 0) load_state<DK, 1>(a.states + (((int64_t)src * a.heads + h) * a.dv + col0) * DK, st);
  else zero_state<DK, 1>(st);
  f4_t(&s)[KT] = st.s[0];
  uint32_t raw[NT][4];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = 16 * t + 4 * g + e;
      const int64_t at = (first + (i < a.nodes ? i : a.nodes - 1)) * a.v_stride + value_at;
      if constexpr (BF16) raw[t][e] = static_cast<const uint16_t*>(a.v)[at];
      else raw[t][e] = static_cast<const uint32_t*>(a.v)[at];
    }
  float* keys = TREE && h % group == 0 && blockIdx.y == 0 ? a.keys + (first * a.key_heads + kh) * DK : nullptr;
  prepare_block<DK, BF16, NT, TREE, true>(a, rows, n, sh, nullptr, nullptr, keys, (int64_t)a.key_heads * DK, a.nodes);
  __syncthreads();
  float m = 0.0f;
#pragma unroll
  for (int t = 0; t < KT; ++t) m = max4(m, s[t]);
  const float m_state = max_of_groups(m);
  const int es = 5 - exponent_of(m_state);
  const f4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
  f4_t ks[NT], qs[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) ks[t] = qs[t] = zero;
#pragma unroll
  for (int x = 0; x < Ops::kSteps; ++x) {
    h8_t hi, lo;
    operand_parts(scale4(s[2 * x], es), scale4(s[2 * x + 1], es), hi, lo);
#pragma unroll
    for (int part = 0; part < P + 1; ++part)
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int at = (part == 2 ? Ops::kRows : 0) + (t * Ops::kSteps + x) * 64 + lane;
        ks[t] = mfma16x16x32(sh.key[at], part == 1 ? lo : hi, ks[t]);
        qs[t] = mfma16x16x32(sh.query[at], part == 1 ? lo : hi, qs[t]);
      }
  }
  const auto factor = [&](const float* of, int t) { return *reinterpret_cast<const f4_t*>(of + 16 * t + 4 * g); };
  f4_t v[NT], w[NT], pu[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const f4_t f = factor(sh.factor[kFactorR], t), beta = factor(sh.beta, t), y = scale4(ks[t], -es);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const float x = __uint_as_float(BF16 ? raw[t][e] << 16 : raw[t][e]);
      v[t][e] = 16 * t + 4 * g + e < n ? beta[e] * __builtin_fmaf(f[e], y[e], x) : 0.0f;
    }
  }
  const uint64_t lost = lost_values<NT>(lost_tokens(sh), v);
  const bool any_lost = __any(lost != 0);
  const float nan = __builtin_nanf("");
  lower_product<NT>([&](int t) { return tile_rows(sh.a[t]); }, v, w);
  lower_product<NT>([&](int t) { return tile_rows(sh.p[t]); }, w, pu);
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const f4_t fq = factor(sh.factor[kFactorQ], t), y = scale4(qs[t], -es);
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = 16 * t + 4 * g + e;
      if (i >= a.nodes) continue;
      const bool in = i < n;
      float u = w[t][e], o = __builtin_fmaf(fq[e], y[e], pu[t][e]);
      if (any_lost && ((TREE ? sh.line[i] : up_to(i)) & lost)) u = o = nan;
      if constexpr (TREE) a.updates[(first + i) * row + value_at] = in ? u : 0.0f;
      store1<BF16>(a.out, (first + i) * row + value_at, in ? o : 0.0f);
    }
  }
  if constexpr (!TREE) {
    if (!used) return;
    const int to = delta_dst(a.src, a.dst, a.seqs, a.slots, b);
    if (to < 0) return;
    if (n > 0) {
      // S <- e^G_end S + K^T X, X = diag(e^(G_end - G)) u
      f4_t x[NT + (NT & 1)];
      float mx = 0.0f;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        x[t] = w[t] * factor(sh.factor[kFactorX], t);
        mx = max4(mx, x[t]);
      }
      if constexpr (NT & 1) x[NT] = zero;
      const int en = 5 - exponent_of(max_of_groups(fmaxf(mx, m_state * sh.end)));
#pragma unroll
      for (int t = 0; t < KT; ++t) s[t] = scale4(s[t] * sh.end, en);
#pragma unroll
      for (int y = 0; y < Ops::kTokenSteps; ++y) {
        h8_t hi, lo;
        operand_parts(scale4(x[2 * y], en), scale4(x[2 * y + 1], en), hi, lo);
#pragma unroll
        for (int t = 0; t < KT; ++t) {
          const h8_t k = transposed_operand<DK, BF16, NT>(sh.key, 0, t, y);
          s[t] = mfma16x16x32(k, hi, s[t]);
          s[t] = mfma16x16x32(k, lo, s[t]);
          if constexpr (P == 2) s[t] = mfma16x16x32(transposed_operand<DK, BF16, NT>(sh.key, 1, t, y), hi, s[t]);
        }
      }
#pragma unroll
      for (int t = 0; t < KT; ++t) s[t] = scale4(s[t], -en);
      if (any_lost && lost)
#pragma unroll
        for (int t = 0; t < KT; ++t) s[t] = f4_t{nan, nan, nan, nan};
    }
    store_state<DK, 1>(a.states + (((int64_t)to * a.heads + h) * a.dv + col0) * DK, st);
  }
}

template <int DK, bool BF16, int NT>
void run(const DeltaArgs& a, hipStream_t stream) {
  const dim3 grid(a.heads, a.dv / 64, a.seqs);
  if (a.parent) delta_block_kernel<DK, BF16, NT, true><<<grid, 256, 0, stream>>>(a);
  else delta_block_kernel<DK, BF16, NT, false><<<grid, 256, 0, stream>>>(a);
}

template <int DK, bool BF16>
void run(const DeltaArgs& a, hipStream_t stream) {
  if (a.nodes <= 16) run<DK, BF16, 1>(a, stream);
  else if (a.nodes <= 32) run<DK, BF16, 2>(a, stream);
  else if (a.nodes <= 48) run<DK, BF16, 3>(a, stream);
  else run<DK, BF16, 4>(a, stream);
}

}  // namespace

void launch_delta_block(const DeltaArgs& a, hipStream_t stream) {
  if (a.dk == 64) a.bf16 ? run<64, true>(a, stream) : run<64, false>(a, stream);
  else if (a.dk == 128) a.bf16 ? run<128, true>(a, stream) : run<128, false>(a, stream);
  else a.bf16 ? run<256, true>(a, stream) : run<256, false>(a, stream);
}

}  // namespace nvfp4
