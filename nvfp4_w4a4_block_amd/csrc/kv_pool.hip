// Sharing, growing and freeing the pages of the KV cache, on the device.
//
// The page "TensorRT Edge-LLM Completes the MLPerf Edge Agentic Benchmark
// 6.4x Faster on Jetson AGX Thor" (section "Reusing KV cache across agent
// turns") starts a turn from the cached pages of its prefix.  Here a page is
// held by any number of sequences: refs[p] counts them, table[s][0 .. held[s])
// names a sequence's pages, and free_list holds the others: its first word is
// their number F, the rest a stack whose top is free_list[F].  All of it stays
// in device memory, so a step that needs pages, or drops some, has no host
// round trip and can be captured in a graph.
//
// One workgroup does the bookkeeping: every phase is a loop over the flattened
// (entry, page) list with the running offsets of the entries in LDS, and the
// phases are separated by barriers.  Nothing depends on the order in which the
// atomics land: the counts are sums, and a page that falls to zero goes back
// on the list at the rank of its first occurrence, which the occurrences agree
// on by an atomic minimum in the page's own count (zero at that point) that is
// reset afterwards.  Bound by the latency of its dependent accesses.
#include "device_common.h"
#include "launch.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 1024;
constexpr int kClaim = 1 << 30;  // claims lie below any count: occurrence - kClaim

__device__ __forceinline__ int load_agent(const int32_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void store_agent(int32_t* p, int v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Inclusive sum over the workgroup; `sums` has one word per wave.
__device__ __forceinline__ int block_scan(int v, int* sums, int* total) {
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  for (int off = 1; off < 64; off <<= 1) {
    const int o = __shfl_up(v, off);
    v += lane >= off ? o : 0;
  }
  if (lane == 63) sums[wave] = v;
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < kThreads / 64; ++w) {
    const int s = sums[w];
    before += w < wave ? s : 0;
    all += s;
  }
  __syncthreads();
  *total = all;
  return v + before;
}

// Entry of flattened index x: the last e with start[e] <= x among those that
// have a page (start is the exclusive running sum of n entries).
__device__ __forceinline__ int entry_of(const int* start, int n, int x) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (start[mid] <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

template <bool FORK>
__global__ __launch_bounds__(kThreads) void kv_pool_kernel(KvPoolArgs a) {
  __shared__ int src[kThreads], dst[kThreads];           // sequences (dst: the one that changes)
  __shared__ int first[kThreads];                        // resize: first page to take or give back
  __shared__ int take_at[kThreads], drop_at[kThreads], share_at[kThreads];  // running offsets
  __shared__ int sums[kThreads / 64];
  const int t = threadIdx.x, n = a.n, W = a.width, P = a.pages;
  const int page = 1 << a.page_shift;

  // The entries, and which of them count.
  const bool in = t < n;
  const int d = in ? a.dst[t] : -1, tok = in ? a.tokens[t] : -1, s = FORK && in ? a.src[t] : -1;
  dst[t] = d;
  src[t] = s;
  __syncthreads();
  bool ok = in && d >= 0 && d < a.seqs && tok >= 0 && (!FORK || (s >= 0 && s < a.seqs));
  for (int j = 0; j < n && ok; ++j) {
    if (j < t && dst[j] == d) ok = false;
    if (FORK && dst[j] == s) ok = false;
  }
  int have = 0;
  if (ok) {
    have = a.held[d];
    have = have < 0 ? 0 : have < W ? have : W;
  }
  const int full = ok ? tok >> a.page_shift : 0;                    // whole pages
  const int part = ok ? tok & (page - 1) : 0;                       // tokens in a partial one
  const int need = full + (part > 0);
  if (FORK) {
    if (ok) {
      int of = a.held[s];
      of = of < 0 ? 0 : of < W ? of : W;
      ok = need <= of;
    }
  } else {
    ok = ok && need <= W;
  }
  const int take = !ok ? 0 : FORK ? (part > 0) : need > have ? need - have : 0;
  const int drop = !ok ? 0 : FORK ? have : have > need ? have - need : 0;
  const int share = FORK && ok ? full : 0;
  int takes, drops, shares = 0;
  take_at[t] = block_scan(take, sums, &takes) - take;
  drop_at[t] = block_scan(drop, sums, &drops) - drop;
  if (FORK) share_at[t] = block_scan(share, sums, &shares) - share;
  first[t] = FORK ? 0 : need < have ? need : have;
  int F = a.free_list[0];
  F = F < 0 ? 0 : F < P ? F : P;
  __syncthreads();

  if (takes > F) {  // all or nothing
    if (FORK && in) a.moves[3 * t] = -1;
    if (t == 0) a.shortage[0] = takes - F;
    return;
  }

  // Pages taken off the list, and shared ones.
  int fresh = -1;
  if (FORK) {
    if (take) {
      fresh = a.free_list[F - take_at[t]];
      if (fresh >= 0 && fresh < P) store_agent(a.refs + fresh, 1);
    }
    if (in) {
      a.moves[3 * t] = take ? a.table[(int64_t)s * W + full] : -1;
      a.moves[3 * t + 1] = fresh;
      a.moves[3 * t + 2] = part;
    }
    for (int x = t; x < shares; x += kThreads) {
      const int e = entry_of(share_at, n, x);
      const int p = a.table[(int64_t)src[e] * W + (x - share_at[e])];
      if (p >= 0 && p < P) atomicAdd(a.refs + p, 1);
    }
  } else {
    for (int x = t; x < takes; x += kThreads) {
      const int e = entry_of(take_at, n, x);
      const int p = a.free_list[F - x];
      a.table[(int64_t)dst[e] * W + first[e] + (x - take_at[e])] = p;
      if (p >= 0 && p < P) store_agent(a.refs + p, 1);
    }
  }
  __syncthreads();

  // Pages given up: one holder less each, then the claims of those at zero.
  for (int x = t; x < drops; x += kThreads) {
    const int e = entry_of(drop_at, n, x);
    const int p = a.table[(int64_t)dst[e] * W + first[e] + (x - drop_at[e])];
    if (p >= 0 && p < P) atomicSub(a.refs + p, 1);
  }
  __syncthreads();
  for (int x = t; x < drops; x += kThreads) {
    const int e = entry_of(drop_at, n, x);
    const int p = a.table[(int64_t)dst[e] * W + first[e] + (x - drop_at[e])];
    if (p >= 0 && p < P) {
      const int r = load_agent(a.refs + p);
      if (r == 0 || r < -(kClaim >> 1)) atomicMin(a.refs + p, x - kClaim);
    }
  }
  __syncthreads();
  const int top = F - takes;
  int back = 0;
  for (int x0 = 0; x0 < drops; x0 += kThreads) {
    const int x = x0 + t;
    int p = -1;
    bool mine = false;
    if (x < drops) {
      const int e = entry_of(drop_at, n, x);
      int32_t* at = a.table + (int64_t)dst[e] * W + first[e] + (x - drop_at[e]);
      p = *at;
      mine = p >= 0 && p < P && load_agent(a.refs + p) == x - kClaim;
      *at = -1;
    }
    int all;
    const int rank = back + block_scan(mine ? 1 : 0, sums, &all);
    if (mine) {
      store_agent(a.refs + p, 0);
      if (top + rank <= P) a.free_list[top + rank] = p;
    }
    back += all;
  }
  __syncthreads();

  if (FORK) {
    for (int x = t; x < shares; x += kThreads) {
      const int e = entry_of(share_at, n, x);
      const int j = x - share_at[e];
      a.table[(int64_t)dst[e] * W + j] = a.table[(int64_t)src[e] * W + j];
    }
    if (take) a.table[(int64_t)d * W + full] = fresh;
  }
  if (ok) a.held[d] = need;
  if (t == 0) {
    a.free_list[0] = top + back < P ? top + back : P;
    a.shortage[0] = 0;
  }
}

// The used slots of the partial pages: block (head, layer and K or V, entry).
__global__ __launch_bounds__(256) void kv_move_kernel(const int32_t* moves, KvCache c) {
  const int32_t* m = moves + 3 * blockIdx.z;
  const int from = m[0];
  if (from < 0 || from >= c.pages) return;
  const int to = m[1], slots = m[2];
  if (to < 0 || to >= c.pages) return;
  const int64_t off = (int64_t)(blockIdx.y >> 1) * c.layer_stride + (((int64_t)blockIdx.x << c.page_shift) * c.dim);
  uint8_t* base = ((blockIdx.y & 1) ? c.v : c.k) + off;
  const u4_t* x = reinterpret_cast<const u4_t*>(base + from * c.page_stride);
  u4_t* y = reinterpret_cast<u4_t*>(base + to * c.page_stride);
  const int chunks = (slots * c.dim) >> 4;
  for (int i = threadIdx.x; i < chunks; i += 256) y[i] = x[i];
}

}  // namespace

hipError_t launch_kv_resize(const KvPoolArgs& a, hipStream_t stream) {
  kv_pool_kernel<false><<<1, kThreads, 0, stream>>>(a);
  return hipGetLastError();
}

hipError_t launch_kv_fork(const KvPoolArgs& a, const KvCache& c, hipStream_t stream) {
  kv_pool_kernel<true><<<1, kThreads, 0, stream>>>(a);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || a.n == 0 || c.layers == 0) return e;
  kv_move_kernel<<<dim3(c.heads, 2 * c.layers, a.n), 256, 0, stream>>>(a.moves, c);
  return hipGetLastError();
}

}  // namespace nvfp4
