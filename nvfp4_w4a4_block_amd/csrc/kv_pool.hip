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
// (entry, page) list with the running offsets of the entries in LDS, one place a
// thread and turn, and the phases are separated by barriers.  (Four places, whose
// loads overlap, cost the usual call more than they gave the largest: 33 forks
// 25.9 us against 22.7, 20 sequences to 23552 tokens and back 41.1 against 41.5.)
// What bounds it is the one compute unit's rate of accesses to the counts, which
// lie at random; a given-up page costs one of them, the atomic that takes its
// holder off.  The one that takes the last holder off pushes the page, so the
// place of a page in the list must not depend on the order in which the atomics
// land: only where a call itself gives up a page more than once could it, and
// there the occurrences settle on the first by an atomic minimum in the page's
// count, which is zero by then and is reset afterwards.  A step of one sequence
// takes 4.5 us, of which the launch is about 2; 20 sequences to 23552 tokens (7360
// pages) 16, all of them back 25.  Several workgroups would need a launch, or a
// wait for one another, between the phases.
#include "device_common.h"
#include "kv_launch.h"

namespace nvfp4 {
namespace {

constexpr int kThreads = 1024, kWaves = kThreads / 64;
constexpr int kClaim = 1 << 30;           // claims lie below any count: place - kClaim

__device__ __forceinline__ int load_agent(const int32_t* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void store_agent(int32_t* p, int v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// Exclusive sums over the workgroup of N values a thread, and their totals.
template <int N>
__device__ __forceinline__ void block_scan(int (&v)[N], int (&total)[N], int (*sums)[N]) {
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  int mine[N];
#pragma unroll
  for (int i = 0; i < N; ++i) mine[i] = v[i];
  for (int off = 1; off < 64; off <<= 1) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const int o = __shfl_up(v[i], off);
      v[i] += lane >= off ? o : 0;
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i)
    if (lane == 63) sums[wave][i] = v[i];
  __syncthreads();
#pragma unroll
  for (int i = 0; i < N; ++i) {
    int before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) {
      const int s = sums[w][i];
      before += w < wave ? s : 0;
      all += s;
    }
    total[i] = all;
    v[i] += before - mine[i];
  }
}

// Entry of flattened place x: the last e with start[e] <= x, which has a page
// (start is the exclusive running sum of n entries, x is below the total).
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
  __shared__ int sums[kWaves][3], counts[2][kWaves], flags[2];
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6, n = a.n, W = a.width, P = a.pages;
  const int page = 1 << a.page_shift;

  // The entries, and which of them count.
  const bool in = t < n;
  const int d = in ? a.dst[t] : -1, tok = in ? a.tokens[t] : -1, s = FORK && in ? a.src[t] : -1;
  int F = a.free_list[0];
  F = F < 0 ? 0 : F < P ? F : P;
  dst[t] = d;
  src[t] = s;
  if (t < 2) flags[t] = 0;
  bool ok = in && d >= 0 && d < a.seqs && tok >= 0 && (!FORK || (s >= 0 && s < a.seqs));
  int have = ok ? a.held[d] : 0, of = FORK && ok ? a.held[s] : 0;
  __syncthreads();
  if (64 * wave < n) {
    bool again = false;
    for (int j = 0; j < n; j += 8) {  // places behind the last entry hold -1
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int other = dst[j + i];
        again |= (j + i < t && other == d) || (FORK && other == s);
      }
    }
    ok = ok && !again;
  }
  have = !ok || have < 0 ? 0 : have < W ? have : W;
  of = of < 0 ? 0 : of < W ? of : W;
  const int full = ok ? tok >> a.page_shift : 0;                    // whole pages
  const int part = ok ? tok & (page - 1) : 0;                       // tokens in a partial one
  const int need = full + (part > 0);
  ok = ok && need <= (FORK ? of : W);
  const int take = !ok ? 0 : FORK ? (part > 0) : need > have ? need - have : 0;
  const int drop = !ok ? 0 : FORK ? have : have > need ? have - need : 0;
  int at3[3] = {take, drop, FORK && ok ? full : 0}, total3[3];
  block_scan<3>(at3, total3, sums);
  const int takes = total3[0], drops = total3[1], shares = total3[2];
  take_at[t] = at3[0];
  drop_at[t] = at3[1];
  share_at[t] = at3[2];
  first[t] = FORK ? 0 : need < have ? need : have;
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
      fresh = a.free_list[F - at3[0]];
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
      const int p = a.free_list[F - x], e = entry_of(take_at, n, x);
      a.table[(int64_t)dst[e] * W + first[e] + (x - take_at[e])] = p;
      if (p >= 0 && p < P) store_agent(a.refs + p, 1);
    }
  }
  __syncthreads();

  // Pages given up: one holder less each.  An entry of the table that did not
  // take the last holder off is kept as -2 - page meanwhile.
  auto place = [&](int y) {
    const int e = entry_of(drop_at, n, y);
    return a.table + (int64_t)dst[e] * W + first[e] + (y - drop_at[e]);
  };
  for (int x = t; x < drops; x += kThreads) {
    int32_t* at = place(x);
    const int p = *at;
    if (p < 0 || p >= P) {
      *at = -1;
    } else if (atomicSub(a.refs + p, 1) != 1) {
      *at = -2 - p;
      flags[0] = 1;
    }
  }
  __syncthreads();
  // A page that has no holder left although this place did not take the last
  // one off is given up twice: its places claim it.
  if (flags[0]) {
    for (int x = t; x < drops; x += kThreads) {
      const int p = -2 - *place(x);
      if (p < 0) continue;
      const int r = load_agent(a.refs + p);
      if (r == 0 || r < -(kClaim >> 1)) {
        flags[1] = 1;
        atomicMin(a.refs + p, x - kClaim);
      }
    }
    __syncthreads();
  }
  const bool twice = flags[1] != 0;
  if (twice) {
    for (int x = t; x < drops; x += kThreads) {
      const int p = *place(x);
      if (p >= 0) atomicMin(a.refs + p, x - kClaim);
    }
    __syncthreads();
  }
  const int top = F - takes;
  int back = 0;
  for (int x0 = 0, turn = 0; x0 < drops; x0 += kThreads, turn ^= 1) {
    const int x = x0 + t;
    bool push = false;
    int p = -1;
    if (x < drops) {
      int32_t* at = place(x);
      const int v = *at;
      p = v < -1 ? -2 - v : v;
      push = twice ? p >= 0 && load_agent(a.refs + p) == x - kClaim : v >= 0;
      *at = -1;
    }
    const uint64_t own = __ballot(push);
    if (lane == 0) counts[turn][wave] = __popcll(own);
    __syncthreads();
    int rank = back;
    for (int w = 0; w < kWaves; ++w) {
      const int c = counts[turn][w];
      rank += w < wave ? c : 0;
      back += c;
    }
    if (push) {
      const int r = top + rank + 1 + __popcll(own & ((1ull << lane) - 1));
      if (r <= P) a.free_list[r] = p;
      if (twice) store_agent(a.refs + p, 0);
    }
  }
  __syncthreads();

  if (FORK) {
    for (int x = t; x < shares; x += kThreads) {
      const int e = entry_of(share_at, n, x), at = x - share_at[e];
      a.table[(int64_t)dst[e] * W + at] = a.table[(int64_t)src[e] * W + at];
    }
    if (take) a.table[(int64_t)d * W + full] = fresh;
  }
  if (ok) a.held[d] = need;
  if (t == 0) {
    a.free_list[0] = top + back < P ? top + back : P;
    a.shortage[0] = 0;
  }
}

// The used slots of the partial pages: block (head, layer and K or V, entry);
// bound by memory once there are many (33 half-filled pages of 128 tokens, 16
// layers of 4 x 128: 13.6 us for about 69 MB read and written).
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
