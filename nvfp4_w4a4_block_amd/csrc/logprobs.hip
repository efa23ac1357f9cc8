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
// its column, so keys are unique and descend by value, then column.
//
// Work.  A wave takes batches of 1024 logits, 16 a lane, each read once.  Its maximum
// is one number for all lanes, which a batch seldom moves; then a logit costs eight
// instructions, an exponential among them.  Of every 64 neighbouring columns the
// maximum is kept (a block's key: its maximum above the complement of its place).
// `top` blocks with keys no smaller than some bound are enough: the first `top`
// logits are in blocks that reach it.  The blocks' keys lie in 64 lanes; the top-th
// largest of the lanes' largest is such a bound, and little more than `top` blocks
// reach it.  Their logits are read again, and what reaches the bound's value is
// sorted.  So the loop over the logits does nothing for `top` but the maxima, where
// lists of first keys that are kept up batch by batch cost 26 us of 58 (512 rows of
// 151,936, five alternatives) and 9 of 21 (16 rows, twenty).
//
// Bounds (us of calls one after the other).  512 bf16 rows of 151,936, five
// alternatives: 39.7, 3.9 TB/s of 156 MB (32.5, 4.8 TB/s, without alternatives, whose
// blocks are found and sorted behind the last logit).  16 fp32 rows, twenty alternatives:
// 18.9, by trace 6.3 for the parts and 10.2 for the rows, of which the 9.7 MB are 2: what
// is left is latency, of the launches, loads and sorts.
#include <type_traits>

#include "device_common.h"
#include "hybrid_launch.h"

namespace nvfp4 {
namespace {

constexpr int kWaves = 8;
constexpr int kBatch = 16;            // logits of a lane at a time
constexpr int kCols = 64 * kBatch;    // of a wave
constexpr float kLog2E = 1.4426950408889634f;

struct Stat {
  float m, a, t;
};

// e^d of d <= 0: off by 2^-24 |d| of itself, from the product's rounding, and 2^-23.  A
// term so far down weighs e^d; a second multiply-add for it would be one of nine
// instructions a logit.
__device__ __forceinline__ float exp_of(float d) { return __builtin_amdgcn_exp2f(d * kLog2E); }

__device__ __forceinline__ Stat join(const Stat& x, const Stat& y) {
  const bool first = x.m >= y.m;
  const Stat hi = first ? x : y, lo = first ? y : x;
  if (lo.a == -1.0f) return hi;  // nothing there
  const float d = lo.m - hi.m, f = exp_of(d), w = 1.0f + lo.a;
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

template <int CTRL>
__device__ __forceinline__ uint64_t dpp(uint64_t x) {
  const uint32_t lo = __builtin_amdgcn_update_dpp(0, (uint32_t)x, CTRL, 0xF, 0xF, true);
  const uint32_t hi = __builtin_amdgcn_update_dpp(0, (uint32_t)(x >> 32), CTRL, 0xF, 0xF, true);
  return ((uint64_t)hi << 32) | lo;
}

template <int CTRL>
__device__ __forceinline__ float dpp_float(float x) {
  return __uint_as_float(__builtin_amdgcn_update_dpp(0, __float_as_uint(x), CTRL, 0xF, 0xF, true));
}

// A lane's key, for all.
__device__ __forceinline__ uint64_t lane_key(uint64_t x, int with) {
  const uint32_t lo = __builtin_amdgcn_readlane((uint32_t)x, with), hi = __builtin_amdgcn_readlane((uint32_t)(x >> 32), with);
  return ((uint64_t)hi << 32) | lo;
}

// The wave's own LDS stores before its loads: no other wave has part in them.
__device__ __forceinline__ void wave_sync() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
}

// quad_perm three times, row_half_mirror, row_ror:8, row_mirror
constexpr int kXor1 = 0xB1, kXor2 = 0x4E, kXor3 = 0x1B, kXor7 = 0x141, kXor8 = 0x128, kXor15 = 0x140;

// The key of the lane D from this one, D 16 or 32.
template <int D>
__device__ __forceinline__ uint64_t swap_halves(uint64_t x) {
  typedef uint32_t pair_t __attribute__((ext_vector_type(2)));
  const uint32_t l = (uint32_t)x, h = (uint32_t)(x >> 32);
  pair_t lo, hi;  // the pair's two words, in either lane alike
  if constexpr (D == 16) {
    lo = __builtin_bit_cast(pair_t, __builtin_amdgcn_permlane16_swap(l, l, false, false));
    hi = __builtin_bit_cast(pair_t, __builtin_amdgcn_permlane16_swap(h, h, false, false));
  } else {
    lo = __builtin_bit_cast(pair_t, __builtin_amdgcn_permlane32_swap(l, l, false, false));
    hi = __builtin_bit_cast(pair_t, __builtin_amdgcn_permlane32_swap(h, h, false, false));
  }
  const bool lower = (threadIdx.x & D) == 0;
  return lower ? ((uint64_t)hi.y << 32) | lo.y : ((uint64_t)hi.x << 32) | lo.x;
}

// A lane and the one `D` from it: the larger key to the lower lane.
template <int D>
__device__ __forceinline__ uint64_t compare(uint64_t x) {
  const bool lower = (threadIdx.x & D) == 0;
  uint64_t o;
  if constexpr (D >= 16) o = swap_halves<D>(x);
  else o = D == 8 ? dpp<kXor8>(x) : D == 4 ? dpp<kXor3>(dpp<kXor7>(x)) : D == 2 ? dpp<kXor2>(x) : dpp<kXor1>(x);
  return (o > x) == lower ? o : x;
}

// Lists have one key a lane, in descending order, 0 behind the last.  The first 64 of
// two of them: of a key of one and its mirror in the other the larger is among them;
// what they make rises and falls at most once, and is sorted by halving distances.
__device__ __forceinline__ uint64_t merge_lists(uint64_t x, uint64_t y) {
  y = swap_halves<32>(swap_halves<16>(dpp<kXor15>(y)));
  x = x > y ? x : y;
  x = compare<32>(x);
  x = compare<16>(x);
  x = compare<8>(x);
  x = compare<4>(x);
  x = compare<2>(x);
  return compare<1>(x);
}

// A lane and its mirror among `K` neighbours: the larger key to the lower lane.
template <int K>
__device__ __forceinline__ uint64_t compare_mirror(uint64_t x) {
  const bool lower = (threadIdx.x & (K / 2)) == 0;
  uint64_t o = K == 2 ? dpp<kXor1>(x) : K == 4 ? dpp<kXor3>(x) : K == 8 ? dpp<kXor7>(x) : dpp<kXor15>(x);
  if constexpr (K >= 32) o = swap_halves<16>(o);
  if constexpr (K == 64) o = swap_halves<32>(o);
  return (o > x) == lower ? o : x;
}

// The lanes' keys in descending order; those of the first n lanes alone are not 0.
// Sorted pieces of 1, 2, 4 .. lanes are merged as lists are.  A loop of few
// instructions: what runs once a row waits for its code, too.
__device__ __forceinline__ uint64_t sort_lanes(uint64_t x, int n) {
#pragma unroll 1
  for (int k = 2; k < 2 * n && k <= 64; k *= 2) {
    if (k == 2) x = compare_mirror<2>(x);
    else if (k == 4) x = compare_mirror<4>(x);
    else if (k == 8) x = compare_mirror<8>(x);
    else if (k == 16) x = compare_mirror<16>(x);
    else if (k == 32) x = compare_mirror<32>(x);
    else x = compare_mirror<64>(x);
    if (k > 32) x = compare<16>(x);
    if (k > 16) x = compare<8>(x);
    if (k > 8) x = compare<4>(x);
    if (k > 4) x = compare<2>(x);
    if (k > 2) x = compare<1>(x);
  }
  return x;
}

// 16 logits of a lane from the wave's first column on, -infinity outside [0, n).
// `off` logits stand between a 16-byte border and the row's first one; column c of a
// batch is logit c - off of the row, so that loads are whole.
template <bool BF16>
__device__ __forceinline__ int column_of(int e) {
  const int lane = threadIdx.x & 63;
  return BF16 ? (e >> 3) * 512 + 8 * lane + (e & 7) : (e >> 2) * 256 + 4 * lane + (e & 3);
}

template <bool BF16>
struct Raw {
  u4_t w[BF16 ? 2 : 4];
};

template <bool BF16>
__device__ __forceinline__ void fetch(const void* row, int n, int first, Raw<BF16>& raw) {
  constexpr int per = BF16 ? 8 : 4, bits = BF16 ? 16 : 32;
  typedef std::conditional_t<BF16, uint16_t, uint32_t> value_t;
  const value_t* z = static_cast<const value_t*>(row);
#pragma unroll
  for (int i = 0; i < 16 / per; ++i) {
    const int c = first + column_of<BF16>(i * per);
    if (c >= 0 && c + per <= n) {
      raw.w[i] = __builtin_nontemporal_load(reinterpret_cast<const u4_t*>(z + c));
      continue;
    }
    uint64_t half[2] = {0, 0};  // the row's ends
#pragma unroll
    for (int h = 0; h < 2; ++h)
#pragma unroll 1
      for (int e = 0; e < per / 2; ++e) {
        const int at = c + h * (per / 2) + e;
        const uint64_t x = at >= 0 && at < n ? z[at] : BF16 ? 0xFF80u : 0xFF800000u;
        half[h] |= x << (bits * e);
      }
    raw.w[i] = u4_t{(uint32_t)half[0], (uint32_t)(half[0] >> 32), (uint32_t)half[1], (uint32_t)(half[1] >> 32)};
  }
}

template <bool BF16>
__device__ __forceinline__ void unpack(const Raw<BF16>& raw, float (&z)[kBatch]) {
#pragma unroll
  for (int e = 0; e < kBatch; ++e) {
    if constexpr (BF16) {
      const uint32_t w = raw.w[e >> 3][(e & 7) >> 1];
      z[e] = __uint_as_float((e & 1) ? w & 0xFFFF0000u : w << 16);
    } else {
      z[e] = __uint_as_float(raw.w[e >> 2][e & 3]);
    }
  }
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

constexpr float kLow = -3.4028234663852886e38f;

// A lane's share of its wave's sums; the maximum is the wave's, and one lane's a
// leaves out the 1 of one logit that is it.
struct Sums {
  float m, a, t;
  int owner;  // that lane, -1 before the first logit above kLow
};

__device__ __forceinline__ void add_batch(const float (&z)[kBatch], float top, Sums& s) {
  const int lane = threadIdx.x & 63;
  if (__any(top > s.m)) {
    const float m = max_of_wave(top);
    const float d = s.m - m, f = exp_of(d);
    // the 1 that was left out belongs to the sum from now on
    const float w = s.a + (lane == s.owner ? 1.0f : 0.0f);
    s.t = f == 0.0f && w == w ? 0.0f : f * (s.t + w * d);
    s.a = f == 0.0f && w == w ? 0.0f : f * w;
    s.m = m;
    s.owner = __builtin_ctzll(__ballot(top == m));
    bool left = lane == s.owner;
#pragma unroll
    for (int e = 0; e < kBatch; ++e) {
      const float x = z[e] - m;
      const bool out = left && x == 0.0f;
      left &= !out;
      const float p = exp_of(x);
      s.a += out ? 0.0f : p;
      s.t = __builtin_fmaf(p, fmaxf(x, kLow), s.t);
    }
    return;
  }
  float a = 0.0f, t = 0.0f;
#pragma unroll
  for (int e = 0; e < kBatch; ++e) {
    const float x = z[e] - s.m, p = exp_of(x);  // NaN and +infinity stay in p
    a += p;
    t = __builtin_fmaf(p, fmaxf(x, kLow), t);   // 0 * kLow, not 0 * -infinity
  }
  s.a += a;
  s.t += t;
}

constexpr int kBlock = 64;         // columns that share a maximum
constexpr int kLocalBlocks = 4096;  // blocks of a row whose maxima stay in LDS

__device__ __forceinline__ float larger(float x, float y) { return __builtin_elementwise_maximum(x, y); }

// Largest numbers of the blocks of a wave's batch, from `blocks` on.  +0.0 is above -0.0,
// as it is in the keys (fmaxf leaves that open); a NaN stays, and its row has no results.
template <bool BF16>
__device__ __forceinline__ void store_maxima(const float (&z)[kBatch], uint32_t* blocks) {
  constexpr int per = BF16 ? 8 : 4, lanes = kBlock / per;
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int i = 0; i < kBatch / per; ++i) {
    float m = z[i * per];
#pragma unroll
    for (int e = 1; e < per; ++e) m = larger(m, z[i * per + e]);
    m = larger(m, dpp_float<kXor1>(m));
    m = larger(m, dpp_float<kXor2>(m));
    m = larger(m, dpp_float<kXor7>(m));
    if constexpr (!BF16) m = larger(m, dpp_float<kXor8>(m));  // of either half's eight alike
    if ((lane & (lanes - 1)) == 0) blocks[i * (64 / lanes) + lane / lanes] = ordered(m);
  }
}

// Parts of a row: their numbers; and the row's blocks.
struct Plan {
  int parts, columns;  // of a row; of a part
  int blocks;          // of a row, at most
  bool local;          // the maxima stay in LDS (one part)
  Stat* stats;         // [rows][parts]
  uint32_t* maxima;    // [rows][blocks]
};

template <bool BF16>
__device__ __forceinline__ float logit_at(const char* row, int column) {
  if constexpr (BF16) return __uint_as_float((uint32_t)reinterpret_cast<const uint16_t*>(row)[column] << 16);
  else return reinterpret_cast<const float*>(row)[column];
}

// What the waves share while the row's first logits are looked for.
constexpr int kEach = 64 + 64;  // keys that a wave leaves, at most
struct Shared {
  Stat stats[kWaves];
  uint64_t room[kWaves][kEach];  // a wave's keys that wait to be sorted
  uint64_t left[kWaves * kEach];
  int lefts;
  uint64_t most[kWaves][64];     // the lanes' largest blocks
  uint32_t ids[kWaves][8 * 64];  // a wave's blocks that reach the bound
};

// n keys, one a lane, into a list.
__device__ __forceinline__ void add_keys(uint64_t x, int n, uint64_t& list) {
  x = sort_lanes(x, n);
  list = lane_key(list, 0) ? merge_lists(list, x) : x;
}

__device__ __forceinline__ int below(uint64_t lanes) {
  return __builtin_amdgcn_mbcnt_hi((uint32_t)(lanes >> 32), __builtin_amdgcn_mbcnt_lo((uint32_t)lanes, 0));
}

// The row's first `top` keys, lane i the i-th, by the whole workgroup (right in wave
// 0).  `row` starts `off` columns after the blocks' first column.
template <bool BF16>
__device__ __forceinline__ uint64_t first_keys(const LogprobArgs& a, const Plan& p, const char* row, int off,
                                               const uint32_t* maxima, Shared& sh) {
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int blocks = (a.vocab + off + kBlock - 1) / kBlock;
  // each lane's largest of the blocks lane, lane + 64 ..: the first of equal ones.  The
  // waves look through an eighth each.
  uint32_t best = 0, where = 0;
  for (int j = 64 * wave + lane; j < blocks; j += 4 * 64 * kWaves) {
    uint32_t m[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) m[u] = j + 64 * kWaves * u < blocks ? maxima[j + 64 * kWaves * u] : 0;
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      where = m[u] > best ? j + 64 * kWaves * u : where;
      best = m[u] > best ? m[u] : best;
    }
  }
  sh.most[wave][lane] = best ? ((uint64_t)best << 32) | (0xFFFFFFFFu - where) : 0;
  if (threadIdx.x == 0) sh.lefts = 0;
  __syncthreads();
  uint64_t most = sh.most[0][lane];
#pragma unroll
  for (int w = 1; w < kWaves; ++w) most = sh.most[w][lane] > most ? sh.most[w][lane] : most;
  uint64_t bound = lane_key(sort_lanes(most, 64), a.top - 1);
  bound = bound ? bound : 1;
  const uint32_t least = (uint32_t)(bound >> 32), latest = 0xFFFFFFFFu - (uint32_t)bound;
  uint64_t list = 0, last = (uint64_t)least << 32;  // no logit's key below it is among the first
  uint64_t* room = sh.room[wave];
  uint32_t* ids = sh.ids[wave];
  int at = 0;
  // the waves take 64 blocks in turn, eight times
  for (int j = wave; 64 * j < blocks; j += 8 * kWaves) {
    uint32_t m[8];
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = 64 * (j + u * kWaves) + lane;
      m[u] = i < blocks ? maxima[i] : 0;
    }
    int found = 0;
    wave_sync();
#pragma unroll
    for (int u = 0; u < 8; ++u) {
      const int i = 64 * (j + u * kWaves) + lane;
      const bool in = m[u] > least || (m[u] != 0 && m[u] == least && (uint32_t)i <= latest);
      const uint64_t w = __ballot(in);
      if (in) ids[found + below(w)] = i;
      found += __popcll(w);
    }
    wave_sync();
    for (int f = 0; f < found; f += 8) {
      // eight blocks' logits at a time, one a lane
      uint64_t key[8];
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const int n = f + u < found ? (int)ids[f + u] * kBlock + lane - off : -1;
        key[u] = n >= 0 && n < a.vocab
                     ? ((uint64_t)ordered(logit_at<BF16>(row, n)) << 32) | (0xFFFFFFFFu - (uint32_t)n) : 0;
      }
#pragma unroll
      for (int u = 0; u < 8; ++u) {
        const bool in = key[u] >= last;
        const uint64_t w = __ballot(in);
        if (w == 0) continue;
        if (in) room[at + below(w)] = key[u];
        at += __popcll(w);
        if (at < 64) continue;
        wave_sync();
        add_keys(room[lane], 64, list);
        at -= 64;
        const uint64_t rest = room[64 + lane], l = lane_key(list, a.top - 1);
        wave_sync();
        if (lane < at) room[lane] = rest;
        last = l > last ? l : last;
      }
    }
  }
  wave_sync();
  // what every wave has left, sorted by the first: mostly little more than `top` keys
  const uint64_t mine = __ballot(lane < a.top && list != 0);
  const int n = at + __popcll(mine);
  int to = 0;
  if (lane == 0 && n > 0) to = atomicAdd(&sh.lefts, n);
  to = __builtin_amdgcn_readfirstlane(to);
  if (lane < at) sh.left[to + lane] = room[lane];
  if (lane < a.top && list != 0) sh.left[to + at + below(mine)] = list;
  __syncthreads();
  if (wave != 0) return 0;
  list = 0;
  for (int i = 0; i < sh.lefts; i += 64) {
    const int k = sh.lefts - i < 64 ? sh.lefts - i : 64;
    add_keys(lane < k ? sh.left[i + lane] : 0, k, list);
  }
  return list;
}

// The lanes' numbers as one, in all lanes: as `join` does with two.
__device__ __forceinline__ Stat join_lanes(const Stat& s) {
  const bool some = s.a != -1.0f;
  const float m = max_of_wave(some ? s.m : -__builtin_inff());
  const uint64_t first = __ballot(some && s.m == m);
  const bool mine = first && (int)(threadIdx.x & 63) == __builtin_ctzll(first);
  const float d = s.m - m, f = exp_of(d), w = 1.0f + s.a;
  const bool in = some && !(f == 0.0f && w == w);
  const float a = sum_of_wave(mine ? s.a : in ? f * w : 0.0f);
  const float t = sum_of_wave(mine ? s.t : in ? f * (s.t + w * d) : 0.0f);
  return first ? Stat{m, a, t} : Stat{-__builtin_inff(), __any(some) ? __builtin_nanf("") : -1.0f, 0.0f};
}

// The waves' numbers as one, in all of them.
__device__ __forceinline__ Stat join_waves(const Stat& s, Stat* stats) {
  const int lane = threadIdx.x & 63;
  if (lane == 0) stats[threadIdx.x >> 6] = s;
  __syncthreads();
  return join_lanes(lane < kWaves ? stats[lane] : Stat{0.0f, -1.0f, 0.0f});
}

// The given token's logit.
template <bool BF16>
__device__ __forceinline__ float token_logit(const LogprobArgs& a, int64_t row, const char* from) {
  const int token = a.tokens[row];
  return token >= 0 && token < a.vocab ? logit_at<BF16>(from, token) : __builtin_nanf("");
}

// The row's results, by wave 0; lane i has the i-th key.
__device__ __forceinline__ void finish(const LogprobArgs& a, int64_t row, float given, const Stat& s, uint64_t k) {
  const int lane = threadIdx.x & 63;
  const bool none = !(s.m > -__builtin_inff()) || s.a != s.a || s.a < 0.0f;
  const float nan = __builtin_nanf(""), l = log1pf(s.a);
  if (lane == 0) {
    a.logprobs[row] = none ? nan : (given - s.m) - l;
    a.entropy[row] = none ? nan : l - s.t / (1.0f + s.a);
  }
  if (lane < a.top) {
    const float z = from_ordered((uint32_t)(k >> 32));
    a.top_logprobs[row * a.top + lane] = none ? nan : (z - s.m) - l;
    a.top_tokens[row * a.top + lane] = none ? -1 : (int32_t)(0xFFFFFFFFu - (uint32_t)k);
  }
}

// grid (parts, rows).  LOCAL: one part, whose maxima stay in LDS and which goes on to
// the results.
template <bool BF16, bool LOCAL>
__global__ __launch_bounds__(64 * kWaves) void logprob_part_kernel(LogprobArgs a, Plan p) {
  __shared__ Shared sh;
  __shared__ uint32_t maxima[LOCAL ? kLocalBlocks + kCols / kBlock : 1];
  constexpr int size = BF16 ? 2 : 4;
  const int64_t row = blockIdx.y;
  const int wave = threadIdx.x >> 6;
  const char* from = static_cast<const char*>(a.logits) + row * a.stride * size;
  const int off = (int)((uintptr_t)from & 15) / size;
  const int end = (blockIdx.x + 1) * p.columns < a.vocab + off ? (blockIdx.x + 1) * p.columns : a.vocab + off;
  uint32_t* blocks = LOCAL ? maxima : p.maxima + row * p.blocks;
  const float given = LOCAL ? token_logit<BF16>(a, row, from) : 0.0f;
  Sums s = {kLow, 0.0f, 0.0f, -1};
  Raw<BF16> raw, ahead;
  int c = blockIdx.x * p.columns + (wave - kWaves) * kCols;  // of the batch in raw; none yet
  for (bool any = false;; any = true) {
    const int next = c + kWaves * kCols;
    if (next < end) fetch<BF16>(from, a.vocab, next - off, ahead);
    if (any) {
      float z[kBatch];
      unpack<BF16>(raw, z);
      float top = z[0];
#pragma unroll
      for (int e = 1; e < kBatch; ++e) top = fmaxf(top, z[e]);
      add_batch(z, top, s);
      if (a.top > 0) store_maxima<BF16>(z, blocks + c / kBlock);
    }
    if (next >= end) break;
    raw = ahead;
    c = next;
  }
  // a wave that saw nothing above kLow has no owner: if there is a kLow, a counts it
  Stat sum = {s.m, sum_of_wave(s.a), sum_of_wave(s.t)};
  if (s.owner < 0) sum.a -= 1.0f;
  const Stat all = join_waves(sum, sh.stats);
  if constexpr (LOCAL) {
    const uint64_t k = a.top > 0 ? first_keys<BF16>(a, p, from, off, maxima, sh) : 0;
    if (wave == 0) finish(a, row, given, all, k);
  } else {
    if (threadIdx.x == 0) p.stats[row * p.parts + blockIdx.x] = all;
  }
}

// grid (rows): joins the parts of a row.  STAGED: the blocks' maxima, written by other
// parts of the chip, are fetched once, by all waves together.
template <bool BF16, bool STAGED>
__global__ __launch_bounds__(64 * kWaves) void logprob_row_kernel(LogprobArgs a, Plan p) {
  __shared__ Shared sh;
  __shared__ uint32_t staged[STAGED ? kLocalBlocks : 1];
  constexpr int size = BF16 ? 2 : 4;
  const int64_t row = blockIdx.x;
  const char* from = static_cast<const char*>(a.logits) + row * a.stride * size;
  const int off = (int)((uintptr_t)from & 15) / size;
  const uint32_t* maxima = p.maxima + row * p.blocks;
  if (STAGED && a.top > 0) {
    u4_t m[kLocalBlocks / (256 * kWaves)];
#pragma unroll
    for (int u = 0; u < kLocalBlocks / (256 * kWaves); ++u) {
      const int i = 4 * (64 * kWaves * u + threadIdx.x);
      m[u] = i < p.blocks ? *reinterpret_cast<const u4_t*>(maxima + i) : u4_t{0, 0, 0, 0};
    }
#pragma unroll
    for (int u = 0; u < kLocalBlocks / (256 * kWaves); ++u)
      *reinterpret_cast<u4_t*>(staged + 4 * (64 * kWaves * u + threadIdx.x)) = m[u];
    maxima = staged;
  }
  const float given = token_logit<BF16>(a, row, from);
  Stat s = {-__builtin_inff(), -1.0f, 0.0f};
  for (int i = threadIdx.x; i < p.parts; i += 64 * kWaves) s = join(s, p.stats[row * p.parts + i]);
  __syncthreads();
  const Stat all = p.parts <= 64 ? join_lanes(s) : join_waves(join_lanes(s), sh.stats);
  const uint64_t k = a.top > 0 ? first_keys<BF16>(a, p, from, off, maxima, sh) : 0;
  if (threadIdx.x < 64) finish(a, row, given, all, k);
}

// Parts of a row: one where there are rows enough for the chip (two workgroups a
// CU), else as many as give it that, a batch for every wave at least.  With one, two
// and four workgroups a CU, us a call, rows of 151,936: 16 fp32 with twenty alternatives
// and 64 bf16 with five 18.9 to 19.0 each; 300 bf16 38.8, 36.0, 33.8; 512 bf16 39.6, 39.7,
// 43.6 (two parts a row).  Columns are counted from the 16-byte border before the row.
Plan plan_of(const LogprobArgs& a) {
  constexpr int batch = kWaves * kCols;
  const int columns = a.vocab + (a.bf16 ? 7 : 3);
  const int most = (columns + batch - 1) / batch, want = (512 + a.rows - 1) / a.rows;
  Plan p = {};
  p.parts = want < most ? want : most;
  p.blocks = (columns + kCols - 1) / kCols * (kCols / kBlock);
  if (p.parts == 1 && p.blocks > kLocalBlocks) p.parts = 2;
  p.columns = ((columns + p.parts - 1) / p.parts + kCols - 1) / kCols * kCols;
  p.parts = (columns + p.columns - 1) / p.columns;
  p.local = p.parts == 1;
  return p;
}

int64_t stats_bytes(const LogprobArgs& a, const Plan& p) {
  return ((int64_t)a.rows * p.parts * (int64_t)sizeof(Stat) + 15) / 16 * 16;
}

template <bool BF16>
void launch(const LogprobArgs& a, const Plan& p, hipStream_t stream) {
  if (p.local) {
    logprob_part_kernel<BF16, true><<<dim3(1, a.rows), 64 * kWaves, 0, stream>>>(a, p);
    return;
  }
  logprob_part_kernel<BF16, false><<<dim3(p.parts, a.rows), 64 * kWaves, 0, stream>>>(a, p);
  if (p.blocks <= kLocalBlocks) logprob_row_kernel<BF16, true><<<a.rows, 64 * kWaves, 0, stream>>>(a, p);
  else logprob_row_kernel<BF16, false><<<a.rows, 64 * kWaves, 0, stream>>>(a, p);
}

}  // namespace

int64_t token_logprobs_workspace_bytes(const LogprobArgs& a) {
  const Plan p = plan_of(a);
  return p.local ? 16 : stats_bytes(a, p) + (a.top > 0 ? (int64_t)a.rows * p.blocks * 4 : 0);
}

hipError_t launch_token_logprobs(const LogprobArgs& a, hipStream_t stream) {
  Plan p = plan_of(a);
  p.stats = static_cast<Stat*>(a.workspace);
  p.maxima = reinterpret_cast<uint32_t*>(static_cast<char*>(a.workspace) + stats_bytes(a, p));
  if (a.bf16) launch<true>(a, p, stream);
  else launch<false>(a, p, stream);
  return hipGetLastError();
}

}  // namespace nvfp4
