// Attention of a step's nodes over the paged FP8 KV cache.
//
// The page "TensorRT Edge-LLM Completes the MLPerf Edge Agentic Benchmark
// 6.4x Faster on Jetson AGX Thor" verifies a 16-node tree of drafted tokens in
// one pass over an FP8 cache of up to 23.5K tokens (sections "Using tree-based
// multi-token prediction to accelerate LLM inference", "Using NVFP4
// quantization to accelerate Qwen3.6-27B inference") and prefills the suffix
// of a turn over its reused prefix ("Reusing KV cache across agent turns").
//
// Mathematics.  For a row (node v, query head) z_t = c * sum_d q_d k_td in
// exponent units of 2 (c = sm_scale * k_scale * log2 e), p_t = 2^(z_t - m), out
// = v_scale * sum_t p_t v_t / sum_t p_t.  Any m gives the same quotient, so m
// follows the running maximum lazily: p is held as 2^(z + lift), lift = 7 - m (one
// rounded number, which the sums are scaled by exactly), and only when
// the sum of a lane's eight p, which the softmax needs anyway, exceeds 2^15 (a
// score is 5 to 8 above m, or more) does m move up to the maximum, the sums are
// rescaled and the eight are taken again.  So p stays inside f16's range, normal
// down to 2^-21 of the largest, and no maximum is taken in an ordinary step.  z +
// lift is one fused operation, c * s unrounded, while lift holds m rounded: past
// 2^24 that alone would move p by more than f16 has room for, so from there on z is
// rounded as well, and the largest p is 1 to 2^8 whatever the scores are.
//
// Work.  The rows that share a KV head (nodes x group) are packed into tiles
// of 16.  A workgroup has 8 waves in RG groups of rows; a wave holds up to RT row
// tiles and takes 32 tokens of a key tile of 32 * 8 / RG, which it loads straight
// from memory to registers and converts itself, so the loop has no barrier.  An
// item is RG * RT row tiles of one (sequence, KV head); RG is 1 where all rows
// fit, so that every cache byte is loaded and converted once (the rule for more rows
// stands at row_split).  The items of all heads, each a set-up cost and its key tiles, form one
// list that is cut into equal ranges over a fixed grid: long and short sequences
// of a batch share the chip evenly, and a range that cuts an item leaves a partial
// sum (at most two per workgroup) that a second kernel joins.
//
// Bounds.  Times are those of a call on the device, both kernels, one call after
// the other in a graph.  One query per KV head and long sequences: the cache's
// bytes (64 x 8000 tokens, 8 heads of 128, 1.05 GB: 183 us, 5.7 TB/s).  Many rows:
// the vector and the matrix instructions, whose times add up here (512 nodes x 40
// heads of 128 after 23040 tokens: 253 to 256 us over five runs, 0.97 PFLOP/s; matrix
// units 49% busy, vector instructions 61%).  One tree or a few sequences: the set-up
// (4.5 us until the first product), 1 us per row tile to join the waves, and the
// second kernel's 4 to 5 (16 nodes x 40 heads after 23552 tokens: 25.9 us, of which
// the cache's 48 MB are 10).
//
// Operands.  Scores are computed transposed (A = keys, B = queries), 16x16x32
// bf16: E4M3 is exact in bf16, and so is a bf16 query.  The result has a
// query's scores in the lanes that need them as the B operand of the second
// product (A = values transposed, f16: E4M3 is exact there too), if that
// product's key order is 4q .. 4q + 3 and 16 + 4q .. for lane group q, which
// the value loads follow; the 2 x 2 byte transposes are v_perm.  fp32 calls
// split q into three bf16 parts and p into two f16 parts.  bf16 calls round p to
// f16 for the product (2^-11, an eighth of the result's own half step; the sum that
// divides takes p as it is): a second part would be another product per value.  It
// moves 7 to 9% of the results across a rounding border, and their error against
// 64 bits by 0.2 to 0.6% of itself.
#include <type_traits>

#include "device_common.h"
#include "kv_launch.h"

namespace nvfp4 {
namespace {

typedef __bf16 bf8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf2_t __attribute__((ext_vector_type(2)));

constexpr int kWaves = 8;              // waves of a workgroup
constexpr float kStart = 1e38f;        // lift before the first score
constexpr float kLift = 7.0f;          // lift is kLift less the running maximum
constexpr float kFar = 16777216.0f;    // a lift past it may be off by more than a half (2^24)
constexpr float kMost = 32768.0f;      // a lane's eight p sum up to no more, so each fits f16

struct Plan {
  int items;       // per KV head: sequences * row tiles
  int row_items;   // items of a sequence
  int rows;        // rows of an item
  int tile;        // tokens of a key tile
  int start;       // what an item's set-up and join cost, in tiles
  int groups;      // workgroups that share the list; 0: one per item, nothing is cut
  int cap;         // tokens a table row covers
  uint32_t magic;  // ceil(2^32 / group), 0 for a group of one
  float* part;     // [2 * groups][rows][dim], then [2 * groups][rows][2]
};

// Node of a row.  The quotient is exact while row * group < 2^32: a group has
// at most 256 heads and a step 65535 nodes.
__device__ __forceinline__ int node_of(const Plan& p, int row) {
  return p.magic ? (int)__umulhi((uint32_t)row, p.magic) : row;
}

// Committed length (negative: unused), nodes and first row of an item.
struct Item {
  int b, len, count, row0;
};

__device__ __forceinline__ Item item_of(const KvAttentionArgs& a, const Plan& p, int it) {
  Item x;
  x.b = p.row_items == 1 ? it : it / p.row_items;
  x.row0 = (it - x.b * p.row_items) * p.rows;
  const int len = a.c.lens[x.b];
  x.len = len < (1 << 30) ? len : 1 << 30;  // no table covers more
  int n = a.counts ? a.counts[x.b] : a.nodes;
  n = n < a.nodes ? n : a.nodes;
  x.count = n > 0 && x.len >= 0 ? n : 0;
  return x;
}

// Tokens the item's rows may see: 0 .. end - 1.
__device__ __forceinline__ int item_end(const KvAttentionArgs& a, const Plan& p, const Item& x) {
  if (x.row0 >= x.count * a.group) return 0;
  int last = x.count;
  if (!a.parent) {
    const int n = node_of(p, x.row0 + p.rows - 1) + 1;
    last = n < last ? n : last;
  }
  const int end = x.len + last;
  return end < p.cap ? end : p.cap;
}

__device__ __forceinline__ int tiles_of(const Plan& p, int end) {
  return end > p.tile ? (int)((uint32_t)(end + p.tile - 1) >> (31 - __clz(p.tile))) : 1;
}

// An item's length in the list: its tiles behind `start` places for its set-up.
__device__ __forceinline__ int item_places(const KvAttentionArgs& a, const Plan& p, int it) {
  return p.start + tiles_of(p, item_end(a, p, item_of(a, p, it)));
}

// Sum of the items' places and this thread's exclusive part of it; every thread
// of the workgroup calls it.  Thread t has the items [t * per, (t + 1) * per), or,
// where a wave's lanes hold all items, every wave works out the same by itself
// with lane = item, which saves the barriers here and in find_item (16 ragged fp32
// trees 19.2 -> 18.1 us, 32 ragged sequences of one token 58.2 -> 57.4).
constexpr int kOneWave = 64;

struct Scan {
  int per, before, mine, total;
};

template <int WAVES>
__device__ __forceinline__ Scan scan_items(const KvAttentionArgs& a, const Plan& p, int* sums) {
  const int t = threadIdx.x, lane = t & 63, wave = t >> 6;
  const bool one_wave = p.items <= kOneWave;
  Scan s;
  s.per = one_wave ? 1 : (p.items + 64 * WAVES - 1) / (64 * WAVES);
  s.mine = 0;
  for (int i = 0; i < s.per; ++i) {
    const int it = (one_wave ? lane : t) * s.per + i;
    if (it < p.items) s.mine += item_places(a, p, it);
  }
  int v = s.mine;
  for (int off = 1; off < 64; off <<= 1) {
    const int o = __shfl_up(v, off);
    v += lane >= off ? o : 0;
  }
  s.before = v - s.mine;
  if (one_wave) {
    s.total = __builtin_amdgcn_readlane(v, 63);
    return s;
  }
  if (lane == 63) sums[wave] = v;
  __syncthreads();
  s.total = 0;
  for (int w = 0; w < WAVES; ++w) {
    const int x = sums[w];
    s.before += w < wave ? x : 0;
    s.total += x;
  }
  s.total = __builtin_amdgcn_readfirstlane(s.total);
  return s;
}

// floor(x / y) for x < 2^53: the rounded quotient is at most one too large.
__device__ __forceinline__ int divide(uint64_t x, uint32_t y) {
  const uint32_t q = (uint32_t)((double)x / (double)y);
  return __builtin_amdgcn_readfirstlane((int)(x < (uint64_t)q * y ? q - 1 : q));
}

// The list of all heads' items, place by place: range g of n begins at place
// floor(g * all / n), so that ranges and equal items stay aligned.
__device__ __forceinline__ int range_begin(int g, int all, int n) { return divide((uint64_t)g * (uint32_t)all, n); }

// The range that holds place y: the last that begins at or before it, g * all <
// (y + 1) * n.
__device__ __forceinline__ int range_of(int y, int all, int n) {
  return divide((uint64_t)(uint32_t)(y + 1) * (uint32_t)n - 1, all);
}

// The item with place `at` of one head's list, and the places of the list before
// it.
struct Place {
  int it, before;
};

__device__ __forceinline__ Place find_item(const KvAttentionArgs& a, const Plan& p, const Scan& s, int at, int* found) {
  if (p.items <= kOneWave) {
    const uint64_t here = __ballot(s.before <= at && at < s.before + s.mine);
    const int it = here ? __builtin_ctzll(here) : 0;
    return {it, __builtin_amdgcn_readlane(s.before, it)};
  }
  const int t = threadIdx.x;
  int x = s.before;
  for (int i = 0; i < s.per && x <= at; ++i) {
    const int it = t * s.per + i;
    if (it >= p.items) break;
    const int n = item_places(a, p, it);
    if (at < x + n) {
      found[0] = it;
      found[1] = x;
    }
    x += n;
  }
  __syncthreads();
  return {__builtin_amdgcn_readfirstlane(found[0]), __builtin_amdgcn_readfirstlane(found[1])};
}

// Ancestor-or-self bits of node v of a tree of at most 64 nodes, lane = node:
// parent pointers doubled six times.  A parent outside [0, v) makes v a root.
__device__ __forceinline__ uint64_t ancestors_of_wave(int par) {
  const int lane = threadIdx.x & 63;
  uint64_t mask = 1ull << lane;
  int p = par >= 0 && par < lane ? par : -1;
#pragma unroll
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

// The thread's index, computed anew where it is called: what derives from it is
// not kept in registers over the loop.
__device__ __forceinline__ int fresh_thread() {
  int t = threadIdx.x;
  asm volatile("" : "+v"(t));
  return t;
}

template <int N>
struct Words {
  uint32_t w[N];
};

// One wave's 32 tokens of a key tile, as loaded.  Each half is refilled as soon
// as its product has read it, so no second buffer is needed.
template <int D>
struct KeyTile {
  u4_t k[2][D / 64];          // block kb, 64-byte chunk: token lane % 16, bytes 16 (lane / 16) ..
  Words<D / 64> v[8];         // token 16 (e / 4) + 4 (lane / 16) + e % 4, bytes (D / 16) (lane % 16) ..
};

template <int N>
__device__ __forceinline__ Words<N> load_words(const uint8_t* p) {
  Words<N> r;
  if constexpr (N == 1) {
    r.w[0] = *reinterpret_cast<const uint32_t*>(p);
  } else if constexpr (N == 2) {
    const u2_t x = *reinterpret_cast<const u2_t*>(p);
    r.w[0] = x.x;
    r.w[1] = x.y;
  } else {
    const u4_t x = *reinterpret_cast<const u4_t*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) r.w[i] = x[i];
  }
  return r;
}

// Page table entries are read through the scalar cache: a wave-uniform vector
// load would be waited for together with every key and value load before it.
typedef const int32_t __attribute__((address_space(4))) * table_ptr;

// Table entries of the two 16-token blocks at a token (wave-uniform), fetched a
// step before they are used.
struct Entries {
  int page[2];
};

__device__ __forceinline__ int entry_at(const KvAttentionArgs& a, table_ptr row, int pos) {
  const int at = pos >> a.c.page_shift;
  const int p = row[at < a.c.width ? at : a.c.width - 1];
  return at < a.c.width ? p : -1;
}

__device__ __forceinline__ Entries fetch_entries(const KvAttentionArgs& a, table_ptr row, int key) {
  Entries e;
  e.page[0] = entry_at(a, row, key);
  e.page[1] = a.c.page_shift >= 5 ? e.page[0] : entry_at(a, row, key + 16);
  return e;
}

// Where the blocks stand; one whose page does not exist is read from page 0 and
// masked.
struct Blocks {
  uint64_t at[2];
  bool there[2];
};

__device__ __forceinline__ Blocks find_blocks(const KvAttentionArgs& a, const Entries& e, int h, int key) {
  Blocks b;
  const uint32_t shift = a.c.page_shift, pages = a.c.pages, slots = (1u << shift) - 1;
#pragma unroll
  for (int kb = 0; kb < 2; ++kb) {
    const uint32_t p = e.page[kb];  // a negative entry is past the pages, too
    b.there[kb] = p < pages;
    b.at[kb] = (uint64_t)(b.there[kb] ? p : 0u) * (uint32_t)a.c.page_stride +
               (((uint32_t)h << shift) + ((uint32_t)(key + 16 * kb) & slots)) * (uint32_t)a.c.dim;
  }
  return b;
}

// `lanes` is all ones, or zero for a load that is not needed: the loop issues
// the same loads in every step, so that the wait for one kind never includes
// the other, and an unneeded one reads a single line.
template <int D>
__device__ __forceinline__ void load_keys(const KvAttentionArgs& a, const Blocks& b, uint32_t lanes, KeyTile<D>& t) {
  const uint32_t lane = threadIdx.x & 63, off = ((lane & 15) * D + 16 * (lane >> 4)) & lanes;
#pragma unroll
  for (int kb = 0; kb < 2; ++kb)
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      t.k[kb][c] = *reinterpret_cast<const u4_t*>(a.c.k + b.at[kb] + (off + 64 * c));
}

template <int D>
__device__ __forceinline__ void load_values(const KvAttentionArgs& a, const Blocks& b, uint32_t lanes,
                                            KeyTile<D>& t) {
  const uint32_t lane = threadIdx.x & 63, off = (4 * (lane >> 4) * D + (D / 16) * (lane & 15)) & lanes;
#pragma unroll
  for (int kb = 0; kb < 2; ++kb)
#pragma unroll
    for (int e = 0; e < 4; ++e) t.v[4 * kb + e] = load_words<D / 64>(a.c.v + b.at[kb] + (off + e * D));
}

// Eight E4M3 bytes (two words) -> eight bf16, exact.
__device__ __forceinline__ bf8_t to_bf16x8(uint32_t lo, uint32_t hi) {
  const bf2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, false);
  const bf2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(lo, 1.0f, true);
  const bf2_t c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, false);
  const bf2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(hi, 1.0f, true);
  return bf8_t{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

// Four words of E4M3 byte pairs (half `hi` of each) -> eight f16, exact.
template <bool HI>
__device__ __forceinline__ h8_t to_f16x8(const uint32_t (&w)[4]) {
  const h2_t a = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[0], 1.0f, HI);
  const h2_t b = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[1], 1.0f, HI);
  const h2_t c = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[2], 1.0f, HI);
  const h2_t d = __builtin_amdgcn_cvt_scalef32_pk_f16_fp8(w[3], 1.0f, HI);
  return h8_t{a.x, a.y, b.x, b.y, c.x, c.y, d.x, d.y};
}

__device__ __forceinline__ f4_t mfma_bf16(bf8_t a, bf8_t b, f4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

template <int D, int RT, int RG, bool F32>
struct Smem {
  union {
    bf8_t q[F32 ? 3 : 1][RG * RT][D / 32][64];  // queries in operand order: value 64 (s / 2) + 16 (lane / 16) + 8 (s % 2)
                                           // + e of row lane % 16
    float o[kWaves][16][D + 4];            // one row tile of the waves' sums (rows padded by 16 bytes)
  };
  float lift[kWaves][16 * RT], l[kWaves][16 * RT];
  uint64_t line[16 * RG * RT];       // what a row sees of the nodes: bits (trees), or its node (chains)
  int sums[kWaves], found[2];
};

template <int RT, int NT>
struct Sums {
  f4_t o[RT][NT];
  float lift[RT], l[RT];
};

// Barrier for what is passed through LDS: unlike __syncthreads it does not wait
// for the workgroup's loads and stores in memory.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// A value that is alike in all lanes, without a vector register.
__device__ __forceinline__ float uniform(float x) {
  return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(x)));
}

// Nothing is moved across: without it the compiler converts all operands early
// and runs out of registers.
__device__ __forceinline__ void fence() { __builtin_amdgcn_sched_barrier(0); }

// Scores of a wave's 32 tokens against its row tiles r0 .. r0 + RT - 1: their
// sum over the 32 values of step s.  Where they fit (kAhead), the query operands
// of step s are in `ahead`, and those of the next one are fetched to it before
// the products (3% of a step: the LDS latency shows otherwise).
template <int RT, bool F32>
constexpr bool kAhead = !F32 && RT <= 4;

template <int NR, int D, int RT, int RG, bool F32>
__device__ __forceinline__ void score(const Smem<D, RT, RG, F32>& sm, const KeyTile<D>& kt, int r0, int s,
                                      bf8_t (&ahead)[RT], f4_t (&z)[2][RT]) {
  const int lane = threadIdx.x & 63;
  bf8_t kop[2], now[RT];
  if constexpr (kAhead<RT, F32>) {
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      now[r] = ahead[r];
      if (s + 1 < D / 32) ahead[r] = sm.q[0][r0 + r][s + 1][lane];
    }
  }
#pragma unroll
  for (int kb = 0; kb < 2; ++kb) {
    const u4_t w = kt.k[kb][s >> 1];
    kop[kb] = (s & 1) ? to_bf16x8(w.z, w.w) : to_bf16x8(w.x, w.y);
  }
#pragma unroll
  for (int n = F32 ? 2 : 0; n >= 0; --n)  // small parts first
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      if constexpr (!kAhead<RT, F32>) now[r] = sm.q[n][r0 + r][s][lane];
#pragma unroll
      for (int kb = 0; kb < 2; ++kb)
        z[kb][r] = mfma_bf16(kop[kb], now[r], s == 0 && n == (F32 ? 2 : 0) ? f4_t{0.0f, 0.0f, 0.0f, 0.0f} : z[kb][r]);
    }
}

// Scores of tokens that a row does not see become -infinity, and the values of
// tokens that nobody sees, which may be anything, zero.  The lane's four tokens
// of block kb are the nodes u .. u + 3 (negative: committed tokens).
template <int NR, int D, int RT, int RG, bool F32>
__device__ __forceinline__ void mask(const KvAttentionArgs& a, const Smem<D, RT, RG, F32>& sm, KeyTile<D>& kt,
                                     int r0, f4_t (&z)[2][RT], int key0, const Item& x, const Blocks& here) {
  const int lane = fresh_thread() & 63, j = lane & 15, q4 = lane >> 4;
#pragma unroll
  for (int kb = 0; kb < 2; ++kb) {
    const int u = key0 + 16 * kb + 4 * q4 - x.len;
    int have = here.there[kb] ? x.count - u : 0;  // how many of the four anybody sees
    have = have < 0 ? 0 : have < 4 ? have : 4;
    const uint32_t some = (1u << have) - 1;
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const uint32_t keep = (uint32_t)__builtin_amdgcn_sbfe((int)some, e, 1);
#pragma unroll
      for (int n = 0; n < D / 64; ++n) kt.v[4 * kb + e].w[n] &= keep;
    }
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      const uint64_t line = sm.line[16 * (r0 + r) + j];
      uint32_t seen;  // of the four: bits 0 .. 3
      if (a.parent) {
        const uint32_t ahead = u < 0 ? (uint32_t)(line << (-u & 3)) | ((1u << (-u & 3)) - 1) : (uint32_t)(line >> (u & 63));
        seen = u < -3 ? 15u : u < 64 ? ahead : 0u;
      } else {
        int n = (int)line + 1 - u;  // nodes 0 .. the row's own
        n = n < 0 ? 0 : n < 4 ? n : 4;
        seen = (1u << n) - 1;
      }
      seen &= some;
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const uint32_t keep = (uint32_t)__builtin_amdgcn_sbfe((int)seen, e, 1);
        const uint32_t bits = __float_as_uint(z[kb][r][e]);
        z[kb][r][e] = __uint_as_float((bits & keep) | (0xFF800000u & ~keep));
      }
      fence();
    }
  }
}

// NaN codes among the values of a masked tile reach the rows that see their
// tokens and no other (0 * NaN would): they are taken out of the values, and the
// sums that one belongs to are set to NaN, found by the product of the codes' places with
// what the rows see.
template <int NR, int D, int RT>
__device__ __forceinline__ void spread_nans(KeyTile<D>& kt, const f4_t (&z)[2][RT], Sums<RT, D / 16>& acc) {
  uint32_t any = 0;
#pragma unroll
  for (int e = 0; e < 8; ++e)
#pragma unroll
    for (int n = 0; n < D / 64; ++n) any |= (kt.v[e].w[n] & 0x7F7F7F7Fu) + 0x01010101u;
  if (!__any((any & 0x80808080u) != 0)) return;
#pragma unroll
  for (int n = 0; n < D / 64; ++n) {
    uint32_t one[8];  // E4M3 ones in the codes' places
#pragma unroll
    for (int e = 0; e < 8; ++e) {
      const uint32_t nan = ((kt.v[e].w[n] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
      one[e] = nan >> 2 | nan >> 3 | nan >> 4;
      kt.v[e].w[n] &= ~(nan | (nan - (nan >> 7)));
    }
#pragma unroll
    for (int u = 0; u < 4; ++u) {
      uint32_t pair[4];
#pragma unroll
      for (int e = 0; e < 4; ++e)
        pair[e] = __builtin_amdgcn_perm(one[2 * e + 1], one[2 * e], u < 2 ? 0x05010400u : 0x07030602u);
      const h8_t places = u & 1 ? to_f16x8<true>(pair) : to_f16x8<false>(pair);
#pragma unroll
      for (int r = 0; r < NR; ++r) {
        h8_t seen;
#pragma unroll
        for (int e = 0; e < 8; ++e) seen[e] = z[e >> 2][r][e & 3] == -__builtin_inff() ? (_Float16)0.0f : (_Float16)1.0f;
        const f4_t hits = mfma16x16x32(places, seen, f4_t{0.0f, 0.0f, 0.0f, 0.0f});
#pragma unroll
        for (int e = 0; e < 4; ++e)
          acc.o[r][4 * n + u][e] = hits[e] > 0.0f ? __builtin_nanf("") : acc.o[r][4 * n + u][e];
        fence();
      }
    }
  }
}

// Scores in exponent units, rounded (a masked one stays -infinity).
template <int NR, int RT>
__device__ __forceinline__ void scale(f4_t (&z)[2][RT], float c) {
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    z[0][r] *= c;
    z[1][r] *= c;
  }
}

// Moves the running maxima to the largest score so far; whether one of them is
// past kFar now.
template <int NR, int RT, int NT>
__device__ __forceinline__ bool raise(const f4_t (&z)[2][RT], Sums<RT, NT>& acc, float c) {
  bool far = false;
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    float x = __builtin_fmaxf(__builtin_fmaxf(__builtin_fmaxf(z[0][r][0], z[0][r][1]),
                                              __builtin_fmaxf(z[0][r][2], z[0][r][3])),
                              __builtin_fmaxf(__builtin_fmaxf(z[1][r][0], z[1][r][1]),
                                              __builtin_fmaxf(z[1][r][2], z[1][r][3]))) * c;
    x = __builtin_fmaxf(x, __shfl_xor(x, 16));
    x = __builtin_fmaxf(x, __shfl_xor(x, 32));
    x = __builtin_fminf(acc.lift[r], kLift - x);
    const float f = __builtin_amdgcn_exp2f(x - acc.lift[r]);
    acc.lift[r] = x;
    acc.l[r] *= f;
    far |= __builtin_fabsf(x) > kFar && x != kStart;
#pragma unroll
    for (int n = 0; n < NT; ++n) acc.o[r][n] *= f;
    fence();
  }
  return __any(far);
}

// Softmax of the scores; the lane's sums of p, by row tile, in `sum`.
template <int NR, bool F32, int NT, int RT>
__device__ __forceinline__ void weigh(const f4_t (&z)[2][RT], const Sums<RT, NT>& acc, float c, h8_t (&ph)[RT],
                                      h8_t (&pl)[F32 ? RT : 1], float (&sum)[RT]) {
#pragma unroll
  for (int r = 0; r < NR; ++r) {
    const float lift = acc.lift[r];
    float p[8];
#pragma unroll
    for (int e = 0; e < 8; ++e) p[e] = __builtin_amdgcn_exp2f(__builtin_fmaf(z[e >> 2][r][e & 3], c, lift));
#pragma unroll
    for (int e = 0; e < 8; e += 2) {
      const h2_t y = {(_Float16)p[e], (_Float16)p[e + 1]};
      ph[r][e] = y.x;
      ph[r][e + 1] = y.y;
      if constexpr (F32) {
        pl[r][e] = (_Float16)(p[e] - (float)y.x);
        pl[r][e + 1] = (_Float16)(p[e + 1] - (float)y.y);
      }
    }
    sum[r] = ((p[0] + p[1]) + (p[2] + p[3])) + ((p[4] + p[5]) + (p[6] + p[7]));
    if (r & 1) fence();
  }
}

// O += V^T P for word n of the tokens' bytes: it holds d = (D / 16) i + 4 n ..
template <int NR, bool F32, int D, int RT>
__device__ __forceinline__ void accumulate(const KeyTile<D>& kt, int n, const h8_t (&ph)[RT],
                                           const h8_t (&pl)[F32 ? RT : 1], Sums<RT, D / 16>& acc) {
  uint32_t lo[4], hi[4];
#pragma unroll
  for (int e = 0; e < 4; ++e) {
    lo[e] = __builtin_amdgcn_perm(kt.v[2 * e + 1].w[n], kt.v[2 * e].w[n], 0x05010400u);
    hi[e] = __builtin_amdgcn_perm(kt.v[2 * e + 1].w[n], kt.v[2 * e].w[n], 0x07030602u);
  }
#pragma unroll
  for (int u = 0; u < 4; ++u) {
    const h8_t vop = u == 0 ? to_f16x8<false>(lo) : u == 1 ? to_f16x8<true>(lo)
                   : u == 2 ? to_f16x8<false>(hi) : to_f16x8<true>(hi);
#pragma unroll
    for (int r = 0; r < NR; ++r) {
      if constexpr (F32) acc.o[r][4 * n + u] = mfma16x16x32(vop, pl[r], acc.o[r][4 * n + u]);
      acc.o[r][4 * n + u] = mfma16x16x32(vop, ph[r], acc.o[r][4 * n + u]);
    }
  }
}

// One workgroup a CU, two waves a SIMD: with up to 256 registers the matrix
// instructions keep their sums in ordinary ones.  The kernels of one row tile fit
// in half, but two workgroups a CU are slower (64 x 8000 tokens, 8 queries a head:
// 194 us against 191; 16 trees of 16 over 8000: 60.9 against 57.8).
constexpr int kWavesPerSimd = 2;

template <int D, int RT, int RG, bool F32>
__global__ __launch_bounds__(64 * kWaves, kWavesPerSimd) void kv_attention_kernel(KvAttentionArgs a,
                                                                                          Plan plan) {
  constexpr int R = 16 * RT * RG, KS = D / 32, NT = D / 16, KW = kWaves / RG, TILE = 32 * KW;
  __shared__ Smem<D, RT, RG, F32> sm;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int kw = wave % KW;  // which 32 tokens of a tile
  const int rows_all = a.nodes * a.group;
  const float c0 = a.sm_scale * *a.k_scale * 1.44269504088896340736f;
  // not 0, infinite or NaN: a masked score stays -infinity.  Where k_scale gives none, the sums of the rows that
  // see something (theirs are not 0) become NaN.
  const float c = __builtin_isfinite(c0) ? __builtin_fmaxf(__builtin_fabsf(c0), 1.17549435e-38f) : 1.0f;
  const float spoil = __builtin_isfinite(c0) ? 0.0f : __builtin_nanf("");
  const bool flip = c0 < 0.0f;
  const float vs = *a.v_scale;

  // This workgroup's range of the list.
  int h, it, at, left;  // head, item, first place within it, places to do
  int group = 0;
  if (plan.groups == 0) {
    h = blockIdx.x / plan.items;
    it = blockIdx.x - h * plan.items;
    at = 0;
    left = item_places(a, plan, it);
  } else {
    Scan s;
    if (plan.items == 1) s.total = item_places(a, plan, 0);
    else s = scan_items<kWaves>(a, plan, sm.sums);
    const int all = s.total * a.c.heads, n = plan.groups < all ? plan.groups : all;
    group = blockIdx.x;
    if (group >= n) return;
    const int begin = range_begin(group, all, n);
    left = range_begin(group + 1, all, n) - begin;
    h = divide((uint32_t)begin, s.total);
    at = begin - h * s.total;
    it = 0;
    if (plan.items > 1) {
      const Place x = find_item(a, plan, s, at, sm.found);
      it = x.it;
      at -= x.before;
    }
  }

  bool first_item = true;
  while (left > 0) {
    const Item x = item_of(a, plan, it);
    const int end = item_end(a, plan, x);
    const int tiles = tiles_of(plan, end);
    const int past = at + left - plan.start;
    const int t0 = at > plan.start ? at - plan.start : 0, t1 = past < tiles ? past : tiles;
    if (t1 <= t0) break;  // the range ends in the item's set-up
    // Tokens before it are seen by every row: the committed ones, and in a chain the first row's.
    int clear = x.len + (a.parent ? 0 : node_of(plan, x.row0) + 1);
    clear = clear < end ? clear : end;

    // The item's row tiles in use are shared out evenly over the row groups.
    int used = (rows_all - x.row0 + 15) / 16;
    used = used < RG * RT ? used : RG * RT;
    const int r0 = wave / KW * used / RG, mine = (wave / KW + 1) * used / RG - r0;

    const int t = fresh_thread(), lane = t & 63, j = lane & 15, q4 = lane >> 4;
    // The queries, one operand of one row tile at a time, all loads first.
    constexpr int FRAGS = RG * RT * KS, PER_WAVE = (FRAGS + kWaves - 1) / kWaves, NV = F32 ? 2 : 1;
    u4_t raw[PER_WAVE][NV];
#pragma unroll
    for (int i = 0; i < PER_WAVE; ++i) {
      const int f = i * kWaves + wave < FRAGS ? i * kWaves + wave : FRAGS - 1;
      const int s = f % KS;
      int row = x.row0 + 16 * (f / KS) + j;
      row = row < rows_all ? row : rows_all - 1;
      const int node = node_of(plan, row);
      const int64_t off = ((int64_t)x.b * a.nodes + node) * a.q_stride +
                          (h * a.group + (row - node * a.group)) * D + 16 * q4 + 64 * (s >> 1) + 8 * (s & 1);
      const u4_t* from = reinterpret_cast<const u4_t*>(static_cast<const char*>(a.q) + off * (F32 ? 4 : 2));
#pragma unroll
      for (int v = 0; v < NV; ++v) raw[i][v] = from[v];
    }
    const table_ptr pages = (table_ptr)(uintptr_t)(a.c.table + (int64_t)x.b * a.c.width);
    KeyTile<D> kt;
    int key0 = t0 * TILE + 32 * kw;
    Entries entries = fetch_entries(a, pages, key0);
    Blocks here = find_blocks(a, entries, h, key0);
    load_keys<D>(a, here, ~0u, kt);
    load_values<D>(a, here, ~0u, kt);
    entries = fetch_entries(a, pages, key0 + TILE);

    int par = -1;
    if (a.parent && wave == 0 && lane < a.nodes) par = a.parent[(int64_t)x.b * a.nodes + lane];
    if (!first_item) __syncthreads();  // the last item's sums have been read
    first_item = false;
    if (wave == 0) {
      const uint64_t tree = a.parent ? ancestors_of_wave(par) : 0;
#pragma unroll
      for (int i = 0; i < (R + 63) / 64; ++i) {
        int row = x.row0 + 64 * i + lane;
        row = row < rows_all ? row : rows_all - 1;
        const int node = node_of(plan, row);
        const uint64_t bits = __shfl(tree, node & 63);
        if (64 * i + lane < R) sm.line[64 * i + lane] = a.parent ? bits : (uint64_t)node;
      }
    }
#pragma unroll
    for (int i = 0; i < PER_WAVE; ++i) {
      const int f = i * kWaves + wave;
      if (f >= FRAGS) continue;
      const int r = f / KS, s = f % KS;
      if constexpr (F32) {
        bf8_t part[3];
#pragma unroll
        for (int e = 0; e < 8; ++e) {
          float y = __uint_as_float(raw[i][e >> 2][e & 3]);
          y = flip ? -y : y;
#pragma unroll
          for (int n = 0; n < 3; ++n) {
            const __bf16 b = (__bf16)y;
            part[n][e] = b;
            y -= (float)b;
          }
        }
#pragma unroll
        for (int n = 0; n < 3; ++n) sm.q[n][r][s][lane] = part[n];
      } else {
        u4_t w = raw[i][0];
        if (flip) w ^= 0x80008000u;
        sm.q[0][r][s][lane] = __builtin_bit_cast(bf8_t, w);
      }
    }
    __syncthreads();

    Sums<RT, NT> acc;
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      acc.lift[r] = kStart;
      acc.l[r] = 0.0f;
#pragma unroll
      for (int n = 0; n < NT; ++n) acc.o[r][n] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
    }
    // NR: the row tiles that the wave works on.
    auto walk = [&](auto nr) {
      constexpr int NR = decltype(nr)::value;
      float cz = uniform(c);      // the factor that the scores have left
      bool far = false;
      for (int tile = t0; tile < t1; ++tile) {
        const uint32_t more = tile + 1 < t1 ? ~0u : 0u;
        // A SIMD's two waves take turns to go first: left alone the older one does, and the younger one
        // works on by itself at the end.
        if ((tile ^ (wave >> 2)) & 1) __builtin_amdgcn_s_setprio(1);
        else __builtin_amdgcn_s_setprio(0);
        asm volatile("" ::: "memory");  // the queries are read again from LDS: kept in registers they would spill
        f4_t z[2][RT];
        bf8_t ahead[RT];
        if constexpr (kAhead<RT, F32>) {
#pragma unroll
          for (int r = 0; r < NR; ++r) ahead[r] = sm.q[0][r0 + r][0][threadIdx.x & 63];
        }
#pragma unroll
        for (int s = 0; s < KS; ++s) {
          score<NR>(sm, kt, r0, s, ahead, z);
          fence();
        }
        if (key0 + 32 > clear || !here.there[0] || !here.there[1]) {
          mask<NR>(a, sm, kt, r0, z, key0, x, here);
          spread_nans<NR>(kt, z, acc);
        }
        const Blocks next = find_blocks(a, entries, h, key0 + TILE);
        load_keys<D>(a, next, more, kt);
        entries = fetch_entries(a, pages, key0 + 2 * TILE);
        // Moves the maxima.  From the first one past kFar on the scores are rounded as the maxima are.
        auto up = [&] {
          if (!raise<NR>(z, acc, cz) || far) return;
          scale<NR>(z, cz);
          cz = 1.0f;
          far = true;
        };
        if (far) scale<NR>(z, uniform(c));
        if (tile == t0) up();
        h8_t ph[RT], pl[F32 ? RT : 1];
        float sum[RT];
        weigh<NR, F32>(z, acc, cz, ph, pl, sum);
        float most = sum[0];
#pragma unroll
        for (int r = 1; r < NR; ++r) most = __builtin_fmaxf(most, sum[r]);
        fence();
        if (__any(most > kMost)) {
          up();
          weigh<NR, F32>(z, acc, cz, ph, pl, sum);
          fence();
        }
#pragma unroll
        for (int r = 0; r < NR; ++r) acc.l[r] += sum[r];
        fence();
#pragma unroll
        for (int n = 0; n < D / 64; ++n) {
          accumulate<NR, F32>(kt, n, ph, pl, acc);
          fence();
        }
        load_values<D>(a, next, more, kt);
        here = next;
        key0 += TILE;
      }
    };
    if (RT == 1 || mine == RT) walk(std::integral_constant<int, RT>{});
    else walk(std::integral_constant<int, RT == 1 ? 1 : RT - 1>{});
    __builtin_amdgcn_s_setprio(0);

    // Join the waves, one row tile at a time.
    const int te = fresh_thread(), le = te & 63, je = le & 15, qe = le >> 4;
    const bool whole = t0 == 0 && t1 == tiles;
    const int slot = 2 * group + (t0 == 0 ? 1 : 0);
#pragma unroll
    for (int r = 0; r < RT; ++r) {
      float l = acc.l[r];
      l += __shfl_xor(l, 16);
      l += __shfl_xor(l, 32);
      if (qe == 0) {
        sm.lift[wave][16 * r + je] = acc.lift[r];
        sm.l[wave][16 * r + je] = l;
      }
    }
    constexpr int THREADS = 64 * KW, PER = 16 * D / THREADS;  // of a row tile, values of a thread
    constexpr int VEC = PER < 4 ? PER : 4, LANES = D / PER;   // values side by side, threads of a row
    typedef float vec_t __attribute__((ext_vector_type(VEC)));
    const int rg = te / THREADS, row16 = te % THREADS / LANES, d0 = VEC * (te % LANES);
    const int first = rg * used / RG, tiles_here = (rg + 1) * used / RG - first;
#pragma nounroll
    for (int r = 0; r < RT; ++r) {
      lds_barrier();
#pragma unroll
      for (int y = 0; y < RT; ++y) {
        if (y != r || r >= mine) continue;
#pragma unroll
        for (int e = 0; e < 4; ++e)
#pragma unroll
          for (int n = 0; n < NT; n += 4)
            *reinterpret_cast<f4_t*>(&sm.o[wave][je][NT * (4 * qe + e) + n]) =
                f4_t{acc.o[y][n][e], acc.o[y][n + 1][e], acc.o[y][n + 2][e], acc.o[y][n + 3][e]};
      }
      lds_barrier();
      const int row = 16 * (first + r) + row16, grow = x.row0 + row;
      if (r >= tiles_here || grow >= rows_all) continue;
      float lifts[KW], low = kStart, sum = 0.0f;
      vec_t y[PER / VEC];
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        lifts[w] = sm.lift[rg * KW + w][16 * r + row16];
        low = __builtin_fminf(low, lifts[w]);
      }
#pragma unroll
      for (int n = 0; n < PER / VEC; ++n) y[n] = 0.0f;
#pragma unroll
      for (int w = 0; w < KW; ++w) {
        const float f = __builtin_amdgcn_exp2f(low - lifts[w]);
        sum += f * sm.l[rg * KW + w][16 * r + row16];
#pragma unroll
        for (int n = 0; n < PER / VEC; ++n)
          y[n] += f * *reinterpret_cast<const vec_t*>(&sm.o[rg * KW + w][row16][d0 + VEC * LANES * n]);
      }
      sum = sum == 0.0f ? 0.0f : sum + spoil;
      if (!whole) {
        const uint32_t at_row = (uint32_t)slot * R + row;
        float* to = plan.part + (uint64_t)at_row * D + d0;
#pragma unroll
        for (int n = 0; n < PER / VEC; ++n) *reinterpret_cast<vec_t*>(to + VEC * LANES * n) = y[n];
        if (d0 == 0)
          *reinterpret_cast<f2_t*>(plan.part + (uint64_t)2 * plan.groups * R * D + (uint64_t)at_row * 2) = f2_t{low, sum};
        continue;
      }
      const int node = node_of(plan, grow);
      const bool live = node < x.count && sum != 0.0f;
      const float f = live ? vs / sum : 0.0f;
      const int64_t orow = ((int64_t)x.b * a.nodes + node) * (a.c.heads * a.group) + h * a.group +
                           (grow - node * a.group);
#pragma unroll
      for (int n = 0; n < PER / VEC; ++n) {
        const int64_t to = orow * D + d0 + VEC * LANES * n;
        const vec_t out = live ? y[n] * f : (vec_t)0.0f;
        if constexpr (F32) {
          *reinterpret_cast<vec_t*>(static_cast<float*>(a.out) + to) = out;
        } else {
          typedef __bf16 half_t __attribute__((ext_vector_type(VEC)));
          *reinterpret_cast<half_t*>(static_cast<uint16_t*>(a.out) + to) = __builtin_convertvector(out, half_t);
        }
      }
      if (a.lse && d0 == 0)
        a.lse[orow] = live ? (__builtin_log2f(sum) - low) * 0.69314718055994530942f : -__builtin_inff();
    }

    // The next item of the list.
    left -= plan.start + tiles - at;
    at = 0;
    if (++it == plan.items) {
      it = 0;
      ++h;
    }
  }
}

// Joins the partial sums of the items that a range boundary cut: block (item,
// or boundary, whichever are fewer; four rows, and every fourth of gridDim.y
// further ones), a wave a row.  Blocks go by items where those are fewer: one
// tree of 80 rows, 8 items: 4.7 us, by its 255 boundaries 10.  Bound by the chain
// of loads that finds the item (3 us where nothing was cut), then by the partial
// sums' bytes (512-node suffix of 40 heads: 16 us for 44 MB).
template <int D, bool F32, bool BY_ITEM>
__global__ __launch_bounds__(256) void kv_attention_join_kernel(KvAttentionArgs a, Plan plan) {
  const int R = plan.rows;
  __shared__ int sums[4], found[2];
  const int t = threadIdx.x, lane = t & 63, wave = __builtin_amdgcn_readfirstlane(t >> 6);
  int h, it = 0, before = 0;  // before: places of the head's list before the item
  Scan s;
  if (plan.items == 1) s.total = item_places(a, plan, 0);
  else s = scan_items<4>(a, plan, sums);
  const int all = s.total * a.c.heads, n = plan.groups < all ? plan.groups : all;
  int boundary = 0;
  if constexpr (BY_ITEM) {
    h = blockIdx.x / plan.items;
    it = blockIdx.x - h * plan.items;
    if (plan.items > kOneWave) {
      if (it / s.per == t) {
        int y = s.before;
        for (int i = t * s.per; i < it; ++i) y += item_places(a, plan, i);
        found[1] = y;
      }
      __syncthreads();
      before = __builtin_amdgcn_readfirstlane(found[1]);
    } else if (plan.items > 1) {
      before = __builtin_amdgcn_readlane(s.before, it);
    }
  } else {
    boundary = blockIdx.x + 1;
    if (boundary >= n) return;
    const int begin = range_begin(boundary, all, n);
    h = divide((uint32_t)begin, s.total);
    if (plan.items > 1) {
      const Place x = find_item(a, plan, s, begin - h * s.total, found);
      it = x.it;
      before = x.before;
    }
  }
  const Item x = item_of(a, plan, it);
  const int tiles = tiles_of(plan, item_end(a, plan, x)), first = h * s.total + before + plan.start;
  const int g0 = range_of(first, all, n), g1 = range_of(first + tiles - 1, all, n);
  // the boundary behind the item's first range joins it, if that range does not hold the item
  if (g0 == g1 || (!BY_ITEM && g0 != boundary - 1)) return;

  const int rows_all = a.nodes * a.group;
  const float* ml = plan.part + (uint64_t)2 * plan.groups * R * D;
  constexpr int N = D / 64;  // values of a lane
  typedef float vec_t __attribute__((ext_vector_type(N)));
  for (int row = blockIdx.y * 4 + wave; row < R && x.row0 + row < rows_all; row += 4 * gridDim.y) {
    const int grow = x.row0 + row;
    float low = kStart, sum = 0.0f;
    vec_t acc = (vec_t)0.0f;
    for (int base = g0; base <= g1; base += 64) {
      // the statistics of up to 64 partial sums, a lane each
      float lift = kStart, l = 0.0f;
      if (base + lane <= g1) {
        const int g = base + lane;
        const f2_t y = *reinterpret_cast<const f2_t*>(ml + ((uint32_t)(2 * g + (g == g0 ? 1 : 0)) * R + row) * 2);
        lift = y.x;
        l = y.y;
      }
      const int many = g1 - base + 1 < 64 ? g1 - base + 1 : 64;
      float f = 0.0f;
      // `fly` sums at a time; their weights are worked out while the first ones arrive
      auto add = [&](auto fly, int k) {
        constexpr int FLY = decltype(fly)::value;
        vec_t y[FLY];
#pragma unroll
        for (int u = 0; u < FLY; ++u) {
          const int g = base + (k + u < many ? k + u : k);
          y[u] = *reinterpret_cast<const vec_t*>(
              plan.part + (uint64_t)((uint32_t)(2 * g + (g == g0 ? 1 : 0)) * R + row) * D + N * lane);
        }
        if (k == 0) {
          float lowest = lift;
          for (int off = 32; off > 0; off >>= 1) lowest = __builtin_fminf(lowest, __shfl_xor(lowest, off));
          lowest = __builtin_fminf(lowest, low);
          const float old = __builtin_amdgcn_exp2f(lowest - low);
          f = __builtin_amdgcn_exp2f(lowest - lift);
          sum = sum * old + f * l;
          acc *= old;
          low = lowest;
        }
#pragma unroll
        for (int u = 0; u < FLY; ++u) {
          const int from = k + u < many ? k + u : 0;
          const float w = __builtin_bit_cast(float, __builtin_amdgcn_readlane(__builtin_bit_cast(int, f), from));
          acc += (k + u < many ? w : 0.0f) * y[u];
        }
      };
      int k = 0;
      for (; k + 16 <= many; k += 16) add(std::integral_constant<int, 16>{}, k);
      for (; k < many; k += 4) add(std::integral_constant<int, 4>{}, k);
    }
    for (int off = 32; off > 0; off >>= 1) sum += __shfl_xor(sum, off);
    const int node = node_of(plan, grow);
    const bool live = node < x.count && sum != 0.0f;
    const float scale = live ? *a.v_scale / sum : 0.0f;
    const int64_t orow = ((int64_t)x.b * a.nodes + node) * (a.c.heads * a.group) + h * a.group + (grow - node * a.group);
#pragma unroll
    for (int i = 0; i < N; ++i) {
      const float y = live ? acc[i] * scale : 0.0f;
      if constexpr (F32) static_cast<float*>(a.out)[orow * D + N * lane + i] = y;
      else static_cast<__bf16*>(a.out)[orow * D + N * lane + i] = (__bf16)y;  // nearest even, NaN stays NaN
    }
    if (a.lse && lane == 0)
      a.lse[orow] = live ? (__builtin_log2f(sum) - low) * 0.69314718055994530942f : -__builtin_inff();
  }
}

int compute_units() {
  static int cus[64] = {0};
  int dev = 0;
  if (hipGetDevice(&dev) != hipSuccess || dev < 0 || dev >= 64) return 256;
  if (cus[dev] == 0) {
    int v = 0;
    if (hipDeviceGetAttribute(&v, hipDeviceAttributeMultiprocessorCount, dev) != hipSuccess || v <= 0) v = 256;
    cus[dev] = v;
  }
  return cus[dev];
}

// A wave holds up to `most` row tiles (a tile's sums take D / 4 registers; fewer
// convert each byte for fewer rows: with 3, 4 and 1 for dimensions 128, 64 and 256
// a 512-node suffix takes 297 us instead of 275, 32 trees of 96 rows of 256 379
// instead of 265).  More rows than that take
//   up to 2 `most`: two groups of rows in a workgroup, which share the key tile
//     (32 trees of 80 rows after 8000 tokens of 8 x 128: 150 us; as two items, each
//     of which reads the cache, 203; one tree after 23552 27.6 and 28.1);
//   up to 4 `most`: further items, as long as the cache that is read again is one
//     that the Infinity Cache holds (one tree of 96 rows after 8000 tokens of 4 x
//     256, 16 MB: 25.9 us; as four groups, whose partial sums have four times the
//     rows, 31.8; 32 of those trees, 524 MB: 292 and 265);
//   beyond: four groups and further items (1024-token prompt 58 us; one group 62).
// The cache's size is taken from the table's width: the tree of 96 rows under a table
// of 160000 tokens takes four groups, 31.0 us instead of 23.9 in a graph.
constexpr int most_row_tiles(int dim, bool f32) {
  return f32 ? (dim == 256 ? 1 : 2) : dim == 64 ? 6 : dim == 128 ? 4 : 2;
}

constexpr int64_t kCached = 256ll << 20;

void row_split(const KvAttentionArgs& a, int* rt, int* rg, int* row_items) {
  const int most = most_row_tiles(a.c.dim, !a.bf16);
  const int all = (int)(((int64_t)a.nodes * a.group + 15) / 16);
  const int64_t cache = 2 * ((int64_t)a.c.seqs * a.c.heads * a.c.dim) * ((int64_t)a.c.width << a.c.page_shift);
  *rg = all <= most ? 1 : all <= 2 * most ? 2 : all <= 4 * most && cache <= kCached ? 1 : 4;
  *row_items = (all + *rg * most - 1) / (*rg * most);
  *rt = (all + *row_items * *rg - 1) / (*row_items * *rg);
}

// Where no sequence can have more than kWhole tiles, none is split: the second
// kernel costs more (one token after 511, 8 heads of 128: 9.9 us split, 7.6 us
// whole).  An item's set-up counts as kStartCost tiles; with 0, 2, 4 and 8 of them
// 16 ragged fp32 trees take 24.0, 20.7, 21.2 and 22.4 us, 32 ragged sequences of
// one bf16 token 62.6, 62.3, 64 and 68.8 us.  Lengths stand on the device, so both
// this rule and row_split's go by what the table covers: under a table of 23552
// tokens the first of these calls is split, 9.0 us instead of 6.9 in a graph.  kWhole
// was measured at two tiles and 8 heads only, its border nowhere.
constexpr int kWhole = 4, kStartCost = 2;

Plan make_plan(const KvAttentionArgs& a, int* rt, int* rg, int64_t* bytes) {
  Plan p;
  row_split(a, rt, rg, &p.row_items);
  p.items = a.c.seqs * p.row_items;
  p.rows = 16 * *rt * *rg;
  p.tile = 32 * kWaves / *rg;
  p.cap = a.c.width << a.c.page_shift;
  p.magic = a.group == 1 ? 0 : (uint32_t)((((uint64_t)1 << 32) + a.group - 1) / a.group);
  p.start = kStartCost;
  const int64_t tiles = ((int64_t)p.cap + p.tile - 1) / p.tile;
  const int64_t most = (int64_t)p.items * a.c.heads * (tiles + p.start);
  const int64_t groups = (int64_t)compute_units() * (4 * kWavesPerSimd / kWaves);
  // too short to cut, or more places than 32 bits count
  p.groups = tiles <= kWhole || most >= ((int64_t)1 << 31) ? 0 : (int)(groups < most ? groups : most);
  *bytes = (int64_t)2 * p.groups * p.rows * (a.c.dim + 2) * 4;
  p.part = nullptr;
  return p;
}

template <int D, int RT, int RG, bool F32>
hipError_t launch_one(const KvAttentionArgs& a, const Plan& p, hipStream_t stream) {
  const int64_t items = (int64_t)p.items * a.c.heads;
  kv_attention_kernel<D, RT, RG, F32><<<(unsigned)(p.groups ? p.groups : items), 64 * kWaves, 0, stream>>>(a, p);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess || p.groups < 2) return e;
  // more workgroups than the chip holds at once would find their item anew for each four rows
  const int joins = items < p.groups ? (int)items : p.groups - 1;
  const int many = (8 * compute_units() + joins - 1) / joins, y = many < p.rows / 4 ? many : p.rows / 4;
  if (items < p.groups) kv_attention_join_kernel<D, F32, true><<<dim3(joins, y), 256, 0, stream>>>(a, p);
  else kv_attention_join_kernel<D, F32, false><<<dim3(joins, y), 256, 0, stream>>>(a, p);
  return hipGetLastError();
}

// RT row tiles a wave, for the numbers of row groups that lead to it.
template <int D, int RT, bool F32>
hipError_t launch_tiles(const KvAttentionArgs& a, const Plan& p, int rt, int rg, hipStream_t stream) {
  constexpr int most = most_row_tiles(D, F32);
  if (rt != RT) {
    if constexpr (RT < most) return launch_tiles<D, RT + 1, F32>(a, p, rt, rg, stream);
    return hipErrorInvalidValue;
  }
  if constexpr (2 * RT > most) {  // more than `most` tiles over the groups
    if (rg == 2) return launch_one<D, RT, 2, F32>(a, p, stream);
    if (rg == 4) return launch_one<D, RT, 4, F32>(a, p, stream);
  }
  return rg == 1 ? launch_one<D, RT, 1, F32>(a, p, stream) : hipErrorInvalidValue;
}

template <int D>
hipError_t launch_dim(const KvAttentionArgs& a, const Plan& p, int rt, int rg, hipStream_t stream) {
  return a.bf16 ? launch_tiles<D, 1, false>(a, p, rt, rg, stream) : launch_tiles<D, 1, true>(a, p, rt, rg, stream);
}

}  // namespace

bool kv_attention_supported(const KvAttentionArgs& a) {
  int rt, rg, row_items;
  row_split(a, &rt, &rg, &row_items);
  return (int64_t)a.c.seqs * row_items * a.c.heads * 64 * kWaves < ((int64_t)1 << 32);  // threads of a launch
}

int64_t kv_attention_workspace_bytes(const KvAttentionArgs& a) {
  int rt, rg;
  int64_t bytes;
  make_plan(a, &rt, &rg, &bytes);
  return bytes;
}

hipError_t launch_kv_attention(const KvAttentionArgs& a, hipStream_t stream) {
  int rt, rg;
  int64_t bytes;
  Plan p = make_plan(a, &rt, &rg, &bytes);
  if (a.workspace_bytes < bytes) p.groups = 0;
  p.part = static_cast<float*>(a.workspace);
  switch (a.c.dim) {
    case 64: return launch_dim<64>(a, p, rt, rg, stream);
    case 128: return launch_dim<128>(a, p, rt, rg, stream);
    default: return launch_dim<256>(a, p, rt, rg, stream);
  }
}

}  // namespace nvfp4
