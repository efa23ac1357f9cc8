// The gated delta rule for a block of tokens at once, on the matrix cores.
//
// Mathematics.  In a block that begins with state S, with G_i the sums of the log
// decays up to token i (along its line in a tree),
//   u_i + beta_i sum_j e^(G_i - G_j) (k_i . k_j) u_j = beta_i (v_i - e^G_i S k_i),
// j the tokens before i (its ancestors): (I + A) u = diag(beta) r with A strictly
// lower triangular.  Once T = (I + A)^-1 diag(beta) is known, a block is five matrix
// products: r = v - e^G (K S), u = T r, o = e^G (Q S) + P u with P_ij = e^(G_i - G_j)
// q_i . k_j, and S <- e^G_end S + K^T diag(e^(G_end - G)) u.  T and P need neither S
// nor v: they are prepared for all blocks at once, and what one block waits for in
// the one before it are the five products alone.
//
// Operands.  A 16x16x32 f16 product wants 8 values of its inner dimension a lane.
// With the inner order 32 s + 4 g .. + 3, 32 s + 16 + 4 g .. + 3 for lane group g, a
// result (rows 4 g .. 4 g + 3 of a tile, one column a lane) is an operand as it
// stands; so it is of four 16x16x4 fp32 products, one for each of its values.  So S, r
// and u stay in the registers of the wave whose columns they are, and everything
// prepared is stored in operand order: one 16-byte load a lane.
//
// Accuracy.  T r and P u add up tokens, between which a decay may stand: a value of
// any size counts as e^(G_i - G_j) leaves it, or not at all beside another branch of a
// tree.  Their factors keep fp32's range: fp32 products in the one-block kernel and in
// T r of a scan by 64 columns, where T's 10 KB count more than the products; else bf16
// parts, three each (24 bits, six products; P and u of bf16 calls two, 16 bits, three).
// A scan waits for T r: 40 fp32 products of 32 cycles there take 27.4 us for 512 tokens,
// 36 bf16 ones of 16 cycles 24.5.  4 sequences of 2,047 tokens, by 64 columns: 428 us in
// parts, 392 in tiles.
// K S and Q S add up a row's values, K^T X what is in a state at one time: there every
// factor on the way to a state keeps 22 bits of its row's or column's largest value, in
// two f16 parts (rounded to nearest, the second the rest of the first), of which the
// product of the two second ones is left out, 2^-22.  A bf16 row of k is exact in one
// part.  f16's least step is 2^-24: rows of k and q are scaled by a power of two to a
// largest value of 1 to 2, and a column of S, with what is added to it, by one to 32
// to 64, so that 64 products fit; values are off by 2^-25 of the one, by 2^-30 of the
// other, at least.
//
// NaN and infinities.  A product of a whole tile adds 0 times what a row does not see.  So
// a token whose k, g or beta is not finite takes part with zeros, a column's values that
// are not are taken as zeros, and what sees either of them is made NaN in the end.  In a
// scan the fetching wave looks at the values, so that no state waits for it: 512 tokens
// 37.3 us with and without, 3 prompts of up to 4,099 fp32 tokens 140 -> 144, 4 of 2,047
// bf16 tokens 356 -> 374.
#pragma once

#include "delta_common.h"
#include "kv_tree.h"

namespace nvfp4 {

typedef _Float16 h4_t __attribute__((ext_vector_type(4)));

// NaN stays.
__device__ __forceinline__ float max4_nan(float m, f4_t x) {
  m = __builtin_elementwise_maximum(__builtin_elementwise_maximum(m, fabsf(x[0])), fabsf(x[1]));
  return __builtin_elementwise_maximum(__builtin_elementwise_maximum(m, fabsf(x[2])), fabsf(x[3]));
}

// Over the four lane groups, in all of them: rows of lanes exchanged in registers.
__device__ __forceinline__ float max_of_groups(float x) {
  typedef uint32_t pair_t __attribute__((ext_vector_type(2)));
  const uint32_t a = __float_as_uint(x);
  const pair_t p = __builtin_bit_cast(pair_t, __builtin_amdgcn_permlane16_swap(a, a, false, false));
  const uint32_t b = __float_as_uint(fmaxf(__uint_as_float(p.x), __uint_as_float(p.y)));
  const pair_t q = __builtin_bit_cast(pair_t, __builtin_amdgcn_permlane32_swap(b, b, false, false));
  return fmaxf(__uint_as_float(q.x), __uint_as_float(q.y));
}

__device__ __forceinline__ h4_t to_half(f4_t x) { return __builtin_convertvector(x, h4_t); }
// x - hi, exact; as a multiply-add it takes hi as it stands, in one instruction
__device__ __forceinline__ f4_t rest_of(f4_t x, h4_t hi) {
  return f4_t{__builtin_fmaf((float)hi[0], -1.0f, x[0]), __builtin_fmaf((float)hi[1], -1.0f, x[1]),
              __builtin_fmaf((float)hi[2], -1.0f, x[2]), __builtin_fmaf((float)hi[3], -1.0f, x[3])};
}
__device__ __forceinline__ h8_t join8(h4_t a, h4_t b) { return __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7); }

// Two result tiles as the operand of a product over their rows, in N bf16 parts: each
// the nearest to what the ones before it leave.
typedef __bf16 b4_t __attribute__((ext_vector_type(4)));
typedef __bf16 b8_t __attribute__((ext_vector_type(8)));

template <int N>
__device__ __forceinline__ void wide_parts(f4_t a, f4_t b, b8_t (&part)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) {
    const b4_t p = __builtin_convertvector(a, b4_t), q = __builtin_convertvector(b, b4_t);
    part[i] = __builtin_shufflevector(p, q, 0, 1, 2, 3, 4, 5, 6, 7);
    a -= __builtin_convertvector(p, f4_t);
    b -= __builtin_convertvector(q, f4_t);
  }
}

__device__ __forceinline__ f4_t mfma16x16x32(b8_t a, b8_t b, f4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_bf16(a, b, c, 0, 0, 0);
}

// Two result tiles as the operand of a product over their rows.
__device__ __forceinline__ h8_t operand_hi(f4_t a, f4_t b) { return join8(to_half(a), to_half(b)); }

__device__ __forceinline__ void operand_parts(f4_t a, f4_t b, h8_t& hi, h8_t& lo) {
  const h4_t p = to_half(a), q = to_half(b);
  hi = join8(p, q);
  lo = join8(to_half(rest_of(a, p)), to_half(rest_of(b, q)));
}

// What is prepared of a block, in units of an operand of one lane (16 bytes).  PARTS:
// f16 parts of rows of k and q.  TILES: T as the fp32 tiles of a lower triangle, row
// after row, instead of three bf16 parts.
template <int DK, bool BF16, int NT, bool TILES = false>
struct BlockOps {
  static constexpr int kParts = BF16 ? 1 : 2;
  static constexpr int kSteps = DK / 32;            // inner steps over dk
  static constexpr int kTokenSteps = (NT + 1) / 2;  // over tokens
  static constexpr int kTiles = NT * (NT + 1) / 2;  // of a lower triangle
  static constexpr int kLower = kTokenSteps * (kTokenSteps + 1) - (NT & 1 ? kTokenSteps : 0);  // steps of its rows
  static constexpr int kRows = NT * kSteps * 64;            // K or Q, one part
  static constexpr int kCols = DK / 16 * kTokenSteps * 64;  // K transposed, one part
  // of a key head: K and its transpose, what a scan's states need, before Q
  static constexpr int kKey = 0, kKeyT = kParts * kRows, kQuery = kKeyT + kParts * kCols;
  static constexpr int kKeyUnits = kQuery + kParts * kRows;
  // of a value head: the factors [3][16 NT], behind them e^G_end, a word of nothing and
  // the tokens that are not finite (64 bits); T, and P in two bf16 parts (bf16 calls) or
  // three
  static constexpr int kPartsOfP = BF16 ? 2 : 3;
  static constexpr int kFactors = 0, kT = (3 * 4 * NT + 1 + 63) / 64 * 64;
  static constexpr int kP = kT + (TILES ? kTiles : 3 * kLower) * 64;
  static constexpr int kHeadUnits = kP + kPartsOfP * kLower * 64;
  // steps of the rows of tile rt begin at this one
  static __device__ constexpr int lower(int rt) { return rt == 0 ? 0 : rt == 1 ? 1 : rt == 2 ? 2 : 4; }
};

__device__ constexpr int tile_at(int row, int column) { return row * (row + 1) / 2 + column; }

// Factors of a block's rows.
enum { kFactorR, kFactorX, kFactorQ };

constexpr int kPitch = 20;  // of a tile's rows in LDS: rows 0 .. 7 begin in banks of their own

template <int DK, bool BF16, int NT, bool LOCAL>
struct BlockShared {
  h8_t key[BlockOps<DK, BF16, NT>::kParts * BlockOps<DK, BF16, NT>::kRows];
  float a[BlockOps<DK, BF16, NT>::kTiles][16 * kPitch];  // A, then (I + A)^-1
  float p[BlockOps<DK, BF16, NT>::kTiles][16 * kPitch];  // P
  double decay[64];                                      // G in exponents of 2
  uint64_t line[64];                                     // trees: ancestors and self
  h8_t query[LOCAL ? BlockOps<DK, BF16, NT>::kParts * BlockOps<DK, BF16, NT>::kRows : 1];
  float beta[64], key_factor[64], query_factor[64];
  float factor[3][16 * NT], end;  // e^G_end
  uint64_t lost[1 + NT];          // tokens that are not finite: g or beta; k, 16 of them each
};

// Tokens of a block that are not finite.
template <int DK, bool BF16, int NT, bool LOCAL>
__device__ __forceinline__ uint64_t lost_tokens(const BlockShared<DK, BF16, NT, LOCAL>& sh) {
  uint64_t lost = sh.lost[0];
#pragma unroll
  for (int t = 0; t < NT; ++t) lost |= sh.lost[1 + t] << (16 * t);
  return lost;
}

__device__ __forceinline__ bool finite(float x) { return fabsf(x) < __builtin_inff(); }

// Takes a column's values that are not finite out of x (rows 16 t + 4 g ..); the tokens
// that are none of a column's any more, or of none.
template <int NT>
__device__ __forceinline__ uint64_t lost_values(uint64_t lost, f4_t (&x)[NT]) {
  float odd = 0.0f;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e) odd = __builtin_fmaf(x[t][e], 0.0f, odd);
  if (!__any(odd != 0.0f)) return lost;  // NaN is not 0, and 0 times an infinity is NaN
  uint64_t own = 0;
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int e = 0; e < 4; ++e)
      if (!finite(x[t][e])) {
        own |= 1ull << (16 * t + 4 * ((threadIdx.x & 63) >> 4) + e);
        x[t][e] = 0.0f;
      }
  own |= __shfl_xor(own, 16);
  return lost | own | __shfl_xor(own, 32);
}

// Token i and those before it.
__device__ __forceinline__ uint64_t up_to(int i) { return (2ull << i) - 1; }

// A row of k or q as it comes: lane j + 16 g has its share of row j of a tile.
template <int DK, bool BF16>
struct RawRow {
  u4_t x[DK / 32][BF16 ? 1 : 2];  // values 32 s + 4 g .., 32 s + 16 + 4 g ..
};

template <int DK, bool BF16>
__device__ __forceinline__ void load_row(const void* rows, int64_t at, RawRow<DK, BF16>& raw) {
  const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
  for (int s = 0; s < DK / 32; ++s) {
    if constexpr (BF16) {
      const uint16_t* p = static_cast<const uint16_t*>(rows) + at + 32 * s + 4 * g;
      const u2_t lo = *reinterpret_cast<const u2_t*>(p), hi = *reinterpret_cast<const u2_t*>(p + 16);
      raw.x[s][0] = u4_t{lo.x, lo.y, hi.x, hi.y};
    } else {
      const float* p = static_cast<const float*>(rows) + at + 32 * s + 4 * g;
      raw.x[s][0] = *reinterpret_cast<const u4_t*>(p);
      raw.x[s][1] = *reinterpret_cast<const u4_t*>(p + 16);
    }
  }
}

// The row as an operand, zeros where it is not there.  Returns the factor that makes
// the stored row the row as used; `as_used` (or NULL) is where that goes.  `lost` (or
// NULL): whether the row as used is not finite; then it is as if it were not there.
template <int DK, bool BF16>
__device__ __forceinline__ float row_operand(const RawRow<DK, BF16>& raw, bool there, float eps,
                                             h8_t (&op)[BF16 ? 1 : 2][DK / 32], float* as_used = nullptr,
                                             bool* lost = nullptr) {
  f4_t x[DK / 32][2];
  float m = 0.0f;
#pragma unroll
  for (int s = 0; s < DK / 32; ++s)
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t w;
        if constexpr (BF16) w = (i & 1) ? raw.x[s][0][2 * h + (i >> 1)] & 0xFFFF0000u : raw.x[s][0][2 * h + (i >> 1)] << 16;
        else w = raw.x[s][h][i];
        x[s][h][i] = there ? __uint_as_float(w) : 0.0f;
      }
      m = max4(m, x[s][h]);
    }
  const int e = exponent_of(max_of_groups(m));
  float ss = 0.0f;
#pragma unroll
  for (int s = 0; s < DK / 32; ++s) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      x[s][h] = scale4(x[s][h], -e);
#pragma unroll
      for (int i = 0; i < 4; ++i) ss = __builtin_fmaf(x[s][h][i], x[s][h][i], ss);
    }
    if constexpr (BF16) op[0][s] = operand_hi(x[s][0], x[s][1]);
    else operand_parts(x[s][0], x[s][1], op[0][s], op[1][s]);
  }
  ss = sum_of_groups(ss);
  float factor = __builtin_amdgcn_ldexpf(1.0f, e);
  if (eps >= 0.0f) {
    // 1 / sqrt of the scaled row's squares; where eps, scaled alike, is past fp32 it is all
    const float small = __builtin_amdgcn_ldexpf(eps, -2 * e);
    const bool all = small > 1e38f;
    const float square = all ? eps : ss + small;
    float y = __builtin_amdgcn_rsqf(square);
    y = square > 0.0f ? __builtin_fmaf(0.5f * y, __builtin_fmaf(-square * y, y, 1.0f), y) : y;
    factor = all ? __builtin_amdgcn_ldexpf(y, e) : y;
  }
  if (as_used) {
    const int g = (threadIdx.x & 63) >> 4;
#pragma unroll
    for (int s = 0; s < DK / 32; ++s)
#pragma unroll
      for (int h = 0; h < 2; ++h)
        *reinterpret_cast<f4_t*>(as_used + 32 * s + 16 * h + 4 * g) =
            there ? x[s][h] * factor : f4_t{0.0f, 0.0f, 0.0f, 0.0f};
  }
  if (lost) {
    // of a finite row ss is 4 DK at most; a row of zeros without eps has no factor
    *lost = there && !(finite(ss) && finite(factor));
    if (__any(*lost)) {
#pragma unroll
      for (int part = 0; part < (BF16 ? 1 : 2); ++part)
#pragma unroll
        for (int s = 0; s < DK / 32; ++s)
          if (*lost) op[part][s] = h8_t{0, 0, 0, 0, 0, 0, 0, 0};
      there &= !*lost;
    }
  }
  return there ? factor : 0.0f;
}

// a b^T of two tiles' rows, with `parts` as above: 16x16.
template <int STEPS, int PARTS>
__device__ __forceinline__ f4_t rows_product(const h8_t (&a)[PARTS][STEPS], const h8_t* b, int pitch) {
  f4_t acc = {0.0f, 0.0f, 0.0f, 0.0f};
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int s = 0; s < STEPS; ++s) {
    const h8_t hi = b[s * 64 + lane];
    acc = mfma16x16x32(a[0][s], hi, acc);
    if constexpr (PARTS == 2) {
      acc = mfma16x16x32(a[0][s], b[pitch + s * 64 + lane], acc);
      acc = mfma16x16x32(a[1][s], hi, acc);
    }
  }
  return acc;
}

// c + a b of 16x16 tiles in fp32, b as a result stands; a: row j's values 4 g .. + 3.
__device__ __forceinline__ f4_t tile_product(f4_t a, f4_t b, f4_t c) {
#pragma unroll
  for (int i = 0; i < 4; ++i) c = __builtin_amdgcn_mfma_f32_16x16x4f32(a[i], b[i], c, 0, 0, 0);
  return c;
}

__device__ __forceinline__ f4_t tile_rows(const float* a) {
  const int lane = threadIdx.x & 63;
  return *reinterpret_cast<const f4_t*>(a + (lane & 15) * kPitch + 4 * (lane >> 4));
}

__device__ __forceinline__ f4_t load_tile(const float* a) {
  const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
  return f4_t{a[(4 * g) * kPitch + j], a[(4 * g + 1) * kPitch + j], a[(4 * g + 2) * kPitch + j],
              a[(4 * g + 3) * kPitch + j]};
}

__device__ __forceinline__ void store_tile(float* a, f4_t x) {
  const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
#pragma unroll
  for (int i = 0; i < 4; ++i) a[(4 * g + i) * kPitch + j] = x[i];
}

// The lower triangle `rows` of tiles, each as tile_rows has it, times x.  Products of
// different rows of tiles stand side by side: one waits for none of its own.
template <int NT, typename F>
__device__ __forceinline__ void lower_product(F rows, const f4_t (&x)[NT], f4_t (&y)[NT]) {
#pragma unroll
  for (int t = 0; t < NT; ++t) y[t] = f4_t{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
  for (int c = 0; c < NT; ++c) {
    f4_t a[NT];
#pragma unroll
    for (int t = c; t < NT; ++t) a[t] = rows(tile_at(t, c));
#pragma unroll
    for (int i = 0; i < 4; ++i)
#pragma unroll
      for (int t = c; t < NT; ++t) y[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(a[t][i], x[c][i], y[t], 0, 0, 0);
  }
}

// y plus the same of rows in N bf16 parts, part p of step l at rows(p, l): the products
// of parts that reach N bits by eight.
template <int NT, int N, typename F>
__device__ __forceinline__ void add_wide_product(F rows, const f4_t (&x)[NT], f4_t (&y)[NT]) {
  static_assert(NT % 2 == 0, "whole steps");
  typedef BlockOps<64, true, NT> Ops;
#pragma unroll
  for (int s = 0; s < NT / 2; ++s) {
    b8_t part[N];
    wide_parts<N>(x[2 * s], x[2 * s + 1], part);
#pragma unroll
    for (int p = 0; p < N; ++p)
#pragma unroll
      for (int q = 0; q < N; ++q) {
        if (p + q >= N && !(N == 3 && p == 1 && q == 1)) continue;
#pragma unroll
        for (int t = 2 * s; t < NT; ++t) y[t] = mfma16x16x32(rows(p, Ops::lower(t) + s), part[q], y[t]);
      }
  }
}

// N bf16 parts of row j of a row of tiles, its own one the `last`: steps from 0 on.
template <int N, typename F>
__device__ __forceinline__ void store_wide(F values, int last, h8_t* to, int pitch) {
  const int lane = threadIdx.x & 63;
#pragma unroll
  for (int s = 0; s < 2; ++s) {
    if (2 * s > last) continue;
    b8_t part[N];
    wide_parts<N>(values(2 * s), 2 * s < last ? values(2 * s + 1) : f4_t{0.0f, 0.0f, 0.0f, 0.0f}, part);
#pragma unroll
    for (int i = 0; i < N; ++i) to[i * pitch + s * 64 + lane] = __builtin_bit_cast(h8_t, part[i]);
  }
}

// (I + A)^-1 of a 16x16 tile in place, by substitution, a column a lane: each value
// found is taken off all rows below it, which do not wait for each other.
__device__ __forceinline__ void invert_tile(float* a) {
  const int j = threadIdx.x & 15;
  f4_t r[16][4];
#pragma unroll
  for (int i = 1; i < 16; ++i)
#pragma unroll
    for (int m = 0; m < (i + 3) / 4; ++m) r[i][m] = *reinterpret_cast<const f4_t*>(a + i * kPitch + 4 * m);
  float x[16];
#pragma unroll
  for (int i = 0; i < 16; ++i) x[i] = i == j ? 1.0f : 0.0f;
#pragma unroll
  for (int m = 0; m < 15; ++m)
#pragma unroll
    for (int i = m + 1; i < 16; ++i) x[i] = __builtin_fmaf(-r[i][m >> 2][m & 3], x[m], x[i]);
  if ((threadIdx.x & 63) < 16)
#pragma unroll
    for (int i = 0; i < 16; ++i) a[i * kPitch + j] = x[i];
}

// An operand of K transposed from K's: lane j + 16 g has tokens 32 s + 4 g .., 32 s +
// 16 + 4 g .. of value 16 t + j.
template <int DK, bool BF16, int NT>
__device__ __forceinline__ h8_t transposed_operand(const h8_t* key, int part, int t, int s) {
  typedef BlockOps<DK, BF16, NT> Ops;
  const _Float16* from = reinterpret_cast<const _Float16*>(key);
  const int lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
  h8_t x;
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int rt = 2 * s + (i >> 2), tok = 4 * g + (i & 3);
    const int unit = part * Ops::kRows + (rt * Ops::kSteps + (t >> 1)) * 64 + tok + 16 * (j >> 2);
    x[i] = rt < NT ? from[unit * 8 + 4 * (t & 1) + (j & 3)] : (_Float16)0.0f;
  }
  return x;
}

// What a block is made of, as it comes from memory.
template <int DK, bool BF16>
struct BlockRows {
  RawRow<DK, BF16> k, q;
  float g, beta;
  int parent;
};

// The rows from `first` on, `rows` of which are in memory (at least one): those behind
// them are the last one again.
template <int DK, bool BF16, int NT, bool TREE>
__device__ __forceinline__ void load_block_rows(const DeltaArgs& a, int64_t first, int rows, int h, int kh,
                                                BlockRows<DK, BF16>& to) {
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, i = 16 * w + (lane & 15);
  if (w >= NT) return;
  const int64_t row = first + (i < rows ? i : rows - 1), token = first + (lane < rows ? lane : rows - 1);
  load_row<DK, BF16>(a.k, row * a.k_stride + (int64_t)kh * DK, to.k);
  load_row<DK, BF16>(a.q, row * a.q_stride + (int64_t)kh * DK, to.q);
  if (w == 0) {
    to.g = a.g[token * a.heads + h];
    to.beta = a.beta[token * a.heads + h];
    if constexpr (TREE) to.parent = a.parent[token];
  }
}

// Prepares the n tokens of a block of value head h, n <= 16 NT, from its rows,
// by a workgroup of at least NT waves, the first NT of which work.  key_to: the key
// head's part (NULL: not wanted), head_to: the value head's.  LOCAL: the workgroup
// goes on with the block itself, after a barrier: K, Q, (I + A)^-1, P and the factors
// stay in sh.  Trees: `keys` (or NULL) takes the keys' rows as used, `key_row` values
// apart, for all `nodes` of them.
template <int DK, bool BF16, int NT, bool TREE, bool LOCAL, bool TILES = false>
__device__ __forceinline__ void prepare_block(const DeltaArgs& a, const BlockRows<DK, BF16>& rows, int n,
                                              BlockShared<DK, BF16, NT, LOCAL>& sh, h8_t* key_to, h8_t* head_to,
                                              float* keys = nullptr, int64_t key_row = 0, int nodes = 0) {
  typedef BlockOps<DK, BF16, NT, TILES> Ops;
  constexpr int P = Ops::kParts;
  const int lane = threadIdx.x & 63, w = threadIdx.x >> 6, j = lane & 15, g = lane >> 4;
  const bool works = w < NT;
  const bool there = works && 16 * w + j < n;
  h8_t key[P][Ops::kSteps], query[P][Ops::kSteps];
  float kf = 0.0f, qf = 0.0f;
  if (works) {
    float* as_used = TREE && keys && 16 * w + j < nodes ? keys + (16 * w + j) * key_row : nullptr;
    bool lost;
    kf = row_operand<DK, BF16>(rows.k, there, a.norm_eps, key, as_used, &lost);
    const uint64_t of_tile = __ballot(lost) & 0xFFFF;
    if (lane == 0) sh.lost[1 + w] = of_tile;
    qf = row_operand<DK, BF16>(rows.q, there, a.norm_eps, query) * a.scale;
    if (g == 0) {
      sh.key_factor[16 * w + j] = kf;
      sh.query_factor[16 * w + j] = qf;
    }
#pragma unroll
    for (int p = 0; p < P; ++p)
#pragma unroll
      for (int s = 0; s < Ops::kSteps; ++s) {
        const int at = p * Ops::kRows + (w * Ops::kSteps + s) * 64 + lane;
        sh.key[at] = key[p][s];
        if constexpr (LOCAL) sh.query[at] = query[p][s];
        else if (key_to) {
          key_to[Ops::kKey + at] = key[p][s];
          key_to[Ops::kQuery + at] = query[p][s];
        }
      }
  }
  if (w == 0) {
    const bool lost = lane < n && !(rows.g < __builtin_inff() && finite(rows.beta));
    const uint64_t tokens = __ballot(lost);
    if (lane == 0) sh.lost[0] = tokens;
    sh.beta[lane] = lane < n && !lost ? rows.beta : 0.0f;
    // e^-1e4 is 0, and differences stay finite
    const float gl = lane >= n || lost ? 0.0f : rows.g < -1e4f ? -1e4f : rows.g;
    double sum = (double)gl * 1.4426950408889634074;  // exponents of 2
    if constexpr (TREE) {
      sh.line[lane] = ancestors_of_wave(lane < n ? rows.parent : -1, [&](int at, bool on) {
        const double d = __shfl(sum, at);
        sum += on ? d : 0.0;
      });
    } else {
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const double o = __shfl_up(sum, off);
        sum += lane >= off ? o : 0.0;
      }
    }
    sh.decay[lane] = sum;
  }
  __syncthreads();
  if (works) {
    double gi[4];
    float bi[4], ki[4], qi[4];
    uint64_t line[4];
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int i = 16 * w + 4 * g + e;
      gi[e] = sh.decay[i];
      bi[e] = sh.beta[i];
      ki[e] = sh.key_factor[i];
      qi[e] = sh.query_factor[i];
      line[e] = TREE ? sh.line[i] : 0;
    }
#pragma unroll
    for (int c = 0; c < NT; ++c) {
      if (c > w) continue;
      const h8_t* kc = sh.key + c * Ops::kSteps * 64;
      f4_t kk = rows_product<Ops::kSteps, P>(key, kc, Ops::kRows);
      f4_t qk = rows_product<Ops::kSteps, P>(query, kc, Ops::kRows);
      const int col = 16 * c + j;
      const double gj = sh.decay[col];
      const float kj = sh.key_factor[col];
#pragma unroll
      for (int e = 0; e < 4; ++e) {
        const int i = 16 * w + 4 * g + e;
        const bool seen = TREE ? ((line[e] >> col) & 1) != 0 : col <= i;
        const float d = __builtin_amdgcn_exp2f((float)(gi[e] - gj)) * kj;
        kk[e] = seen && col < i ? bi[e] * ki[e] * d * kk[e] : 0.0f;
        qk[e] = seen ? qi[e] * d * qk[e] : 0.0f;
      }
      store_tile(sh.a[tile_at(w, c)], kk);
      store_tile(sh.p[tile_at(w, c)], qk);
    }
    if (g == 0) {
      const int i = 16 * w + j;
      const double at = sh.decay[i], end = sh.decay[16 * NT - 1];
      const float into = __builtin_amdgcn_exp2f((float)at);
      sh.factor[kFactorR][i] = -into * kf;
      sh.factor[kFactorX][i] = kf * __builtin_amdgcn_exp2f((float)(end - at));
      sh.factor[kFactorQ][i] = into * qf;
      if (i == 0) sh.end = __builtin_amdgcn_exp2f((float)end);
    }
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    __builtin_amdgcn_wave_barrier();
    invert_tile(sh.a[tile_at(w, w)]);
  }
  const f4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
  if constexpr (NT >= 2) {
    __syncthreads();
    if (w < NT / 2) {  // -T_11 A_10 T_00 of each pair of tiles
      float* at = sh.a[tile_at(2 * w + 1, 2 * w)];
      const f4_t y = tile_product(tile_rows(at), load_tile(sh.a[tile_at(2 * w, 2 * w)]), zero);
      store_tile(at, -tile_product(tile_rows(sh.a[tile_at(2 * w + 1, 2 * w + 1)]), y, zero));
    }
  }
  if constexpr (NT >= 3) {
    __syncthreads();
    // rows of tile r, columns of tile c: -sum_m T_rm (A_m0 T_0c + A_m1 T_1c)
    const int c = w & 1, r = 2 + (w >> 1);
    f4_t z = zero;
    if (works && r < NT) {
      const f4_t t1 = load_tile(sh.a[tile_at(1, c)]);
#pragma unroll
      for (int m = 2; m < NT; ++m) {
        if (m > r) continue;
        f4_t y = tile_product(tile_rows(sh.a[tile_at(m, 1)]), t1, zero);
        if (c == 0) y = tile_product(tile_rows(sh.a[tile_at(m, 0)]), load_tile(sh.a[tile_at(0, 0)]), y);
        z = tile_product(tile_rows(sh.a[tile_at(r, m)]), y, z);
      }
    }
    __syncthreads();
    if (works && r < NT) store_tile(sh.a[tile_at(r, c)], -z);
  }
  if constexpr (!LOCAL) {
    __syncthreads();
    if (works) {
      // T's columns have their rates
      const auto t_rows = [&](int c) {
        return tile_rows(sh.a[tile_at(w, c)]) * *reinterpret_cast<const f4_t*>(&sh.beta[16 * c + 4 * g]);
      };
      if constexpr (TILES) {
#pragma unroll
        for (int c = 0; c < NT; ++c)
          if (c <= w) reinterpret_cast<f4_t*>(head_to + Ops::kT)[tile_at(w, c) * 64 + lane] = t_rows(c);
      } else {
        store_wide<3>(t_rows, w, head_to + Ops::kT + Ops::lower(w) * 64, Ops::kLower * 64);
      }
      store_wide<Ops::kPartsOfP>([&](int c) { return tile_rows(sh.p[tile_at(w, c)]); }, w,
                                 head_to + Ops::kP + Ops::lower(w) * 64, Ops::kLower * 64);
      float* factors = reinterpret_cast<float*>(head_to + Ops::kFactors);
      if (g < 3) factors[g * 16 * NT + 16 * w + j] = sh.factor[g][16 * w + j];
      if (w == 0 && lane == 0) {
        const uint64_t lost = lost_tokens(sh);
        *reinterpret_cast<u4_t*>(factors + 3 * 16 * NT) =
            u4_t{__float_as_uint(sh.end), 0, (uint32_t)lost, (uint32_t)(lost >> 32)};
      }
      if (key_to)
#pragma unroll 1
        for (int u = w; u < P * (DK / 16) * Ops::kTokenSteps; u += NT) {
          const int part = u / ((DK / 16) * Ops::kTokenSteps), v = u - part * ((DK / 16) * Ops::kTokenSteps);
          key_to[Ops::kKeyT + part * Ops::kCols + v * 64 + lane] =
              transposed_operand<DK, BF16, NT>(sh.key, part, v / Ops::kTokenSteps, v % Ops::kTokenSteps);
        }
    }
  }
}

}  // namespace nvfp4
