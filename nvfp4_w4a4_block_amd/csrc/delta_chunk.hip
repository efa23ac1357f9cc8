// Gated delta rule over chains of some length, 64 tokens at a time.
//
// The page "TensorRT Edge-LLM Completes the MLPerf Edge Agentic Benchmark 6.4x
// Faster on Jetson AGX Thor" prefills only the new suffix of a turn and goes on from
// the recurrent state that was kept (section "Reusing KV cache across agent turns").
//
// delta_block.h has the mathematics.  delta_prepare_kernel makes the blocks' T, P and
// operands, all blocks at once; delta_scan_kernel walks each sequence, a wave with
// its 16 columns of the state in registers, which nothing else waits for.
//
// Bounds.  The walk is a chain of dependent products: a block's K S, T r and K^T X,
// half of whose time is the matrix instructions' and the rest LDS and the rounding of
// results into operands.  512 tokens of one sequence, 16 key and 48 value heads of 128,
// bf16: 14.8 us of preparation and 23.8 of walking (memory's share is 5, the products' 1);
// 3 sequences of up to 4,099 tokens, 4 and 8 heads of 64, fp32: 20 and 125.
#include "delta_block.h"

namespace nvfp4 {
namespace {

constexpr int kTiles = kChunk / 16;

// Blocks c0 .. c1 - 1 of the sequences from b0 on; what is prepared of them, and the
// states between two such rounds.
struct Round {
  int b0, c0, c1, last;
  h8_t *keys, *heads;  // [sequence - b0][c1 - c0][key_heads or heads][units]
  float* carry;        // [sequence - b0][heads][dv][dk]
};

// grid (heads, c1 - c0, seqs).
template <int DK, bool BF16, bool TILES>
__global__ __launch_bounds__(64 * kTiles) void delta_prepare_kernel(DeltaArgs a, Round r) {
  typedef BlockOps<DK, BF16, kTiles, TILES> Ops;
  __shared__ BlockShared<DK, BF16, kTiles, false> sh;
  const int h = blockIdx.x, b = r.b0 + blockIdx.z, t0 = (r.c0 + blockIdx.y) * kChunk, group = a.heads / a.key_heads;
  const int kh = h / group;
  BlockRows<DK, BF16> rows;
  load_block_rows<DK, BF16, kTiles, false>(a, (int64_t)b * a.nodes + t0, a.nodes - t0, h, kh, rows);
  const int count = delta_used(a.src[b], a.slots) ? delta_count(a.counts, a.nodes, b) : 0;
  if (t0 >= count) return;
  const int n = count - t0 < kChunk ? count - t0 : kChunk;
  const int64_t block = (int64_t)blockIdx.z * (r.c1 - r.c0) + blockIdx.y;
  h8_t* key_to = h % group == 0 ? r.keys + (block * a.key_heads + kh) * Ops::kKeyUnits : nullptr;
  prepare_block<DK, BF16, kTiles, false, false, TILES>(a, rows, n, sh, key_to, r.heads + (block * a.heads + h) * Ops::kHeadUnits);
}

// 64 rows of 16 values, one after the other in LDS; the pitch keeps the four rows that
// a wave's lane groups read at a time in banks of their own.
template <bool BF16>
struct Rows16 {
  static constexpr int kSize = BF16 ? 2 : 4, kPitch = BF16 ? 48 : 80, kPieces = kSize, kLoads = kSize;
  char x[kChunk * kPitch];  // a row is kPieces pieces of 16 bytes, a lane has kLoads of them
  __device__ __forceinline__ char* piece(int u) {
    const int i = 64 * u + (threadIdx.x & 63);
    return x + i / kPieces * kPitch + i % kPieces * 16;
  }
  __device__ __forceinline__ char* value(int row) { return x + row * kPitch + (threadIdx.x & 15) * kSize; }
};

// A block's values of a wave's columns from memory: rows behind the n-th are the last
// one again (their rate is 0, and so is what they add).
template <bool BF16>
__device__ __forceinline__ void load_values(const char* rows, int64_t stride, int n, u4_t (&x)[BF16 ? 2 : 4]) {
  constexpr int pieces = Rows16<BF16>::kPieces;
#pragma unroll
  for (int u = 0; u < Rows16<BF16>::kLoads; ++u) {
    const int i = 64 * u + (threadIdx.x & 63), row = i / pieces;
    x[u] = *reinterpret_cast<const u4_t*>(rows + (row < n ? row : n - 1) * stride + i % pieces * 16);
  }
}

// The largest bits of magnitudes, two of them in bf16; whether they are not finite.
typedef uint16_t us2_t __attribute__((ext_vector_type(2)));

template <bool BF16>
__device__ __forceinline__ uint32_t most_of(uint32_t most, u4_t x) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if constexpr (BF16)
      most = __builtin_bit_cast(uint32_t, __builtin_elementwise_max(__builtin_bit_cast(us2_t, most),
                                                                    __builtin_bit_cast(us2_t, x[i] & 0x7FFF7FFFu)));
    else
      most = max(most, x[i] & 0x7FFFFFFFu);
  }
  return most;
}

template <bool BF16>
__device__ __forceinline__ bool not_finite(uint32_t most) {
  return BF16 ? (most & 0xFFFF) >= 0x7F80 || most >> 16 >= 0x7F80 : most >= 0x7F800000u;
}

// Zeros in place of values that are not finite; a column's first one to `lost`.
template <bool BF16>
__device__ __forceinline__ void take_out(Rows16<BF16>& v, int* lost) {
  wave_sync();
  const int j = threadIdx.x & 15;
#pragma unroll 1
  for (int i = (threadIdx.x & 63) >> 4; i < kChunk; i += 4) {
    char* at = v.value(i);
    if constexpr (BF16) {
      if ((*reinterpret_cast<uint16_t*>(at) & 0x7F80) != 0x7F80) continue;
      *reinterpret_cast<uint16_t*>(at) = 0;
    } else {
      if (finite(*reinterpret_cast<float*>(at))) continue;
      *reinterpret_cast<float*>(at) = 0.0f;
    }
    atomicMin(&lost[j], i);
  }
}

#define GLOBAL_PTR(p) ((const __attribute__((address_space(1))) void*)(uintptr_t)(p))
#define LDS_PTR(p) ((__attribute__((address_space(3))) void*)(uintptr_t)(p))

// Every wave's LDS work is done and seen by all; memory is not waited for.
__device__ __forceinline__ void lds_barrier() {
  __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
  __builtin_amdgcn_s_barrier();
  __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
}

// T is in a state wave's registers where they have room: with 32 columns a workgroup, and
// rows of k that take one part or are short; else it comes to LDS with the others.
template <int DK, bool BF16, int SLABS, int BUFFERS>
constexpr bool kHoldT = SLABS == 2 && (BF16 || DK == 64 || BUFFERS == 0);

// Units of a block that come to LDS.
template <int DK, bool BF16, int SLABS, int BUFFERS>
constexpr int kUnitsHere = BlockOps<DK, BF16, kTiles, SLABS == 4>::kQuery +
                           (kHoldT<DK, BF16, SLABS, BUFFERS> ? BlockOps<DK, BF16, kTiles, SLABS == 4>::kT
                                                             : BlockOps<DK, BF16, kTiles, SLABS == 4>::kP);

// What a state's wave leaves for the wave of its outputs, and the fetching one for it.  A
// token of which a column keeps nothing (k, g, beta or its value are not finite, or the
// state is not) and what follows it are NaN there; the products go on without it.
template <int DK, bool BF16>
struct Handed {
  h8_t s[2][DK / 32][64];             // S as an operand
  f4_t w[kTiles][64];                 // u
  int es[16];                         // S's exponent, by column
  int first[16];                      // first token of which nothing is left, 64: none
  Rows16<BF16> v;                     // the other way: the block's values,
  int lost[16];                       // and a column's first token that is not finite
};

// grid (heads, dv / (16 SLABS), seqs).  SLABS waves have 16 columns of the state each:
// r, u and the new state, one block after the other.  SLABS more make the outputs of
// the same columns, of which no state waits, and one fetches the next block's operands
// and values, so that none of the others stands in the queue to memory.  BUFFERS:
// blocks whose K, K^T, T and factors are in LDS; 2: those of the next block come while
// one is worked on; 0: they are read where they are.  HANDS: blocks that are handed
// over at a time; 2: outputs are a block behind the states, and all waves meet once a
// block; 1: they meet when S is ready, and when u is.
template <int DK, bool BF16, int SLABS, int BUFFERS, int HANDS>
__global__ __launch_bounds__(64 * (2 * SLABS + 1), 1) void delta_scan_kernel(DeltaArgs a, Round r) {
  constexpr bool kInTiles = SLABS == 4;
  typedef BlockOps<DK, BF16, kTiles, kInTiles> Ops;
  constexpr bool kHold = kHoldT<DK, BF16, SLABS, BUFFERS>;
  constexpr int P = Ops::kParts, KT = DK / 16, kUnits = kUnitsHere<DK, BF16, SLABS, BUFFERS>;
  __shared__ h8_t ops[BUFFERS ? BUFFERS : 1][BUFFERS ? kUnits : 1];
  static_assert(HANDS == 1 || BUFFERS == 2, "outputs a block behind leave no barrier between blocks");
  __shared__ Handed<DK, BF16> handed[HANDS][SLABS];
  __shared__ Rows16<BF16> outs[SLABS];  // on their way to memory
  const int h = blockIdx.x, b = r.b0 + blockIdx.z, lane = threadIdx.x & 63, j = lane & 15, g = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6), slab = wave % SLABS;
  const int col0 = (blockIdx.y * SLABS + slab) * 16, kh = h / (a.heads / a.key_heads);
  const bool states = wave < SLABS;
  const int src = a.src[b];
  const int64_t first = (int64_t)b * a.nodes, state_size = (int64_t)a.dv * DK;
  const int64_t value_at = (int64_t)h * a.dv + col0 + j;
  if (!delta_used(src, a.slots)) {
    if (r.c0 == 0 && states)
      for (int t = 0; t < a.nodes; ++t)
        if (lane < 16) store1<BF16>(a.out, (first + t) * a.heads * a.dv + value_at, 0.0f);
    return;
  }
  const int count = delta_count(a.counts, a.nodes, b);
  const int end_block = (count + kChunk - 1) / kChunk < r.c1 ? (count + kChunk - 1) / kChunk : r.c1;
  const auto keys_of = [&](int c) {
    return r.keys + (((int64_t)blockIdx.z * (r.c1 - r.c0) + c - r.c0) * a.key_heads + kh) * Ops::kKeyUnits;
  };
  const auto heads_of = [&](int c) {
    return r.heads + (((int64_t)blockIdx.z * (r.c1 - r.c0) + c - r.c0) * a.heads + h) * Ops::kHeadUnits;
  };
  const auto buffer_of = [&](int c) { return ops[BUFFERS == 2 ? (c - r.c0) & 1 : 0]; };
  const auto key_ops = [&](int c) { return (BUFFERS ? buffer_of(c) : keys_of(c)) + lane; };
  const auto head_ops = [&](int c) { return BUFFERS ? buffer_of(c) + Ops::kQuery : heads_of(c); };
  const f4_t zero = {0.0f, 0.0f, 0.0f, 0.0f};
  const float nan = __builtin_nanf("");
  const auto hand_of = [&](int c) { return handed[HANDS == 2 ? (c - r.c0) & 1 : 0]; };
  if (states) {
    float* carry = r.carry + ((int64_t)blockIdx.z * a.heads + h) * state_size + (int64_t)col0 * DK;
    StateTile<DK, 1> st;
    if (r.c0 > 0) load_state<DK, 1>(carry, st);
    else if (src >= 0) load_state<DK, 1>(a.states + ((int64_t)src * a.heads + h) * state_size + (int64_t)col0 * DK, st);
    else zero_state<DK, 1>(st);
    f4_t(&s)[KT] = st.s[0];
    bool gone = false;  // nothing is left of the column
    if (r.c0 < end_block) {
      float m = 0.0f;
#pragma unroll
      for (int t = 0; t < KT; ++t) m = max4_nan(m, s[t]);
      const uint64_t odd = __ballot(!finite(m));
      if (odd) {
        gone = ((odd | odd >> 16 | odd >> 32 | odd >> 48) >> j) & 1;
#pragma unroll
        for (int t = 0; t < KT; ++t) s[t] = gone ? zero : s[t];
      }
    }
    // s holds S times 2^es
    int es = 0;
    if (r.c0 < end_block) {
      float m = 0.0f;
#pragma unroll
      for (int t = 0; t < KT; ++t) m = max4(m, s[t]);
      es = 5 - exponent_of(max_of_groups(m));
#pragma unroll
      for (int t = 0; t < KT; ++t) s[t] = scale4(s[t], es);
    }
    h8_t own[kHold ? 3 : 1][kHold ? Ops::kLower : 1];
    const auto load_own = [&](int c) {
      if constexpr (kHold) {
        const h8_t* from = heads_of(c) + Ops::kT + lane;
#pragma unroll
        for (int p = 0; p < 3; ++p)
#pragma unroll
          for (int l = 0; l < Ops::kLower; ++l) own[p][l] = from[(p * Ops::kLower + l) * 64];
      }
    };
    if (r.c0 < end_block) load_own(r.c0);
    for (int c = r.c0; c < end_block; ++c) {
      lds_barrier();  // the block's operands and values are here
      Handed<DK, BF16>& hand = hand_of(c)[slab];
      const h8_t* key = key_ops(c);
      const h8_t* head = head_ops(c) + lane;
      const float* factors = reinterpret_cast<const float*>(head - lane + Ops::kFactors);
      const auto factor = [&](int which, int t) {
        return *reinterpret_cast<const f4_t*>(factors + which * kChunk + 16 * t + 4 * g);
      };
      const int lost = hand.lost[j];
      // K S
      f4_t ks[kTiles];
#pragma unroll
      for (int t = 0; t < kTiles; ++t) ks[t] = zero;
#pragma unroll
      for (int x = 0; x < Ops::kSteps; ++x) {
        h8_t hi, lo;
        operand_parts(s[2 * x], s[2 * x + 1], hi, lo);
        hand.s[0][x][lane] = hi;
        hand.s[1][x][lane] = lo;
#pragma unroll
        for (int part = 0; part < P + 1; ++part)
#pragma unroll
          for (int t = 0; t < kTiles; ++t) {
            const int at = Ops::kKey + (t * Ops::kSteps + x) * 64;
            ks[t] = mfma16x16x32(key[part == 2 ? at + Ops::kRows : at], part == 1 ? lo : hi, ks[t]);
          }
      }
      hand.es[j] = es;
      hand.first[j] = gone ? 0 : lost;
      gone |= lost < kChunk;
      if constexpr (HANDS == 1) lds_barrier();  // S is handed over
      // r, and u = T r
      f4_t v[kTiles], w[kTiles];
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const char* at = hand.v.value(16 * t + 4 * g + e);
          if constexpr (BF16) v[t][e] = __uint_as_float((uint32_t)*reinterpret_cast<const uint16_t*>(at) << 16);
          else v[t][e] = *reinterpret_cast<const float*>(at);
        }
        const f4_t f = factor(kFactorR, t), y = scale4(ks[t], -es);
#pragma unroll
        for (int e = 0; e < 4; ++e) v[t][e] = __builtin_fmaf(f[e], y[e], v[t][e]);
      }
      if constexpr (kInTiles) {
        lower_product<kTiles>([&](int t) { return __builtin_bit_cast(f4_t, head[Ops::kT + t * 64]); }, v, w);
      } else {
#pragma unroll
        for (int t = 0; t < kTiles; ++t) w[t] = zero;
        add_wide_product<kTiles, 3>(
            [&](int p, int l) {
              if constexpr (kHold) return __builtin_bit_cast(b8_t, own[p][l]);
              else return __builtin_bit_cast(b8_t, head[Ops::kT + (p * Ops::kLower + l) * 64]);
            },
            v, w);
        if (kHold && c + 1 < end_block) load_own(c + 1);
      }
#pragma unroll
      for (int t = 0; t < kTiles; ++t) hand.w[t][lane] = w[t];
      if constexpr (HANDS == 1) lds_barrier();  // u is handed over
      // X = diag(e^(G_end - G)) u, and S <- e^G_end S + K^T X
      const float end = factors[3 * kChunk];
      float mx = 0.0f, ms = 0.0f;
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        w[t] *= factor(kFactorX, t);
        mx = max4(mx, w[t]);
      }
#pragma unroll
      for (int t = 0; t < KT; ++t) ms = max4(ms, s[t]);
      const int before = es;
      {
        const float most = fmaxf(mx, __builtin_amdgcn_ldexpf(ms, -es) * end);
        es = 5 - exponent_of(max_of_groups(most));
      }
      // e^G_end times a power of two, one factor: it takes the largest of s, 2^-30 at least
      // or nothing at all, to 64 at most, so it is past fp32 only where s is nothing
      float fade = __builtin_amdgcn_ldexpf(end, es - before);
      fade = fade == __builtin_inff() ? 0.0f : fade;
#pragma unroll
      for (int t = 0; t < KT; ++t) s[t] *= fade;
#pragma unroll
      for (int x = 0; x < Ops::kTokenSteps; ++x) {
        h8_t hi, lo;
        operand_parts(scale4(w[2 * x], es), scale4(w[2 * x + 1], es), hi, lo);
#pragma unroll
        for (int part = 0; part < P + 1; ++part)
#pragma unroll
          for (int t = 0; t < KT; ++t) {
            const int at = Ops::kKeyT + (t * Ops::kTokenSteps + x) * 64;
            s[t] = mfma16x16x32(key[part == 2 ? at + Ops::kCols : at], part == 1 ? lo : hi, s[t]);
          }
      }
      if constexpr (BUFFERS == 1) lds_barrier();  // the operands have been read
    }
    if (HANDS == 2 && r.c0 < end_block) lds_barrier();  // for the last outputs
#pragma unroll
    for (int t = 0; t < KT; ++t) s[t] = gone ? f4_t{nan, nan, nan, nan} : scale4(s[t], -es);
    if (!r.last) {
      store_state<DK, 1>(carry, st);
      return;
    }
    const int to = delta_dst(a.src, a.dst, a.seqs, a.slots, b);
    if (to >= 0) store_state<DK, 1>(a.states + ((int64_t)to * a.heads + h) * state_size + (int64_t)col0 * DK, st);
    return;
  }
  constexpr int size = BF16 ? 2 : 4;
  if (wave == 2 * SLABS) {
    const auto fetch_part = [&](int c, int part) {
      if constexpr (BUFFERS > 0) {
        constexpr int loads = kUnits / 64, third = (loads + 2) / 3;
        const h8_t* keys = keys_of(c) + lane;
        const h8_t* heads = heads_of(c) + lane - Ops::kQuery;
        h8_t* to = buffer_of(c);
#pragma unroll 4
        for (int i = part * third; i < (part + 1) * third; ++i)
          if (i < loads)
            __builtin_amdgcn_global_load_lds(GLOBAL_PTR((i < Ops::kQuery / 64 ? keys : heads) + 64 * i),
                                             LDS_PTR(to + 64 * i), 16, 0, 0);
      }
    };
    u4_t v[SLABS][Rows16<BF16>::kLoads];
    u2_t of_block;  // tokens whose k, g or beta is not finite
    const auto load_next = [&](int c) {
      of_block = *reinterpret_cast<const u2_t*>(reinterpret_cast<const float*>(heads_of(c) + Ops::kFactors) + 3 * kChunk + 2);
#pragma unroll
      for (int u = 0; u < SLABS; ++u)
        load_values<BF16>(static_cast<const char*>(a.v) + ((first + c * kChunk) * a.v_stride + (int64_t)h * a.dv +
                                                           (blockIdx.y * SLABS + u) * 16) * size,
                          a.v_stride * size, count - c * kChunk, v[u]);
    };
    const auto hand_next = [&](int c) {
      const uint64_t lost = of_block.x | (uint64_t)of_block.y << 32;
      uint32_t most = 0;
#pragma unroll
      for (int u = 0; u < SLABS; ++u) {
        if (lane < 16) hand_of(c)[u].lost[lane] = lost ? __builtin_ctzll(lost) : kChunk;
#pragma unroll
        for (int i = 0; i < Rows16<BF16>::kLoads; ++i) {
          *reinterpret_cast<u4_t*>(hand_of(c)[u].v.piece(i)) = v[u][i];
          most = most_of<BF16>(most, v[u][i]);
        }
      }
      if (__any(not_finite<BF16>(most)))
#pragma unroll
        for (int u = 0; u < SLABS; ++u) take_out<BF16>(hand_of(c)[u].v, hand_of(c)[u].lost);
    };
    if (r.c0 < end_block) {
      load_next(r.c0);
      for (int part = 0; part < 3; ++part) fetch_part(r.c0, part);
      hand_next(r.c0);
    }
    for (int c = r.c0; c < end_block; ++c) {
      const bool more = c + 1 < end_block, ahead = BUFFERS == 2 && more;
      __builtin_amdgcn_s_waitcnt(0x0F70);  // vmcnt(0): the operands are in LDS
      lds_barrier();
      if (more) load_next(c + 1);
      if (ahead) fetch_part(c + 1, 0);
      if constexpr (HANDS == 1) lds_barrier();  // S is handed over
      if (ahead) fetch_part(c + 1, 1);
      if constexpr (HANDS == 1) lds_barrier();  // u is handed over, the values have been read
      if (ahead) fetch_part(c + 1, 2);
      if (more) hand_next(c + 1);
      if constexpr (BUFFERS == 1) {
        lds_barrier();
        if (more)
          for (int part = 0; part < 3; ++part) fetch_part(c + 1, part);
      }
    }
    if (HANDS == 2 && r.c0 < end_block) lds_barrier();
    return;
  }
  // Q and P are this wave's alone: straight to registers, Q where it fits.  They come a
  // block ahead; in fp32 calls, where they are twice as large, outputs that are not
  // behind fetch one while they work on the other.
  constexpr int lag = HANDS - 1;
  constexpr bool ahead = BF16 || lag;
  constexpr bool hold = P * Ops::kSteps <= 8;
  h8_t q[P][kTiles][hold ? Ops::kSteps : 1];
  constexpr int kOfP = (Ops::kHeadUnits - Ops::kP) / 64;
  h8_t p[kOfP];
  const auto load_q = [&](int c) {
    if constexpr (!hold) return;
    const h8_t* from = keys_of(c) + Ops::kQuery + lane;
#pragma unroll
    for (int i = 0; i < P; ++i)
#pragma unroll
      for (int t = 0; t < kTiles; ++t)
#pragma unroll
        for (int x = 0; x < (hold ? Ops::kSteps : 1); ++x) q[i][t][x] = from[i * Ops::kRows + (t * Ops::kSteps + x) * 64];
  };
  const auto load_p = [&](int c) {
    const h8_t* from = heads_of(c) + Ops::kP + lane;
#pragma unroll
    for (int i = 0; i < kOfP; ++i) p[i] = from[i * 64];
  };
  const auto store_out = [&](int c) {
    const int64_t out_row = (int64_t)a.heads * a.dv * size;
    char* rows = static_cast<char*>(a.out) + (first + c * kChunk) * out_row + ((int64_t)h * a.dv + col0) * size;
    const int n = count - c * kChunk;
#pragma unroll
    for (int u = 0; u < Rows16<BF16>::kLoads; ++u) {
      const int i = 64 * u + lane, row = i / Rows16<BF16>::kPieces;
      const u4_t x = *reinterpret_cast<const u4_t*>(outs[slab].piece(u));
      if (row < n) *reinterpret_cast<u4_t*>(rows + row * out_row + i % Rows16<BF16>::kPieces * 16) = x;
    }
  };
  if (r.c0 < end_block) {
    load_q(r.c0);
    if (ahead) load_p(r.c0);
  }
  const auto factor = [&](int c, int which, int t) {
    const float* factors = reinterpret_cast<const float*>(head_ops(c) + Ops::kFactors);
    return *reinterpret_cast<const f4_t*>(factors + which * kChunk + 16 * t + 4 * g);
  };
  f4_t fq[kTiles];  // a block that is behind takes them before the next one's come
  const auto load_factors = [&](int c) {
#pragma unroll
    for (int t = 0; t < kTiles; ++t) fq[t] = factor(c, kFactorQ, t);
  };
  if (r.c0 < end_block && lag) {
    lds_barrier();
    load_factors(r.c0);
  }
  for (int c = r.c0; c < end_block; ++c) {
    const bool more = c + 1 < end_block;
    lds_barrier();
    if (c > r.c0) store_out(c - 1);
    const Handed<DK, BF16>& hand = hand_of(c)[slab];
    if constexpr (!lag) lds_barrier();  // S is handed over
    f4_t y[kTiles];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) y[t] = zero;
#pragma unroll
    for (int x = 0; x < Ops::kSteps; ++x) {
      const h8_t hi = hand.s[0][x][lane];
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        const h8_t* in_place = keys_of(c) + Ops::kQuery + (t * Ops::kSteps + x) * 64 + lane;
        const h8_t q0 = hold ? q[0][t][hold ? x : 0] : in_place[0];
        y[t] = mfma16x16x32(q0, hi, y[t]);
        y[t] = mfma16x16x32(q0, hand.s[1][x][lane], y[t]);
        if constexpr (P == 2) {
          const h8_t q1 = hold ? q[1][t][hold ? x : 0] : in_place[Ops::kRows];
          y[t] = mfma16x16x32(q1, hi, y[t]);
        }
      }
    }
    const int es = hand.es[j], none_from = hand.first[j];
    if constexpr (ahead) {
      if (more) load_q(c + 1);
    } else {
      load_p(c);
    }
    const auto add_read = [&](f4_t(&z)[kTiles]) {
#pragma unroll
      for (int t = 0; t < kTiles; ++t) {
        if constexpr (!lag) fq[t] = factor(c, kFactorQ, t);
        z[t] += fq[t] * scale4(y[t], -es);
      }
    };
    // bf16 calls add P u to Q S, which saves registers; in fp32 calls, whose outputs have
    // more products than their states, two sums do not wait for each other (3 prompts of
    // up to 4,099 tokens: 138 us, 166 with one)
    f4_t z[kTiles] = {zero, zero, zero, zero};
    if constexpr (BF16) add_read(z);
    if constexpr (!lag) lds_barrier();  // u is handed over
    f4_t u[kTiles];
#pragma unroll
    for (int t = 0; t < kTiles; ++t) u[t] = hand.w[t][lane];
    add_wide_product<kTiles, Ops::kPartsOfP>(
        [&](int part, int l) { return __builtin_bit_cast(b8_t, p[part * Ops::kLower + l]); }, u, z);
    if (more) {
      if constexpr (ahead) load_p(c + 1);
      else load_q(c + 1);
    }
    if constexpr (!BF16) add_read(z);
#pragma unroll
    for (int t = 0; t < kTiles; ++t)
#pragma unroll
      for (int e = 0; e < 4; ++e) store1<BF16>(outs[slab].value(16 * t + 4 * g + e), 0, z[t][e]);
    if (__any(none_from < kChunk))
#pragma unroll 1
      for (int i = g; i < kChunk; i += 4)
        if (i >= none_from) store1<BF16>(outs[slab].value(i), 0, nan);
    __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
    if (lag && more) load_factors(c + 1);
    if constexpr (BUFFERS == 1) lds_barrier();
  }
  if (r.c0 < end_block) store_out(end_block - 1);
  if (!r.last) return;
  for (int t = count; t < a.nodes; ++t)
    if (lane < 16) store1<BF16>(a.out, (first + t) * a.heads * a.dv + value_at, 0.0f);
}

constexpr int kLds = 160 * 1024;

template <int DK, bool BF16, int SLABS, int BUFFERS, int HANDS>
constexpr int scan_lds() {
  return BUFFERS * 16 * kUnitsHere<DK, BF16, SLABS, BUFFERS> +
         SLABS * (HANDS * (int)sizeof(Handed<DK, BF16>) + (int)sizeof(Rows16<BF16>));
}

// Whether a workgroup has 64 columns: where 32 give more workgroups than there are CUs,
// of which each holds one, and LDS has room.
template <int DK, bool BF16>
bool four_slabs(const DeltaArgs& a) {
  return BF16 && a.bf16 && scan_lds<DK, BF16, 4, 2, 1>() <= kLds && (int64_t)a.seqs * a.heads * (a.dv / 32) > 256;
}

bool four_slabs(const DeltaArgs& a) {
  return a.dk == 64 ? four_slabs<64, true>(a) : a.dk == 128 ? four_slabs<128, true>(a) : four_slabs<256, true>(a);
}

// Bytes of a block of one sequence.
template <int DK, bool BF16>
int64_t block_bytes(const DeltaArgs& a) {
  const int head = four_slabs<DK, BF16>(a) ? BlockOps<DK, BF16, kTiles, true>::kHeadUnits
                                           : BlockOps<DK, BF16, kTiles, false>::kHeadUnits;
  return 16 * ((int64_t)a.key_heads * BlockOps<DK, BF16, kTiles>::kKeyUnits + (int64_t)a.heads * head);
}

int64_t block_bytes(const DeltaArgs& a) {
  if (a.dk == 64) return a.bf16 ? block_bytes<64, true>(a) : block_bytes<64, false>(a);
  if (a.dk == 128) return a.bf16 ? block_bytes<128, true>(a) : block_bytes<128, false>(a);
  return a.bf16 ? block_bytes<256, true>(a) : block_bytes<256, false>(a);
}

// What a round takes on: what is prepared of it, and the states that it leaves to the next
// one, stay within 128 MB, half the Infinity Cache (one block of one sequence is the
// least, whatever its size).
constexpr int64_t kRoundBytes = (int64_t)128 << 20;

struct Rounds {
  int seqs, blocks, all;
};

int64_t state_bytes(const DeltaArgs& a) { return (int64_t)a.heads * a.dv * a.dk * 4; }
int64_t carry_bytes(const DeltaArgs& a, const Rounds& r) { return r.blocks < r.all ? r.seqs * state_bytes(a) : 0; }

// The sequences of a round that cost least, by its number of rounds, each as many blocks
// as the workgroups, one a CU, go over the chip, and four for its launches.  A round that
// does not reach the sequences' ends moves their states as well.  us, 48 heads of 128,
// bf16, by as many sequences as fit with one block each, and so: 64 sequences of 200
// tokens 1,033 (their states go out and in at every block), 713; 4 of 2,047 368, 356.
Rounds rounds_of(const DeltaArgs& a) {
  const auto over = [](int64_t n, int64_t by) { return (n + by - 1) / by; };
  const int64_t bytes = block_bytes(a), groups = over((int64_t)a.heads * a.dv, four_slabs(a) ? 64 : 32);
  const int64_t all = over(a.nodes, kChunk), fit = kRoundBytes / bytes < 1 ? 1 : kRoundBytes / bytes;
  const int64_t most = fit < a.seqs ? fit : a.seqs, filled = over(8 * 256, groups);
  Rounds best = {1, 1, (int)all};
  double least = 0.0;
  // eight times over the chip and more, the sequences that fit are as good as any
  for (int64_t n = 1, next; n <= most; n = next) {
    next = n + n / 16 + 1;
    next = n == most || (next < filled && next < most) ? next : most;
    const int64_t seqs = over(a.seqs, over(a.seqs, n));
    int64_t blocks = all;
    if (seqs * all * bytes > kRoundBytes) {
      blocks = (kRoundBytes - seqs * state_bytes(a)) / (seqs * bytes);
      if (blocks < 1 && n > 1) break;
      blocks = over(all, over(all, blocks < 1 ? 1 : blocks));
    }
    const double moved = blocks < all ? (double)state_bytes(a) / bytes : 0.0;
    const double cost =
        over(a.seqs, seqs) * over(all, blocks) * (over(seqs * groups, 256) * (blocks + moved) + 4.0);
    if (n == 1 || cost < least) {
      least = cost;
      best.seqs = (int)seqs;
      best.blocks = (int)blocks;
    }
  }
  return best;
}

template <int DK, bool BF16, int SLABS, int BUFFERS, int HANDS>
void scan(const DeltaArgs& a, const Round& r, int seqs, hipStream_t stream) {
  const dim3 grid(a.heads, a.dv / (16 * SLABS), seqs);
  delta_scan_kernel<DK, BF16, SLABS, BUFFERS, HANDS><<<grid, 64 * (2 * SLABS + 1), 0, stream>>>(a, r);
}

// A CU holds one workgroup.  32 columns a workgroup spread a few heads over the most
// CUs; where that gives more workgroups than there are CUs, 64 columns share a block's
// operands, if LDS has room (48 heads of 128, bf16, us by 32 and by 64 columns: 4
// sequences of 2,047 tokens 403, 365; 64 of 200 930, 733).  By 32 columns outputs are a
// block behind, if LDS has room: all waves meet once a block, where those that are not
// behind meet three times (8,192 tokens of 48 heads, bf16, 409 us and 450; 2,048 tokens
// 101 and 105; 512 tokens 36.5 and 37.2; 3 of up to 4,099 of 8 heads of 64, fp32, 143 and
// 167).
template <int DK, bool BF16>
void scan(const DeltaArgs& a, const Round& r, int seqs, hipStream_t stream) {
  if constexpr (BF16 && scan_lds<DK, BF16, 4, 2, 1>() <= kLds)
    if (four_slabs<DK, BF16>(a)) {
      scan<DK, BF16, 4, 2, 1>(a, r, seqs, stream);
      return;
    }
  if constexpr (scan_lds<DK, BF16, 2, 2, 2>() <= kLds) {
    scan<DK, BF16, 2, 2, 2>(a, r, seqs, stream);
  } else {
    constexpr int buffers = scan_lds<DK, BF16, 2, 1, 1>() <= kLds ? 1 : 0;
    scan<DK, BF16, 2, buffers, 1>(a, r, seqs, stream);
  }
}

template <int DK, bool BF16>
void run(const DeltaArgs& a, hipStream_t stream) {
  const Rounds n = rounds_of(a);
  const bool tiles = four_slabs<DK, BF16>(a);
  Round r = {};
  r.carry = static_cast<float*>(a.workspace);
  r.keys = reinterpret_cast<h8_t*>(static_cast<char*>(a.workspace) + carry_bytes(a, n));
  r.heads = r.keys + (int64_t)n.seqs * n.blocks * a.key_heads * BlockOps<DK, BF16, kTiles>::kKeyUnits;
  for (r.b0 = 0; r.b0 < a.seqs; r.b0 += n.seqs) {
    const int seqs = a.seqs - r.b0 < n.seqs ? a.seqs - r.b0 : n.seqs;
    for (r.c0 = 0; r.c0 < n.all; r.c0 = r.c1) {
      r.c1 = r.c0 + n.blocks < n.all ? r.c0 + n.blocks : n.all;
      r.last = r.c1 == n.all;
      const dim3 grid(a.heads, r.c1 - r.c0, seqs);
      if (tiles) delta_prepare_kernel<DK, BF16, true><<<grid, 64 * kTiles, 0, stream>>>(a, r);
      else delta_prepare_kernel<DK, BF16, false><<<grid, 64 * kTiles, 0, stream>>>(a, r);
      scan<DK, BF16>(a, r, seqs, stream);
    }
  }
}

}  // namespace

int64_t delta_chunk_workspace_bytes(const DeltaArgs& a) {
  const Rounds r = rounds_of(a);
  return carry_bytes(a, r) + r.seqs * r.blocks * block_bytes(a);
}

void launch_delta_chunks(const DeltaArgs& a, hipStream_t stream) {
  if (a.dk == 64) a.bf16 ? run<64, true>(a, stream) : run<64, false>(a, stream);
  else if (a.dk == 128) a.bf16 ? run<128, true>(a, stream) : run<128, false>(a, stream);
  else a.bf16 ? run<256, true>(a, stream) : run<256, false>(a, stream);
}

}  // namespace nvfp4
