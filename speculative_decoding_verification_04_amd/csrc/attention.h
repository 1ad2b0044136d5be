// Attention of new tokens over a KV cache: the tile kernel shared by prompts
// (causal) and by drafted chains and trees (gfx950).
//
// For a query row q of a KV head's group and the cache rows that it sees,
//   s_j = scale q.k_j,  out = sum_j exp(s_j - m) v_j / sum_j exp(s_j - m),
// with a running maximum m and a running sum in one pass over the rows.
//
// A workgroup of four waves takes 32 * RW query rows of one (sequence, KV head)
// -- a row is a (token, head of the group) pair, so the group's heads share
// every K and V tile -- and walks a range of cache rows in tiles of KT.  RW
// waves side by side take 32 rows each; the 4 / RW waves behind each other
// split a tile's cache rows and are joined at the end, so that few rows still
// use every wave.  The products are S^T = K Q^T and O^T = V^T P^T on 32x32
// matrix instructions: a lane then holds one query row's scores (half of a
// tile's rows, the lane 32 further on the other half), so the row's maximum
// and sum stay in the lane, and the scores are already laid out as the second
// product's operand: the k index of that product is only renumbered, and V's
// operand is read in the same numbering.
#pragma once

#include <type_traits>

#include "cache_view.h"

namespace specv {
namespace attn {

constexpr int kThreads = 256;
constexpr float kSlack = 8.0f;

typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4b __attribute__((__vector_size__(4 * sizeof(__bf16))));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

struct Params {
  CacheView c;
  const char *q;
  long long q_stride;         // bytes from token to token
  char *out;                  // [tokens][Hq][D]
  float *lse;                 // [tokens][Hq] or NULL
  int32_t *status;
  int B, G;
  int T;                      // prompts: tokens in all
  const int32_t *cu;          // prompts: [B + 1]
  int N, words;               // trees: nodes per sequence, mask words per node
  const uint32_t *mask;       // trees: [B][N][words], or NULL: a chain
  float scale, sl;            // sl = scale * log2(e)
  int target, row_tiles;      // trees: pieces aimed at; row tiles per (sequence, KV head)
  int32_t *pieces;            // [group][2]: first slot and number of pieces
  float *part_o;              // [slot][32 * RW][D] partial outputs
  float2 *part_ml;            // [slot][32 * RW] maximum (of q.k) and sum
  int32_t *part_bad;          // [slot] whether a bad page was met
};

// What a workgroup works on: rows [0, R) are (token, group head) pairs of
// sequence b; token i sees cache rows below first_limit + i (prompts, chains).
struct Job {
  int b, h, row0;             // KV head; first row of the tile
  int tokens;                 // tokens of the sequence
  long long token0;           // its first token's index in q and out
  int limit0;                 // token 0 sees cache rows [0, limit0)
  int total;                  // cache rows of the sequence
  int t0, t1;                 // tiles of cache rows to walk
  int start_col;              // rectangle: column of row 0
};

template <typename T, int DP, int RW>
struct Shape {
  static constexpr int kElt = sizeof(T);
  static constexpr int kVec = 16 / kElt;                  // elements in 16 bytes
  static constexpr int kKW = 4 / RW;                      // waves that share a query row
  // cache rows a wave takes per tile, in blocks of 32
  static constexpr int kNB = RW == 4 && kElt == 2 ? 2 : 1;
  static constexpr int kKT = 32 * kNB * kKW;
  static constexpr int kChunks = DP / kVec;               // 16-byte chunks in a row
  static constexpr int kLoads = kKT * kChunks / kThreads; // chunks of K (or V) that a lane brings
  static constexpr int kTile = kKT * DP * kElt;           // bytes of K (or V)
  static constexpr int kLds = 2 * kTile;                  // of one buffer
  static constexpr int kJoin = RW * 32 * DP * 4;          // outputs of the RW waves side by side
  static constexpr int kJoins = kLds / kJoin;             // that many in a buffer
  static_assert(kLoads * kThreads == kKT * kChunks && (kKW == 1 || 2 * kJoins >= kKW) && 2 * kLds <= 160 * 1024 - 2048, "LDS");
};

// Chunk c of row r lies at LDS place r * CHUNKS + (c ^ turn(r)).  Rows of 256
// bytes and more all start at bank 0, so the chunk is exchanged by the row: four
// rows side by side (the block that a transposing read of V takes) get four
// different pairs of chunks, and sixteen rows (a read of K) sixteen different
// chunks.  Rows of 128 bytes start at two places, and eight chunks serve two rows
// each.
template <int CHUNKS>
__device__ inline int turn(int r) {
  if constexpr (CHUNKS >= 16)
    return ((r & 3) << 2) | ((r >> 2) & 3);
  else
    return (((r >> 1) & 1) << 2) | ((r >> 2) & 3);
}

__device__ inline float half_max(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return fmaxf(__uint_as_float(r[0]), __uint_as_float(r[1]));
}
__device__ inline float half_sum(float x) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}

__device__ inline f32x16 mfma(bf16x8 a, bf16x8 b, f32x16 c) {
  return __builtin_amdgcn_mfma_f32_32x32x16_bf16(a, b, c, 0, 0, 0);
}

// The transposing LDS read: of the 4 x 16 block whose row i / 4, columns
// 4 (i % 4) .. + 3 lane i of sixteen points at, lane i gets column i.
__device__ inline bf16x4b read_turned(const char *p) {
  typedef __attribute__((address_space(3))) bf16x4b *Lds;
  return __builtin_amdgcn_ds_read_tr16_b64_v4bf16((Lds) const_cast<char *>(p));
}

// A value that the compiler takes for new: what is computed from it stays where
// it is used.  Two dozen LDS addresses kept across a loop instead cost more
// registers than a wave has beside its tiles, and an xor each is free.
__device__ inline int fresh(int x) {
  asm volatile("" : "+v"(x));
  return x;
}

// The state of one wave's 32 query rows.
template <typename T, int DP>
struct Rows {
  static constexpr int kQ = DP / 16 * (sizeof(T) == 2 ? 1 : 2);
  typedef typename std::conditional<sizeof(T) == 2, bf16x8, f32x4>::type QV;
  QV q[kQ];
  f32x16 o[DP / 32];
  float m, l;                 // reference maximum of q.k; this half's sum
  float base;                 // m * scale * log2(e), 0 while m is -inf
};

// What a wave holds of its rows once the walk is over: with KW waves on the same
// rows the kw-th DP / KW elements, d = 8 (kw DP / 8 / KW + i) + 4 hf .. + 3.
template <int DP, int KW>
struct Done {
  f32x4 o[DP / 8 / KW];
  float m, l;
  int token, head, kw;
  bool mine;
};

// Brings K and V tiles from the cache straight into LDS.  A wave's load writes
// 64 consecutive 16-byte places, so a lane takes the chunk whose place its own
// is.  Where a tile's rows all exist and the kRows rows of a load lie in one
// page, the address is a scalar base and an offset that the lane keeps; else
// (the last tile, odd page sizes) each lane finds its row.  Chunks past D are
// never loaded: they stay zero (clear()).
// ONCE: the rows are read by one workgroup and not soon again: non-temporal.
template <typename T, int DP, int RW, bool PAGED, bool ONCE>
struct Loader {
  using S = Shape<T, DP, RW>;
  static constexpr int kRows = kWave / S::kChunks;        // rows of one wave's load
  const Params &P;
  const Job &J;
  int wave, lrow, c0;                                     // the lane's row in a load, and its chunk in the first
  int page;                                               // lane i: the page of load i of the next tile
  bool steady, bad;

  __device__ Loader(const Params &p, const Job &j) : P(p), J(j), page(0), bad(false) {
    const int lane = threadIdx.x & (kWave - 1);
    wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    lrow = lane / S::kChunks;
    c0 = lane % S::kChunks ^ turn<S::kChunks>(wave * kRows + lrow);
    steady = !PAGED || P.c.cols % kRows == 0;
  }
  // first row of load i of tile t, and the lane's chunk in it (turn() of rows 4 kRows apart: an xor)
  __device__ int row(int t, int i) const { return t * S::kKT + (4 * i + wave) * kRows; }
  __device__ int chunk(int i) const { return c0 ^ turn<S::kChunks>(4 * kRows * i); }
  __device__ bool has(int i) const { return DP == P.c.D || chunk(i) * S::kVec < P.c.D; }
  __device__ void clear(char *buf) const {
    if (P.c.D == DP) return;
    for (int x = threadIdx.x; x < S::kLds / 16; x += kThreads) reinterpret_cast<u32x4 *>(buf)[x] = u32x4{0, 0, 0, 0};
  }
  __device__ int page_of(int r) const {
    return P.c.table[static_cast<long long>(J.b) * P.c.max_pages + cache_page(P.c, r)];
  }
  __device__ int checked(int plane) {
    const bool ok = plane >= 0 && plane < P.c.planes;
    bad |= !ok;
    return ok ? plane : 0;
  }
  __device__ void pages(int t) {
    if constexpr (PAGED) page = page_of(min(row(t, threadIdx.x & (S::kLoads - 1)), J.total - 1));
  }
  __device__ void bring(const char *k, const char *v, int i, char *buf) const {
    typedef __attribute__((address_space(3))) char *Lds;
    typedef const __attribute__((address_space(1))) char *Global;
    char *to = buf + (i * kThreads + wave * kWave) * 16;
    __builtin_amdgcn_global_load_lds((Global)k, (Lds)to, 16, 0, ONCE ? 2 : 0);
    __builtin_amdgcn_global_load_lds((Global)v, (Lds)(to + S::kTile), 16, 0, ONCE ? 2 : 0);
  }
  template <bool FULL>                                    // FULL: D == DP, every chunk exists
  __device__ void load_steady(int t, char *buf) {
    const int row_bytes = P.c.D * S::kElt;
#pragma unroll
    for (int i = 0; i < S::kLoads; ++i) {
      const int r = row(t, i);
      int plane = J.b, col = J.start_col + r;
      if constexpr (PAGED) {
        plane = checked(read_lane(page, i));
        col = r - cache_page(P.c, r) * P.c.cols;
      }
      const long long off = cache_offset(P.c, plane, J.h, col, S::kElt);
      const uint32_t mine = lrow * row_bytes + chunk(i) * 16;
      if (FULL || has(i)) bring(P.c.k + off + mine, P.c.v + off + mine, i, buf);
    }
  }
  __device__ void load(int t, char *buf) {
    if ((t + 1) * S::kKT <= J.total && steady) {
      if (P.c.D == DP) load_steady<true>(t, buf);
      else load_steady<false>(t, buf);
      return;
    }
#pragma unroll
    for (int i = 0; i < S::kLoads; ++i) {
      const int r = min(row(t, i) + lrow, J.total - 1);
      int plane = J.b, col = J.start_col + r;
      if constexpr (PAGED) {
        plane = checked(page_of(r));
        col = r - cache_page(P.c, r) * P.c.cols;
      }
      const long long off = cache_offset(P.c, plane, J.h, col, S::kElt) + chunk(i) * 16;
      if (has(i)) bring(P.c.k + off, P.c.v + off, i, buf);
    }
  }
  // Takes infinities and NaNs out of the lane's own chunks of a V tile; whether
  // there were any.  An exponent of all ones carries into the bit above it.
  __device__ bool clean(char *buf) const {
    u32x4 *own = reinterpret_cast<u32x4 *>(buf + S::kTile) + threadIdx.x;
    constexpr uint32_t kExp = S::kElt == 2 ? 0x7f807f80u : 0x7f800000u, kOne = S::kElt == 2 ? 0x00800080u : 0x00800000u;
    constexpr uint32_t kTop = S::kElt == 2 ? 0x80008000u : 0x80000000u;
    uint32_t seen = 0;
#pragma unroll
    for (int i = 0; i < S::kLoads; ++i) {
      const u32x4 x = own[i * kThreads];
#pragma unroll
      for (int j = 0; j < 4; ++j) seen |= (x[j] & kExp) + kOne;
    }
    if (!(seen & kTop)) return false;
    for (int i = 0; i < S::kLoads; ++i) {
      u32x4 x = own[i * kThreads];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t odd = ((x[j] & kExp) + kOne) & kTop;   // the top bit of each value to clear
        x[j] &= S::kElt == 2 ? ~((odd >> 15) * 0xffffu) : odd ? 0u : ~0u;
      }
      own[i * kThreads] = x;
    }
    return true;
  }
};

// Which of cache rows [k0, k0 + 32) a query row sees, as bits.
template <bool PROMPT>
__device__ inline uint32_t seen(const Params &P, const Job &J, int token, int k0) {
  int limit = J.limit0 + token;                           // prompts and chains
  uint32_t bits = 0;
  if (!PROMPT && P.mask) {
    limit = J.limit0 - 1;                                 // the rows before the tree's
    const int j = k0 - limit;                             // node of bit 0
    if (j > -32 && j < P.N) {
      const uint32_t *w = P.mask + (static_cast<long long>(J.b) * P.N + token) * P.words;
      const int i = j >> 5, s = j & 31;                   // floor: i may be -1
      const uint32_t lo = i >= 0 ? w[i] : 0u, hi = i + 1 < P.words ? w[i + 1] : 0u;
      bits = static_cast<uint32_t>(((static_cast<uint64_t>(hi) << 32) | lo) >> s);
    }
  }
  const int below = limit - k0;
  const uint32_t cached = below >= 32 ? ~0u : below <= 0 ? 0u : (1u << below) - 1u;
  const int left = J.total - k0;                          // bits past the tree's end
  const uint32_t valid = left >= 32 ? ~0u : left <= 0 ? 0u : (1u << left) - 1u;
  return (bits | cached) & valid;
}

// One tile: the wave's scores, the softmax step and the second product.
// kb0: the wave's first cache row in the tile; vis: seen() of its blocks.
// turn() is the same for rows 16 apart and differs by 2 for rows 8 apart, so
// all of a lane's places are one offset, with an xor of constant bits for the
// chunk and a constant distance for the row.
template <typename T, int DP, int RW, bool MASKED>
__device__ inline void step(Rows<T, DP> &W, const char *lds, int kb0, float sl,
                            const uint32_t (&vis)[Shape<T, DP, RW>::kNB]) {
  using S = Shape<T, DP, RW>;
  constexpr int kRow = DP * S::kElt;
  const int lane = threadIdx.x & (kWave - 1), n = lane & 31, hf = lane >> 5;
  const char *ldk = lds, *ldv = lds + S::kTile;
  f32x16 s[S::kNB];
#pragma unroll
  for (int nb = 0; nb < S::kNB; ++nb)
#pragma unroll
    for (int r = 0; r < 16; ++r) s[nb][r] = 0.0f;
  const int ka = fresh((kb0 + n) * kRow + ((hf ^ turn<S::kChunks>(n)) << 4));
  const int i16 = lane & 15, dg = (lane >> 4) & 1, r0 = 4 * hf + (i16 >> 2);
  const int va16 = fresh((kb0 + r0) * kRow + (((2 * dg + ((i16 & 3) >> 1)) ^ turn<S::kChunks>(r0)) << 4) + (i16 & 1) * 8);
  bf16x8 v[2][DP / 32];                                   // V's operand for 16 rows, and the next 16
  auto read_v = [&](int t) __attribute__((always_inline)) {
#pragma unroll
    for (int db = 0; db < DP / 32; ++db) {
      const bf16x4b lo = read_turned(ldv + (va16 ^ (db << 6)) + 16 * t * kRow);
      const bf16x4b hi = read_turned(ldv + (va16 ^ (db << 6 | 2 << 4)) + (16 * t + 8) * kRow);
      v[t & 1][db] = bf16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    }
  };
  if constexpr (S::kElt == 2) {
    // All of a block's K operands are asked for before the first product, the
    // next block's (or V's first) while the products run: left to itself the
    // compiler asks for each just before its use and waits out the LDS latency
    // sixteen times a tile.
    auto read_k = [&](int nb, int d) __attribute__((always_inline)) {
      return *reinterpret_cast<const bf16x8 *>(ldk + (ka ^ (d << 5)) + nb * 32 * kRow);
    };
    bf16x8 a[DP / 16];
#pragma unroll
    for (int d = 0; d < DP / 16; ++d) a[d] = read_k(0, d);
    __builtin_amdgcn_sched_group_barrier(0x100, DP / 16, 0);
#pragma unroll
    for (int nb = 0; nb < S::kNB; ++nb) {
#pragma unroll
      for (int d = 0; d < DP / 16; ++d) {
        s[nb] = mfma(a[d], W.q[d], s[nb]);
        if (nb + 1 < S::kNB) a[d] = read_k(nb + 1, d);
      }
      if (nb + 1 == S::kNB) read_v(0);
#pragma unroll
      for (int d = 0; d < DP / 16; ++d) {
        __builtin_amdgcn_sched_group_barrier(0x008, 1, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
      }
    }
  } else {
#pragma unroll
    for (int nb = 0; nb < S::kNB; ++nb)
#pragma unroll
      for (int d = 0; d < DP / 8; ++d) {
        const f32x4 a = *reinterpret_cast<const f32x4 *>(ldk + (ka ^ (d << 5)) + nb * 32 * kRow);
#pragma unroll
        for (int j = 0; j < 4; ++j) s[nb] = __builtin_amdgcn_mfma_f32_32x32x2f32(a[j], W.q[d][j], s[nb], 0, 0, 0);
      }
  }
  if constexpr (MASKED) {
#pragma unroll
    for (int nb = 0; nb < S::kNB; ++nb) {
      const uint32_t see = vis[nb] >> (4 * hf);
#pragma unroll
      for (int r = 0; r < 16; ++r) s[nb][r] = (see >> (8 * (r / 4) + r % 4)) & 1u ? s[nb][r] : -INFINITY;
    }
  }
  float mx = s[0][0];
#pragma unroll
  for (int nb = 0; nb < S::kNB; ++nb)
#pragma unroll
    for (int r = 0; r < 16; ++r) mx = fmaxf(mx, s[nb][r]);
  // The weights are exp(s - m) for a reference m that follows the maximum only
  // when some row's has outgrown it by 2^kSlack: sums and weights stay within
  // 2^kSlack of what the maximum itself would give, at the same relative
  // precision, and most tiles leave the outputs as they are.
  mx = half_max(mx);
  if (__any(fmaf(mx, sl, -W.base) > kSlack || (W.m == -INFINITY && mx > -INFINITY))) {
    const float m = fmaxf(W.m, mx);
    const float base = m == -INFINITY ? 0.0f : m * sl;    // nothing seen yet: every exponent is -inf
    const float alpha = __builtin_amdgcn_exp2f(fmaf(W.m, sl, -base));
    W.m = m;
    W.base = base;
    W.l *= alpha;
#pragma unroll
    for (int db = 0; db < DP / 32; ++db)
#pragma unroll
      for (int r = 0; r < 16; ++r) W.o[db][r] *= alpha;
  }
  const float base = W.base;
  float sum = 0.0f;
#pragma unroll
  for (int nb = 0; nb < S::kNB; ++nb)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      s[nb][r] = __builtin_amdgcn_exp2f(fmaf(s[nb][r], sl, -base));
      sum += s[nb][r];
    }
  W.l += sum;

  // O^T += V^T P^T.  For the bf16 product the weights are rounded to bf16: off by at
  // most half a step, 2^-8 of a weight, like the one rounding of the result; their
  // sum is of the unrounded ones.
  if constexpr (S::kElt == 2) {
#pragma unroll
    for (int t = 0; t < 2 * S::kNB; ++t) {
      if (t + 1 < 2 * S::kNB) read_v(t + 1);
      bf16x8 p;
#pragma unroll
      for (int j = 0; j < 8; ++j) p[j] = static_cast<__bf16>(s[t / 2][8 * (t % 2) + j]);
#pragma unroll
      for (int db = 0; db < DP / 32; ++db) W.o[db] = mfma(v[t & 1][db], p, W.o[db]);
    }
  } else {
    const int va = fresh((kb0 + 4 * hf) * kRow + ((n / 4 ^ hf) << 4) + n % 4 * 4);
#pragma unroll
    for (int r = 0; r < 16 * S::kNB; ++r) {
      const float p = s[r / 16][r % 16];
      const int row = 32 * (r / 16) + 8 * (r % 16 / 4) + r % 4;
#pragma unroll
      for (int db = 0; db < DP / 32; ++db) {
        const float a = *reinterpret_cast<const float *>(ldv + (va ^ (db << 7) ^ (turn<S::kChunks>(row) << 4)) + row * kRow);
        W.o[db] = __builtin_amdgcn_mfma_f32_32x32x2f32(a, p, W.o[db], 0, 0, 0);
      }
    }
  }
}

// In tiles that some rows do not see whole, V rows may hold anything where they
// are not seen, and 0 * inf is not 0.  Such a tile's infinities and NaNs are
// zero in LDS (clean()); here they are added to the query rows that see them,
// from the cache itself.  Rare: one row of the cache after the other.
template <typename T, int DP, int RW, bool PAGED>
__device__ inline void add_odd(const Params &P, const Job &J, Rows<T, DP> &W, int k0,
                               const uint32_t (&vis)[Shape<T, DP, RW>::kNB]) {
  using S = Shape<T, DP, RW>;
  const int hf = fresh(threadIdx.x & (kWave - 1)) >> 5;
  for (int j = 0; j < 32 * S::kNB; ++j) {
    const int r = k0 + j;
    if (r >= J.total) break;
    uint32_t word = vis[0];
    if constexpr (S::kNB == 2) word = j < 32 ? vis[0] : vis[1];
    const bool see = (word >> (j & 31)) & 1u;
    int plane = J.b, col = J.start_col + r;
    if constexpr (PAGED) {
      plane = P.c.table[static_cast<long long>(J.b) * P.c.max_pages + cache_page(P.c, r)];
      if (plane < 0 || plane >= P.c.planes) plane = 0;
      col = r - cache_page(P.c, r) * P.c.cols;
    }
    const T *v = reinterpret_cast<const T *>(P.c.v + cache_offset(P.c, plane, J.h, col, S::kElt));
#pragma unroll
    for (int db = 0; db < DP / 32; ++db)
#pragma unroll
      for (int i = 0; i < 16; ++i) {
        const int d = 32 * db + 8 * (i / 4) + 4 * hf + i % 4;
        const float x = d < P.c.D ? static_cast<float>(v[d]) : 0.0f;
        if (see && !(fabsf(x) < INFINITY)) W.o[db][i] += x;
      }
  }
}

// Four values of a query row's output, d = d0 .. d0 + 3.
template <typename T>
__device__ inline void put4(char *out, int d0, int D, const float (&x)[4]) {
  if (d0 >= D) return;                                    // D is a multiple of 4
  if constexpr (sizeof(T) == 2) {
    bf16x4 y;
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = static_cast<__bf16>(x[j]);
    *reinterpret_cast<bf16x4 *>(out + d0 * 2) = y;
  } else {
    *reinterpret_cast<f32x4 *>(out + d0 * 4) = f32x4{x[0], x[1], x[2], x[3]};
  }
}

// The walk of one job.  Each wave returns with its share of its rows' unscaled
// outputs (of KW waves on the same rows the kw-th has the kw-th DP / KW
// elements) and with the rows' maxima and sums over all of them; all return
// whether a bad page was met.
template <typename T, int DP, int RW, bool PAGED, bool PROMPT, bool ONCE>
__device__ inline bool walk(const Params &P, const Job &J, Done<DP, Shape<T, DP, RW>::kKW> &D, char *buf0,
                            char *buf1) {
  using S = Shape<T, DP, RW>;
  const int lane = fresh(threadIdx.x & (kWave - 1)), n = lane & 31, hf = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), rw = wave % RW, kw = wave / RW;
  Loader<T, DP, RW, PAGED, ONCE> ld(P, J);
  ld.clear(buf0);
  ld.clear(buf1);
  if (P.c.D != DP) __syncthreads();                       // the zeros are there
  if (J.t0 < J.t1) {
    ld.pages(J.t0);
    ld.load(J.t0, buf0);
    ld.pages(min(J.t0 + 1, J.t1 - 1));
  }
  const int R = J.tokens * P.G;
  const int row = min(J.row0 + rw * 32 + n, R - 1);       // rows past the end repeat the last
  const int token = row / P.G, head = J.h * P.G + (row - token * P.G);
  D.mine = J.row0 + rw * 32 + n < R;
  D.token = token;
  D.head = head;
  D.kw = kw;
  Rows<T, DP> W;
  {
    const char *q = P.q + (J.token0 + token) * P.q_stride + static_cast<long long>(head) * P.c.D * S::kElt;
    typedef typename Rows<T, DP>::QV QV;
#pragma unroll
    for (int d = 0; d < Rows<T, DP>::kQ; ++d) {
      const int at = (2 * d + hf) * S::kVec;
      W.q[d] = at < P.c.D ? *reinterpret_cast<const QV *>(q + at * S::kElt) : QV{};
    }
  }
#pragma unroll
  for (int db = 0; db < DP / 32; ++db)
#pragma unroll
    for (int r = 0; r < 16; ++r) W.o[db][r] = 0.0f;
  W.m = -INFINITY;
  W.l = W.base = 0.0f;
  // cache rows below `plain` are seen by every row of the workgroup
  const int plain = !PROMPT && P.mask ? J.limit0 - 1 : J.limit0 + J.row0 / P.G;
  // Tile t is used from one buffer while tile t + 1 arrives in the other.
  const int kb0 = kw * 32 * S::kNB;
  const int mid = min(J.t1, plain / S::kKT);              // tiles before it every row sees whole
  __shared__ int flags[2];                                // V rows with infinities or NaNs; bad pages: once met, kept
  if (threadIdx.x < 2) flags[threadIdx.x] = 0;
  auto begin = [&](int t, char *next) __attribute__((always_inline)) {
    __builtin_amdgcn_s_waitcnt(0x0f70);                   // vmcnt(0): this wave's part of tile t is in LDS
    __syncthreads();                                      // everyone's is, and tile t - 1 is read
    if (t + 1 < J.t1) {
      ld.load(t + 1, next);
      ld.pages(min(t + 2, J.t1 - 1));
    }
  };
  auto masked = [&](int t, char *now, char *next) __attribute__((always_inline)) {
    begin(t, next);
    uint32_t vis[S::kNB];
#pragma unroll
    for (int nb = 0; nb < S::kNB; ++nb) vis[nb] = ~0u;
    bool odd = false;
    if (t >= mid) {
#pragma unroll
      for (int nb = 0; nb < S::kNB; ++nb) vis[nb] = seen<PROMPT>(P, J, token, t * S::kKT + kb0 + 32 * nb);
      if (ld.clean(now)) flags[0] = 1;
      __syncthreads();
      odd = flags[0] != 0;
    }
    step<T, DP, RW, true>(W, now, kb0, P.sl, vis);
    if (odd) add_odd<T, DP, RW, PAGED>(P, J, W, t * S::kKT + kb0, vis);
  };
  int t = J.t0;
  if constexpr (RW == 4) {
    // bound by the matrix and vector units: whole tiles without the masks
    auto whole = [&](int t, char *now, char *next) __attribute__((always_inline)) {
      begin(t, next);
      const uint32_t all[S::kNB] = {};
      step<T, DP, RW, false>(W, now, kb0, P.sl, all);
    };
    char *now = buf0, *next = buf1;
    for (; t + 1 < mid; t += 2) {
      whole(t, buf0, buf1);
      whole(t + 1, buf1, buf0);
    }
    if (t < mid) {
      whole(t++, buf0, buf1);
      now = buf1;
      next = buf0;
    }
    for (; t < J.t1; ++t) {
      masked(t, now, next);
      char *x = now;
      now = next;
      next = x;
    }
  } else {
    // bound by memory, or short: one code for all tiles, since the first pass of
    // a wave through code that is not in the instruction cache takes longer than
    // the masks (single-token calls end with a partial tile)
    for (; t < J.t1; t += 2) {
      masked(t, buf0, buf1);
      if (t + 1 < J.t1) masked(t + 1, buf1, buf0);
    }
  }
  W.l = half_sum(W.l);
  if constexpr (S::kKW > 1) {
    // Join the waves that shared the rows.  Each leaves its outputs in LDS, four
    // values of a row side by side, and takes its share of the row's elements
    // from all of them, scaled to the common maximum.
    __syncthreads();                                      // the tiles are read
    __shared__ float2 jm[4][32];
    auto place_of = [&](int k) {                          // [rw][DP / 4][32] of the k-th wave behind each other
      char *buf = k < S::kJoins ? buf0 + k * S::kJoin : buf1 + (k - S::kJoins) * S::kJoin;
      return reinterpret_cast<f32x4 *>(buf) + rw * (DP / 4 * 32) + hf * 32 + n;
    };
    f32x4 *mine = place_of(kw);
#pragma unroll
    for (int q = 0; q < DP / 8; ++q)                      // q = 4 db + g: d = 8 q + 4 hf ..
      mine[q * 64] = f32x4{W.o[q / 4][4 * (q % 4)], W.o[q / 4][4 * (q % 4) + 1], W.o[q / 4][4 * (q % 4) + 2],
                           W.o[q / 4][4 * (q % 4) + 3]};
    if (hf == 0) jm[wave][n] = make_float2(W.m, W.l);
    __syncthreads();
    float2 ml[S::kKW];
    float top = -INFINITY;
#pragma unroll
    for (int k = 0; k < S::kKW; ++k) {
      ml[k] = jm[k * RW + rw][n];
      top = fmaxf(top, ml[k].x);
    }
    const float base = top == -INFINITY ? 0.0f : top;
    D.m = top;
    D.l = 0.0f;
    constexpr int kMine = DP / 8 / S::kKW;                // quads of this wave
#pragma unroll
    for (int i = 0; i < kMine; ++i) D.o[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < S::kKW; ++k) {
      const float f = __builtin_amdgcn_exp2f((ml[k].x - base) * P.sl);
      D.l = fmaf(ml[k].y, f, D.l);
      const f32x4 *o = place_of(k) + kw * kMine * 64;
#pragma unroll
      for (int i = 0; i < kMine; ++i) D.o[i] += o[i * 64] * f;
    }
  } else {
    D.m = W.m;
    D.l = W.l;
#pragma unroll
    for (int q = 0; q < DP / 8; ++q)
      D.o[q] = f32x4{W.o[q / 4][4 * (q % 4)], W.o[q / 4][4 * (q % 4) + 1], W.o[q / 4][4 * (q % 4) + 2],
                        W.o[q / 4][4 * (q % 4) + 3]};
  }
  if (!PAGED || !P.status) return false;
  if (ld.bad) flags[1] = 1;
  __syncthreads();
  return flags[1] != 0;
}

// Trees: whether a node's mask row has any bit (else it sees nothing at all).
__device__ inline bool sees_any(const Params &P, int b, int token) {
  if (!P.mask) return true;
  uint32_t any = 0;
  for (int i = 0; i < P.words; ++i) any |= P.mask[(static_cast<long long>(b) * P.N + token) * P.words + i];
  return any != 0;
}

// Final results of a wave's rows.  A row that saw nothing has sum 0 (its
// maximum is -inf): zeros.
template <typename T, int DP, int KW>
__device__ inline void put_rows(const Params &P, const Job &J, const Done<DP, KW> &D, bool sees) {
  const int hf = fresh(threadIdx.x & (kWave - 1)) >> 5;
  if (!D.mine) return;
  const bool none = !sees || D.l == 0.0f;
  const float f = none ? 0.0f : 1.0f / D.l;
  const long long at = (J.token0 + D.token) * P.c.H * P.G + D.head;
  char *o = P.out + at * P.c.D * sizeof(T);
#pragma unroll
  for (int i = 0; i < DP / 8 / KW; ++i) {
    float x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = none ? 0.0f : D.o[i][j] * f;
    put4<T>(o, 8 * (D.kw * (DP / 8 / KW) + i) + 4 * hf, P.c.D, x);
  }
  if (P.lse && hf == 0 && D.kw == 0) P.lse[at] = none ? -INFINITY : D.m * P.scale + logf(D.l);
}

// Zeros for the rows of a job whose sequence's state is out of range.
template <typename T>
__device__ inline void put_zeros(const Params &P, const Job &J, int rows) {
  const int R = J.tokens * P.G, hi = min(J.row0 + rows, R), D = P.c.D;
  for (int x = threadIdx.x; x < (hi - J.row0) * (D / 4); x += kThreads) {
    const int row = J.row0 + x / (D / 4), token = row / P.G;
    const long long at = (J.token0 + token) * P.c.H * P.G + J.h * P.G + (row - token * P.G);
    const float z[4] = {};
    put4<T>(P.out + at * D * sizeof(T), x % (D / 4) * 4, D, z);
    if (P.lse && x % (D / 4) == 0) P.lse[at] = -INFINITY;
  }
}

// Host checks that both calls share; fills what they share.
inline int fill(Params &P, const void *q, int64_t q_stride, const void *kv, spec_dtype dt, int L, int planes, int B,
                int H, int cols, int D, int layer, int G, const int32_t *table, int max_pages, bool paged,
                const int32_t *end_col, const int32_t *kv_len, float scale, void *out, float *lse, int32_t *status) {
  if (!q || !out) return SPEC_EINVAL;
  const int err = cache_view(P.c, kv, dt, L, planes, H, cols, D, layer, table, max_pages, paged, end_col, kv_len);
  if (err) return err;
  if (B < 1 || G < 1 || (!paged && planes != B)) return SPEC_EINVAL;
  if (!(scale > 0.0f) || scale > 2e38f) return SPEC_EINVAL;   // sl stays finite
  if (D > SPEC_ATTN_MAX_D) return SPEC_ECAPACITY;
  if (static_cast<long long>(H) * G >= INT32_MAX / SPEC_ATTN_MAX_D) return SPEC_EINVAL;
  const int elt = dt == SPEC_BF16 ? 2 : 4;
  if (D * elt % 16 || q_stride < static_cast<long long>(H) * G * D || q_stride * elt % 16) return SPEC_EINVAL;
  if (!aligned(q, 16) || !aligned(kv, 16) || !aligned(out, 16) || !aligned(lse, 4) || !aligned(status, 4))
    return SPEC_EINVAL;
  P.q = static_cast<const char *>(q);
  P.q_stride = q_stride * elt;
  P.out = static_cast<char *>(out);
  P.lse = lse;
  P.status = status;
  P.B = B;
  P.G = G;
  P.T = 0;
  P.cu = nullptr;
  P.N = P.words = 0;
  P.mask = nullptr;
  P.scale = scale;
  P.sl = scale * 1.44269504088896340736f;
  P.target = P.row_tiles = 1;
  P.part_o = nullptr;
  P.part_ml = nullptr;
  P.part_bad = P.pieces = nullptr;
  return SPEC_OK;
}

}  // namespace attn
}  // namespace specv
