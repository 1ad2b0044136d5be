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
  int splits, row_tiles;      // trees
  float *part_o;              // [slot][32 * RW][D], slot = ((b * H + h) * row_tiles + rt) * splits + s
  float *part_ml;             // [slot][32 * RW][2]: maximum (of q.k) and sum
  int32_t *part_bad;          // [slot]: status bits found on the way
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
  static constexpr int kRowsPass = kThreads / kChunks;    // rows the workgroup loads at once
  static constexpr int kLoads = kKT / kRowsPass;
  static constexpr int kTile = kKT * DP * kElt;           // bytes of K (or V)
  static constexpr int kJoin = (kKW - 1) * RW * 32 * (DP + 2) * 4;
  static constexpr int kLds = 2 * kTile > kJoin ? 2 * kTile : kJoin;
  static_assert(kRowsPass * kLoads == kKT, "whole passes");
};

// LDS place of chunk c of row r.  Rows of 256 bytes and more all start at bank
// 0, so the chunk is exchanged by the row: four rows side by side (the block
// that a transposing read of V takes) get four different pairs of chunks, and
// sixteen rows (a read of K) sixteen different chunks.  Rows of 128 bytes
// start at two places, and eight chunks serve two rows each.
template <int CHUNKS>
__device__ inline int place(int r, int c) {
  if constexpr (CHUNKS >= 16)
    return r * CHUNKS + (c ^ (((r & 3) << 2) | ((r >> 2) & 3)));
  else
    return r * CHUNKS + (c ^ ((((r >> 1) & 1) << 2) | ((r >> 2) & 3)));
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

// Whether a word of two bf16 values holds an infinity or a NaN.
__device__ inline bool odd2(uint32_t w) {
  return (w & 0x7f800000u) == 0x7f800000u || (w & 0x7f80u) == 0x7f80u;
}

// The state of one wave's 32 query rows.
template <typename T, int DP>
struct Rows {
  static constexpr int kQ = DP / 16 * (sizeof(T) == 2 ? 1 : 2);
  typedef typename std::conditional<sizeof(T) == 2, bf16x8, f32x4>::type QV;
  QV q[kQ];
  f32x16 o[DP / 32];
  float m, l;                 // maximum of q.k so far; this half's sum
  uint32_t sees;              // trees: any bit of the row's mask
};

// Loads of one K and V tile into registers, and their store to LDS.
template <typename T, int DP, int RW, bool PAGED>
struct Loader {
  using S = Shape<T, DP, RW>;
  const Params &P;
  const Job &J;
  int chunk, row;
  bool in;
  int page[S::kLoads];
  int bad;
  u32x4 k[S::kLoads], v[S::kLoads];

  __device__ Loader(const Params &p, const Job &j) : P(p), J(j), bad(0) {
    chunk = threadIdx.x % S::kChunks;
    row = threadIdx.x / S::kChunks;
    in = chunk * S::kVec < P.c.D;
  }
  __device__ int at(int t, int i) const { return min(t * S::kKT + i * S::kRowsPass + row, J.total - 1); }
  __device__ void pages(int t) {
    if constexpr (PAGED) {
#pragma unroll
      for (int i = 0; i < S::kLoads; ++i)
        page[i] = P.c.table[static_cast<long long>(J.b) * P.c.max_pages + cache_page(P.c, at(t, i))];
    }
  }
  __device__ void load(int t) {
#pragma unroll
    for (int i = 0; i < S::kLoads; ++i) {
      const int r = at(t, i);
      int plane = J.b, col = J.start_col + r;
      if constexpr (PAGED) {
        plane = page[i];
        col = r - cache_page(P.c, r) * P.c.cols;
        if (plane < 0 || plane >= P.c.planes) {
          bad = SPEC_ST_BAD_STATE;
          plane = 0;
        }
      }
      const long long off = cache_offset(P.c, plane, J.h, col, S::kElt) + chunk * 16;
      k[i] = v[i] = u32x4{0, 0, 0, 0};
      if (in) {
        k[i] = *reinterpret_cast<const u32x4 *>(P.c.k + off);
        v[i] = *reinterpret_cast<const u32x4 *>(P.c.v + off);
      }
    }
  }
  __device__ void store(char *lds) const {
#pragma unroll
    for (int i = 0; i < S::kLoads; ++i) {
      const int at = place<S::kChunks>(i * S::kRowsPass + row, chunk) * 16;
      *reinterpret_cast<u32x4 *>(lds + at) = k[i];
      *reinterpret_cast<u32x4 *>(lds + S::kTile + at) = v[i];
    }
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
template <typename T, int DP, int RW, bool MASKED>
__device__ inline void step(Rows<T, DP> &W, const char *lds, int kb0, float sl,
                            const uint32_t (&vis)[Shape<T, DP, RW>::kNB]) {
  using S = Shape<T, DP, RW>;
  const int lane = threadIdx.x & (kWave - 1), n = lane & 31, hf = lane >> 5;
  const char *ldk = lds, *ldv = lds + S::kTile;
  f32x16 s[S::kNB];
#pragma unroll
  for (int nb = 0; nb < S::kNB; ++nb) {
#pragma unroll
    for (int r = 0; r < 16; ++r) s[nb][r] = 0.0f;
    const int row = kb0 + nb * 32 + n;
    if constexpr (S::kElt == 2) {
#pragma unroll
      for (int d = 0; d < DP / 16; ++d) {
        const bf16x8 a = *reinterpret_cast<const bf16x8 *>(ldk + place<S::kChunks>(row, 2 * d + hf) * 16);
        s[nb] = mfma(a, W.q[d], s[nb]);
      }
    } else {
#pragma unroll
      for (int d = 0; d < DP / 8; ++d) {
        const f32x4 a = *reinterpret_cast<const f32x4 *>(ldk + place<S::kChunks>(row, 2 * d + hf) * 16);
#pragma unroll
        for (int j = 0; j < 4; ++j) s[nb] = __builtin_amdgcn_mfma_f32_32x32x2f32(a[j], W.q[d][j], s[nb], 0, 0, 0);
      }
    }
  }
  uint32_t see[S::kNB];
  if constexpr (MASKED) {
#pragma unroll
    for (int nb = 0; nb < S::kNB; ++nb) {
      see[nb] = vis[nb] >> (4 * hf);
#pragma unroll
      for (int r = 0; r < 16; ++r)
        s[nb][r] = (see[nb] >> (8 * (r / 4) + r % 4)) & 1u ? s[nb][r] : -INFINITY;
    }
  }
  float mx = s[0][0];
#pragma unroll
  for (int nb = 0; nb < S::kNB; ++nb)
#pragma unroll
    for (int r = 0; r < 16; ++r) mx = fmaxf(mx, s[nb][r]);
  const float m = fmaxf(W.m, half_max(mx));
  const float base = m == -INFINITY ? 0.0f : m * sl;      // nothing seen yet: every exponent is -inf
  const float alpha = __builtin_amdgcn_exp2f(fmaf(W.m, sl, -base));
  W.m = m;
  float sum = 0.0f;
#pragma unroll
  for (int nb = 0; nb < S::kNB; ++nb)
#pragma unroll
    for (int r = 0; r < 16; ++r) {
      s[nb][r] = __builtin_amdgcn_exp2f(fmaf(s[nb][r], sl, -base));
      sum += s[nb][r];
    }
  W.l = fmaf(W.l, alpha, sum);
#pragma unroll
  for (int db = 0; db < DP / 32; ++db)
#pragma unroll
    for (int r = 0; r < 16; ++r) W.o[db][r] *= alpha;

  // O^T += V^T P^T.  In masked tiles V rows that a query does not see may hold
  // anything, and 0 * inf is not 0: infinities and NaNs are taken out of the
  // operand and added by a product of their own with the rows' visibility.
  if constexpr (S::kElt == 2) {
    const int i = lane & 15, dg = (lane >> 4) & 1;
#pragma unroll
    for (int t = 0; t < 2 * S::kNB; ++t) {
      bf16x8 p;
#pragma unroll
      for (int j = 0; j < 8; ++j) p[j] = static_cast<__bf16>(s[t / 2][8 * (t % 2) + j]);
      const int r0 = kb0 + 16 * t + 4 * hf + (i >> 2);
#pragma unroll
      for (int db = 0; db < DP / 32; ++db) {
        const int c = 4 * db + 2 * dg + ((i & 3) >> 1), e = (i & 1) * 8;
        const bf16x4b lo = read_turned(ldv + place<S::kChunks>(r0, c) * 16 + e);
        const bf16x4b hi = read_turned(ldv + place<S::kChunks>(r0 + 8, c) * 16 + e);
        bf16x8 a = {lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
        if constexpr (MASKED) {
          u32x4 w = __builtin_bit_cast(u32x4, a);
          if (__any(odd2(w[0]) || odd2(w[1]) || odd2(w[2]) || odd2(w[3]))) {
            bf16x8 up, down, vs;
#pragma unroll
            for (int j = 0; j < 8; ++j) {
              const float x = static_cast<float>(a[j]);
              const bool nan = x != x;
              up[j] = static_cast<__bf16>(nan || x == INFINITY ? 1.0f : 0.0f);
              down[j] = static_cast<__bf16>(nan || x == -INFINITY ? 1.0f : 0.0f);
              if (nan || fabsf(x) == INFINITY) a[j] = static_cast<__bf16>(0.0f);
              const int r = 8 * (t % 2) + j;
              vs[j] = static_cast<__bf16>((see[t / 2] >> (8 * (r / 4) + r % 4)) & 1u ? 1.0f : 0.0f);
            }
            f32x16 z = {};
            const f32x16 u = mfma(up, vs, z), d = mfma(down, vs, z);
#pragma unroll
            for (int r = 0; r < 16; ++r) W.o[db][r] += (u[r] > 0 ? INFINITY : 0.0f) + (d[r] > 0 ? -INFINITY : 0.0f);
          }
        }
        W.o[db] = mfma(a, p, W.o[db]);
      }
    }
  } else {
#pragma unroll
    for (int r = 0; r < 16 * S::kNB; ++r) {
      const int row = kb0 + 32 * (r / 16) + 8 * (r % 16 / 4) + 4 * hf + r % 4;
      const float p = s[r / 16][r % 16];
#pragma unroll
      for (int db = 0; db < DP / 32; ++db) {
        float a = *reinterpret_cast<const float *>(ldv + place<S::kChunks>(row, 8 * db + n / 4) * 16 + n % 4 * 4);
        if constexpr (MASKED) {
          if (__any(!(fabsf(a) < INFINITY))) {
            const float up = a == INFINITY || a != a ? 1.0f : 0.0f, down = a == -INFINITY || a != a ? 1.0f : 0.0f;
            const float vs = (see[r / 16] >> (8 * (r % 16 / 4) + r % 4)) & 1u ? 1.0f : 0.0f;
            if (!(fabsf(a) < INFINITY)) a = 0.0f;
            f32x16 z = {};
            const f32x16 u = __builtin_amdgcn_mfma_f32_32x32x2f32(up, vs, z, 0, 0, 0);
            const f32x16 d = __builtin_amdgcn_mfma_f32_32x32x2f32(down, vs, z, 0, 0, 0);
#pragma unroll
            for (int x = 0; x < 16; ++x) W.o[db][x] += (u[x] > 0 ? INFINITY : 0.0f) + (d[x] > 0 ? -INFINITY : 0.0f);
          }
        }
        W.o[db] = __builtin_amdgcn_mfma_f32_32x32x2f32(a, p, W.o[db], 0, 0, 0);
      }
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

// The whole walk of one job.  slot < 0: outputs are final; else partials.
template <typename T, int DP, int RW, bool PAGED, bool PROMPT>
__device__ inline int walk(const Params &P, const Job &J, long long slot, char *lds) {
  using S = Shape<T, DP, RW>;
  const int lane = threadIdx.x & (kWave - 1), n = lane & 31, hf = lane >> 5;
  const int wave = threadIdx.x / kWave, rw = wave % RW, kw = wave / RW;
  const int R = J.tokens * P.G;
  const int row = min(J.row0 + rw * 32 + n, R - 1);       // rows past the end repeat the last
  const bool mine = J.row0 + rw * 32 + n < R;
  const int token = row / P.G, head = J.h * P.G + (row - token * P.G);
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
  W.l = 0.0f;
  W.sees = 1;
  if (!PROMPT && P.mask) {
    W.sees = 0;
    for (int i = 0; i < P.words; ++i)
      W.sees |= P.mask[(static_cast<long long>(J.b) * P.N + token) * P.words + i];
  }
  // cache rows below `plain` are seen by every row of the workgroup
  const int plain = !PROMPT && P.mask ? J.limit0 - 1 : J.limit0 + J.row0 / P.G;
  Loader<T, DP, RW, PAGED> ld(P, J);
  if (J.t0 < J.t1) {
    ld.pages(J.t0);
    ld.load(J.t0);
    ld.pages(min(J.t0 + 1, J.t1 - 1));
  }
  for (int t = J.t0; t < J.t1; ++t) {
    __syncthreads();                                      // the tile before is read
    ld.store(lds);
    if (t + 1 < J.t1) {
      ld.load(t + 1);
      ld.pages(min(t + 2, J.t1 - 1));
    }
    __syncthreads();
    const int kb0 = kw * 32 * S::kNB, k0 = t * S::kKT + kb0;
    uint32_t vis[S::kNB] = {};
    if (t * S::kKT + S::kKT <= plain) {
      step<T, DP, RW, false>(W, lds, kb0, P.sl, vis);
    } else {
#pragma unroll
      for (int nb = 0; nb < S::kNB; ++nb) vis[nb] = seen<PROMPT>(P, J, token, k0 + 32 * nb);
      step<T, DP, RW, true>(W, lds, kb0, P.sl, vis);
    }
  }
  float l = half_sum(W.l), m = W.m;
  // Join the waves that shared the rows: each brings its maximum, sum and
  // output; the first adds them, scaled to the common maximum.
  if constexpr (S::kKW > 1) {
    __syncthreads();
    float *jo = reinterpret_cast<float *>(lds);           // [kw - 1][rw][DP][32]
    float *jm = jo + (S::kKW - 1) * RW * 32 * DP;         // [kw - 1][rw][2][32]
    if (kw > 0) {
      float *o = jo + ((kw - 1) * RW + rw) * 32 * DP;
#pragma unroll
      for (int db = 0; db < DP / 32; ++db)
#pragma unroll
        for (int r = 0; r < 16; ++r) o[(32 * db + 8 * (r / 4) + 4 * hf + r % 4) * 32 + n] = W.o[db][r];
      if (hf == 0) {
        float *x = jm + ((kw - 1) * RW + rw) * 64;
        x[n] = m;
        x[32 + n] = l;
      }
    }
    __syncthreads();
    if (kw == 0) {
      float top = m;
#pragma unroll
      for (int k = 0; k < S::kKW - 1; ++k) top = fmaxf(top, jm[(k * RW + rw) * 64 + n]);
      const float base = top == -INFINITY ? 0.0f : top;
      const float a = __builtin_amdgcn_exp2f((m - base) * P.sl);
      l *= a;
#pragma unroll
      for (int db = 0; db < DP / 32; ++db)
#pragma unroll
        for (int r = 0; r < 16; ++r) W.o[db][r] *= a;
      for (int k = 0; k < S::kKW - 1; ++k) {
        const float *x = jm + (k * RW + rw) * 64;
        const float *o = jo + (k * RW + rw) * 32 * DP;
        const float f = __builtin_amdgcn_exp2f((x[n] - base) * P.sl);
        l = fmaf(x[32 + n], f, l);
#pragma unroll
        for (int db = 0; db < DP / 32; ++db)
#pragma unroll
          for (int r = 0; r < 16; ++r)
            W.o[db][r] = fmaf(o[(32 * db + 8 * (r / 4) + 4 * hf + r % 4) * 32 + n], f, W.o[db][r]);
      }
      m = top;
    }
  }
  if (kw == 0 && mine) {
    const int D = P.c.D;
    if (slot >= 0) {
      float *o = P.part_o + (slot * (32 * RW) + rw * 32 + n) * D;
#pragma unroll
      for (int db = 0; db < DP / 32; ++db)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          const float x[4] = {W.o[db][4 * g], W.o[db][4 * g + 1], W.o[db][4 * g + 2], W.o[db][4 * g + 3]};
          put4<float>(reinterpret_cast<char *>(o), 32 * db + 8 * g + 4 * hf, D, x);
        }
      if (hf == 0) {
        float *x = P.part_ml + (slot * (32 * RW) + rw * 32 + n) * 2;
        x[0] = m;
        x[1] = l;
      }
    } else {
      // a row that saw nothing has sum 0 (its maximum is -inf): zeros
      const bool none = W.sees == 0 || l == 0.0f;
      const float f = none ? 0.0f : 1.0f / l;
      const long long at = (J.token0 + token) * P.c.H * P.G + head;
      char *o = P.out + at * D * S::kElt;
#pragma unroll
      for (int db = 0; db < DP / 32; ++db)
#pragma unroll
        for (int g = 0; g < 4; ++g) {
          float x[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) x[j] = none ? 0.0f : W.o[db][4 * g + j] * f;
          put4<T>(o, 32 * db + 8 * g + 4 * hf, D, x);
        }
      if (P.lse && hf == 0) P.lse[at] = none ? -INFINITY : m * P.scale + logf(l);
    }
  }
  return PAGED && __syncthreads_or(ld.bad) ? SPEC_ST_BAD_STATE : 0;
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
  if (!(scale > 0.0f) || scale > 3.4e38f) return SPEC_EINVAL;
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
  P.splits = P.row_tiles = 1;
  P.part_o = P.part_ml = nullptr;
  P.part_bad = nullptr;
  return SPEC_OK;
}

}  // namespace attn
}  // namespace specv
