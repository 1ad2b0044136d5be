// Attention of few query rows over a cache of 4-bit numbers (gfx950): the walk of one
// job by waves that each read, convert and multiply cache rows of their own.
//
// Where a KV head's query rows fit 32 or 64, a cache row is used by one or two waves
// only, and sharing converted tiles through LDS between barriers costs more than it
// saves.  Here RW waves side by side take 32 query rows each, or each wave QB times 32,
// and the waves behind each other take blocks of 32 cache rows in turn, without a barrier
// until they are joined:
//   - a lane asks for 16-byte shares of one cache row's K and V codes a block or two ahead;
//   - K's codes become the first product's operand in registers: the order of the
//     elements in a dot product is free, so each lane keeps the blocks that it read and
//     the queries are laid out to match (in registers, or for QB = 2 in LDS);
//   - V's codes become bf16 in the wave's own LDS, from where the transposing read gives
//     the second product's operand.
// The products are as in attention.h: S^T = K Q^T and O^T = V^T P^T.
//
// float32: codes times scales are exact in bf16, so a product with float32 is the sum
// of products with its three parts of 8 bits, each exact: three products of the bf16
// rate (2.5 PFLOP/s) where one of float32 takes sixteen.
//
// Bound by issue: of a block's 1.1 us a wave at two waves a SIMD (64 rows of bf16, heads of
// 128) the matrix instructions take half, the conversions and exponentials the most of the
// other half, and the two overlap in part.  A workgroup's start, its first loads and its
// join cost 8 or 9 us more.  Not all that a wave holds fits its registers: 19 .. 22 go to
// scratch in the loop for two blocks of 32 rows of heads of 128, 40 for float32 heads of 128
// and 59 of 256.  Measured, both types at the clock under load: 16-node trees over
// 32 sequences of 512 .. 4096 rows, 32 heads over 8, 44 us (the longest sequences' walks;
// all of 4096 rows 53); 4-node trees over 32 sequences of 4096 rows 33 us = 4.4 TB/s of
// codes and scales; chains of 5 in float32, 8 sequences of 64 .. 2048 rows in pages, 28
// heads over 4, 17 us and the join 4; one token over 1100 rows 11 us.
// Not kept: products of the codes themselves (the scaled instructions add their products
// up to 2^-12 of the sum's size apart); the next block's conversions beside this one's
// products (56 us where this took 51: registers); a wave's loads in the order of the rows'
// bytes (no change); float32 queries cut once and passed on through LDS (21 us and 20).
#pragma once

#include "attention.h"

namespace specv {
namespace attn {

template <typename T, int D, int RW, int QB>
struct Few {
  static constexpr int kWaves = D <= 128 ? 8 : 4;         // two a SIMD, or one where registers are short
  static constexpr int kThreads = kWaves * kWave;
  static constexpr int kKW = kWaves / RW;                 // waves behind each other
  static constexpr int kParts = sizeof(T) == 2 ? 1 : 3;   // bf16 parts of a number
  static constexpr int kShares = D / 64;                  // 16-byte shares of a row that a lane takes
  // blocks in registers before they are used: two where the registers hold them.  Float32
  // heads of 128, whose queries take three parts on two waves a SIMD, and of 256 have no
  // room for a second: with it, chains of 5 (28 heads of 128 over 4) take 18.5 us and not
  // 16.2, 4-node trees over 32 sequences of 512 .. 4096 rows (heads of 256) 207 and not 161.
  // (With one, 40 registers of the first and 59 of the second still go to scratch.)
  static constexpr int kAhead = QB == 1 && (sizeof(T) == 2 || D == 64 || D == 192) ? 2 : 1;
  static constexpr int kRow = (D <= 64 ? 64 : D <= 128 ? 128 : 256) * 2;   // bytes of a row of V in LDS
  static constexpr int kStage = 32 * kRow;                // V of one wave
  static constexpr int kJoin = 32 * D * 4;                // outputs of 32 rows of one wave
  static constexpr int kEach = kStage > kJoin ? kStage : kJoin;
  static constexpr int kQueries = QB == 1 ? 0 : QB * 4 * kShares * kWave * 16;   // operands of all waves
  static constexpr int kLds = kWaves * kEach + kQueries;
  static_assert(RW == 1 || QB == 1, "one or the other");
};

// A lane's part of a block of 32 cache rows: row lane % 32, blocks 2 i + lane / 32.
template <int SHARES>
struct FewRaw {
  u32x4 k[SHARES], v[SHARES];
  uint32_t ks[(SHARES + 1) / 2], vs[(SHARES + 1) / 2];    // the row's scales, four to a word
};

// The scale byte of share i.
template <int SHARES>
__device__ inline int few_scale(const uint32_t (&s)[(SHARES + 1) / 2], int i, int hf) {
  return static_cast<int>(s[i / 2] >> (16 * (i % 2) + 8 * hf)) & 255;
}

// 8 values of bf16 from 8 codes.
__device__ inline bf16x8 few_widen(uint32_t codes, float scale) {
  __bf16 x[8];
  mx_widen<__bf16>(codes, scale, x);
  return bf16x8{x[0], x[1], x[2], x[3], x[4], x[5], x[6], x[7]};
}

// The next 8 bits of eight float32 numbers as bf16, cut off, and what is left of them.
__device__ inline bf16x8 cut_part(float (&x)[8]) {
  u32x4 y;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const uint32_t a = __float_as_uint(x[2 * j]), b = __float_as_uint(x[2 * j + 1]);
    y[j] = __builtin_amdgcn_perm(b, a, 0x07060302u);
    x[2 * j] -= __uint_as_float(a & 0xffff0000u);
    x[2 * j + 1] -= __uint_as_float(b & 0xffff0000u);
  }
  return __builtin_bit_cast(bf16x8, y);
}

// The walk of one job; calls store(Done, rw, sees) for each 32 query rows.  J.t0, J.t1 count
// blocks of 32 rows.  lds: kLds bytes.  Returns whether a bad page was met.
template <typename T, int D, int RW, int QB, bool PAGED, class Store>
__device__ inline bool few_walk(const Params &P, const Job &J, Store store, char *lds) {
  using F = Few<T, D, RW, QB>;
  constexpr int S = F::kShares, kRow = F::kRow, kChunks = kRow / 16;
  const int lane = threadIdx.x & (kWave - 1), n = lane & 31, hf = lane >> 5;
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), rw = wave % RW, kw = wave / RW;
  char *const stage = lds + wave * F::kEach;
  bf16x8 *const queries = reinterpret_cast<bf16x8 *>(lds + F::kWaves * F::kEach) + lane;   // [QB][4 S][64 lanes]
  bool bad = false;

  // The page of a block's row is asked for a block before its codes are.
  auto page_at = [&](int t) __attribute__((always_inline)) {
    if constexpr (PAGED) {
      const int r = min(t * 32 + n, J.total - 1);
      return P.c.table[static_cast<long long>(J.b) * P.c.max_pages + cache_page(P.c, r)];
    } else {
      return 0;
    }
  };
  auto fetch = [&](FewRaw<S> &x, int t, int page) __attribute__((always_inline)) {
    const int r = min(t * 32 + n, J.total - 1);
    int plane = J.b, col = J.start_col + r;
    if constexpr (PAGED) {
      const bool ok = page >= 0 && page < P.c.planes;
      bad |= !ok;
      plane = ok ? page : 0;
      col = r - cache_page(P.c, r) * P.c.cols;
    }
    const long long row = (static_cast<long long>(plane) * P.c.H + J.h) * P.c.cols + col;
    const char *k = P.c.k + row * (D / 2) + hf * 16, *v = P.c.v + row * (D / 2) + hf * 16;
#pragma unroll
    for (int i = 0; i < S; ++i) {
      x.k[i] = *reinterpret_cast<const u32x4 *>(k + 32 * i);
      x.v[i] = *reinterpret_cast<const u32x4 *>(v + 32 * i);
    }
    const char *ks = P.c.ks + row * (D / kMxBlock), *vs = P.c.vs + row * (D / kMxBlock);
#pragma unroll
    for (int i = 0; i < (S + 1) / 2; ++i) {
      if constexpr (S % 2 == 0) {
        x.ks[i] = reinterpret_cast<const uint32_t *>(ks)[i];
        x.vs[i] = reinterpret_cast<const uint32_t *>(vs)[i];
      } else {                                            // rows of 2 or 6 bytes
        x.ks[i] = reinterpret_cast<const uint16_t *>(ks)[2 * i];
        x.vs[i] = reinterpret_cast<const uint16_t *>(vs)[2 * i];
        if (2 * i + 1 < S) {
          x.ks[i] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(ks)[2 * i + 1]) << 16;
          x.vs[i] |= static_cast<uint32_t>(reinterpret_cast<const uint16_t *>(vs)[2 * i + 1]) << 16;
        }
      }
    }
  };

  FewRaw<S> raw[F::kAhead];
  const int first = J.t0 + kw, last = J.t1 - 1;           // blocks first, first + kKW, ..; past the last: read again
  auto nth = [&](int i) { return min(first + i * F::kKW, last); };
  int pages[F::kAhead];
#pragma unroll
  for (int i = 0; i < F::kAhead; ++i) pages[i] = page_at(nth(i));
  int page = page_at(nth(F::kAhead));                     // of the block to be fetched next
#pragma unroll
  for (int i = 0; i < F::kAhead; ++i) fetch(raw[i], nth(i), pages[i]);

  const int rows = J.tokens * P.G;
  int token[QB], head[QB];
  bf16x8 q[QB == 1 ? F::kParts : 1][4 * S];
#pragma unroll
  for (int b = 0; b < QB; ++b) {
    const int row = min(J.row0 + (QB == 1 ? rw : b) * 32 + n, rows - 1);      // rows past the end repeat the last
    token[b] = row / P.G;
    head[b] = J.h * P.G + (row - token[b] * P.G);
    const T *from = reinterpret_cast<const T *>(P.q + (J.token0 + token[b]) * P.q_stride) + static_cast<long long>(head[b]) * D;
    auto at = [&](int i) { return from + 32 * (2 * (i / 4) + hf) + 8 * (i % 4); };
    if constexpr (QB > 1) {
      for (int i = wave; i < 4 * S; i += F::kWaves)       // each wave brings its share
        queries[(b * 4 * S + i) * kWave] = *reinterpret_cast<const bf16x8 *>(at(i));
    } else {
#pragma unroll
      for (int i = 0; i < 4 * S; ++i) {
        if constexpr (sizeof(T) == 2) {
          q[0][i] = *reinterpret_cast<const bf16x8 *>(at(i));
        } else {
          const f32x4 a = reinterpret_cast<const f32x4 *>(at(i))[0], b4 = reinterpret_cast<const f32x4 *>(at(i))[1];
          float x[8] = {a[0], a[1], a[2], a[3], b4[0], b4[1], b4[2], b4[3]};
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = x[k] == x[k] ? x[k] : NAN;   // a NaN's first part may be an infinity's
          q[0][i] = cut_part(x);
#pragma unroll
          for (int k = 0; k < 8; ++k) x[k] = fabsf(x[k]) < INFINITY ? x[k] : 0.0f;   // infinity is its first part
#pragma unroll
          for (int p = 1; p < F::kParts; ++p) q[p][i] = cut_part(x);
        }
      }
    }
  }
  bool sees[QB];                                          // whether the rows' nodes see anything at all
#pragma unroll
  for (int b = 0; b < QB; ++b) sees[b] = sees_any(P, J.b, token[b]);
  if constexpr (QB > 1) __syncthreads();
  f32x16 o[QB][D / 32];
  float m[QB], l[QB], base[QB];
#pragma unroll
  for (int b = 0; b < QB; ++b) {
#pragma unroll
    for (int db = 0; db < D / 32; ++db)
#pragma unroll
      for (int r = 0; r < 16; ++r) o[b][db][r] = 0.0f;
    m[b] = -INFINITY;
    l[b] = base[b] = 0.0f;
  }
  const float sl = P.sl;
  // cache rows below `plain` are seen by every row of the workgroup
  const int plain = P.mask ? J.limit0 - 1 : J.limit0 + J.row0 / P.G;
  const int i16 = lane & 15, dg = (lane >> 4) & 1, r0 = 4 * hf + (i16 >> 2);
  const int write0 = n * kRow, turned = turn<kChunks>(n);
  const int va16 = r0 * kRow + (((2 * dg + ((i16 & 3) >> 1)) ^ turn<kChunks>(r0)) << 4) + (i16 & 1) * 8;

  auto block = [&](FewRaw<S> &x, int t) __attribute__((always_inline)) {
    // which of the lane's shares have scales that stand for NaN
    uint32_t odd_k = 0, odd_v = 0;
#pragma unroll
    for (int i = 0; i < S; ++i) {
      odd_k |= few_scale<S>(x.ks, i, hf) > kMxTop ? 1u << i : 0u;
      odd_v |= few_scale<S>(x.vs, i, hf) > kMxTop ? 1u << i : 0u;
    }
    const uint64_t who_k = __ballot(odd_k != 0), who_v = __ballot(odd_v != 0);
    f32x16 s[QB];
#pragma unroll
    for (int b = 0; b < QB; ++b)
#pragma unroll
      for (int r = 0; r < 16; ++r) s[b][r] = 0.0f;
    // V first: it is in LDS by the time the scores are there
#pragma unroll
    for (int i = 0; i < S; ++i) {
      const float scale = mx_scale(few_scale<S>(x.vs, i, hf));
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<bf16x8 *>(stage + write0 + (((4 * (2 * i + hf) + j) ^ turned) << 4)) = few_widen(x.v[i][j], scale);
    }
    if constexpr (QB == 1) {
#pragma unroll
      for (int i = 0; i < S; ++i) {
        const float scale = mx_scale(few_scale<S>(x.ks, i, hf));
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const bf16x8 a = few_widen(x.k[i][j], scale);
#pragma unroll
          for (int p = 0; p < F::kParts; ++p) s[0] = mfma(a, q[p][4 * i + j], s[0]);
        }
      }
    } else {
      // queries' operands are asked for two products ahead: left to itself the compiler
      // asks for each just before its use and waits out the LDS latency each time
      constexpr int kLead = 2, kSteps = 4 * S;
      bf16x8 ahead[kLead][QB];
      __builtin_amdgcn_sched_barrier(0);
#pragma unroll
      for (int i = 0; i < kLead; ++i)
#pragma unroll
        for (int b = 0; b < QB; ++b) ahead[i][b] = queries[(b * kSteps + i) * kWave];
      __builtin_amdgcn_sched_group_barrier(0x100, kLead * QB, 0);
#pragma unroll
      for (int i = 0; i < kSteps; ++i) {
        const float scale = mx_scale(few_scale<S>(x.ks, i / 4, hf));
        const bf16x8 a = few_widen(x.k[i / 4][i % 4], scale);
#pragma unroll
        for (int b = 0; b < QB; ++b) {
          s[b] = mfma(a, ahead[i % kLead][b], s[b]);
          if (i + kLead < kSteps) ahead[i % kLead][b] = queries[(b * kSteps + i + kLead) * kWave];
        }
        __builtin_amdgcn_sched_group_barrier(0x002, 4, 0);
        __builtin_amdgcn_sched_group_barrier(0x008, QB, 0);
        __builtin_amdgcn_sched_group_barrier(0x100, QB, 0);
      }
    }
    // its registers are free
    fetch(x, min(t + F::kAhead * F::kKW, last), page);
    page = page_at(min(t + (F::kAhead + 1) * F::kKW, last));

    if (who_k) {                                          // rare: such a row's scores are NaN
      const uint32_t k = static_cast<uint32_t>(who_k) | static_cast<uint32_t>(who_k >> 32);
#pragma unroll
      for (int b = 0; b < QB; ++b)
#pragma unroll
        for (int r = 0; r < 16; ++r) s[b][r] = k >> (8 * (r / 4) + 4 * hf + r % 4) & 1u ? NAN : s[b][r];
    }
    if (who_v) {                                          // rare: such shares are cleared, see below
      for (int c = 0; c < 4 * S; ++c)
        if (odd_v >> (c / 4) & 1u)
          *reinterpret_cast<u32x4 *>(stage + write0 + (((4 * (2 * (c / 4) + hf) + c % 4) ^ turned) << 4)) = u32x4{0, 0, 0, 0};
    }
    uint32_t vis[QB];
#pragma unroll
    for (int b = 0; b < QB; ++b) vis[b] = ~0u;
    if ((t + 1) * 32 > plain) {
#pragma unroll
      for (int b = 0; b < QB; ++b) {
        vis[b] = seen<false>(P, J, token[b], t * 32);
        const uint32_t see = vis[b] >> (4 * hf);
#pragma unroll
        for (int r = 0; r < 16; ++r) s[b][r] = (see >> (8 * (r / 4) + r % 4)) & 1u ? s[b][r] : -INFINITY;
      }
    }
    float mx[QB];
    bool grows = false;
#pragma unroll
    for (int b = 0; b < QB; ++b) {
      mx[b] = s[b][0];
#pragma unroll
      for (int r = 1; r < 16; ++r) mx[b] = fmaxf(mx[b], s[b][r]);
      mx[b] = half_max(mx[b]);
      grows |= fmaf(mx[b], sl, -base[b]) > kSlack || (m[b] == -INFINITY && mx[b] > -INFINITY);
    }
    // the reference follows the maximum by steps, as in attention.h
    if (__any(grows)) {
#pragma unroll
      for (int b = 0; b < QB; ++b) {
        const float high = fmaxf(m[b], mx[b]);
        const float to = high == -INFINITY ? 0.0f : high * sl;
        const float alpha = __builtin_amdgcn_exp2f(fmaf(m[b], sl, -to));
        m[b] = high;
        base[b] = to;
        l[b] *= alpha;
#pragma unroll
        for (int db = 0; db < D / 32; ++db)
#pragma unroll
          for (int r = 0; r < 16; ++r) o[b][db][r] *= alpha;
      }
    }
    // V's operands are asked for before the exponentials, and the second half's while the
    // first is multiplied
    bf16x8 v[2][D / 32];
    auto read_v = [&](int half, int db) __attribute__((always_inline)) {
      const bf16x4b lo = read_turned(stage + (va16 ^ (db << 6)) + 16 * half * kRow);
      const bf16x4b hi = read_turned(stage + (va16 ^ (db << 6 | 2 << 4)) + (16 * half + 8) * kRow);
      v[half][db] = bf16x8{lo[0], lo[1], lo[2], lo[3], hi[0], hi[1], hi[2], hi[3]};
    };
#pragma unroll
    for (int db = 0; db < D / 32; ++db) read_v(0, db);
    __builtin_amdgcn_sched_group_barrier(0x100, 2 * (D / 32), 1);
#pragma unroll
    for (int b = 0; b < QB; ++b) {
      float sum = 0.0f;
#pragma unroll
      for (int r = 0; r < 16; ++r) {
        s[b][r] = __builtin_amdgcn_exp2f(fmaf(s[b][r], sl, -base[b]));
        sum += s[b][r];
      }
      l[b] += sum;
    }
    __builtin_amdgcn_sched_group_barrier(0x402, 32 * QB, 1);
    // O^T += V^T P^T.  bf16: the weights are rounded, off by at most half a step, 2^-8 of a weight; their sum
    // is of the unrounded ones.  float32: in three parts.
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      bf16x8 p[QB][F::kParts];
#pragma unroll
      for (int b = 0; b < QB; ++b) {
        if constexpr (sizeof(T) == 2) {
#pragma unroll
          for (int j = 0; j < 8; ++j) p[b][0][j] = static_cast<__bf16>(s[b][8 * half + j]);
        } else {
          float y[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) y[j] = s[b][8 * half + j];
#pragma unroll
          for (int k = 0; k < F::kParts; ++k) p[b][k] = cut_part(y);
        }
      }
#pragma unroll
      for (int db = 0; db < D / 32; ++db) {
        if (half == 0) read_v(1, db);
#pragma unroll
        for (int b = 0; b < QB; ++b)
#pragma unroll
          for (int k = 0; k < F::kParts; ++k) o[b][db] = mfma(v[half][db], p[b][k], o[b][db]);
      }
    }
    if (who_v) {                                          // NaN for the query rows that see them
      for (uint64_t left = who_v; left; left &= left - 1) {
        const int from = __ffsll(static_cast<unsigned long long>(left)) - 1;
        const uint32_t bits = read_lane(odd_v, from);
#pragma unroll
        for (int b = 0; b < QB; ++b) {
          const bool see = vis[b] >> (from & 31) & 1u;
#pragma unroll
          for (int i = 0; i < S; ++i)
#pragma unroll
            for (int side = 0; side < 2; ++side) {
              const float nan = bits >> i & 1u && from >> 5 == side && see ? NAN : 0.0f;
#pragma unroll
              for (int r = 0; r < 16; ++r) o[b][2 * i + side][r] += nan;
            }
        }
      }
    }
  };
  for (int t = first; t <= last; t += F::kAhead * F::kKW) {
    block(raw[0], t);
    if constexpr (F::kAhead == 2) {
      if (t + F::kKW <= last) block(raw[1], t + F::kKW);
    }
  }

  // Join the waves behind each other, as walk() does, 32 rows of each at a time.
  __shared__ float2 jm[F::kWaves][32];
  __shared__ int flag;
#pragma unroll
  for (int b = 0; b < QB; ++b) {
    const float total = half_sum(l[b]);
    __syncthreads();                                      // the stages, or the outputs before, are read
    if (threadIdx.x == 0 && b == 0) flag = 0;
    f32x4 *mine = reinterpret_cast<f32x4 *>(lds + wave * F::kEach) + hf * 32 + n;
#pragma unroll
    for (int x = 0; x < D / 8; ++x) {                     // x = 4 db + g: d = 8 x + 4 hf ..
      const f32x16 &y = o[b][x / 4];
      mine[x * 64] = f32x4{y[4 * (x % 4)], y[4 * (x % 4) + 1], y[4 * (x % 4) + 2], y[4 * (x % 4) + 3]};
    }
    if (hf == 0) jm[wave][n] = make_float2(m[b], total);
    __syncthreads();
    if (PAGED && P.status && bad) flag = 1;
    constexpr int kMine = D / 8 / F::kKW;                 // quads of this wave
    float2 ml[F::kKW];
    float top = -INFINITY;
#pragma unroll
    for (int k = 0; k < F::kKW; ++k) {
      ml[k] = jm[k * RW + rw][n];
      top = fmaxf(top, ml[k].x);
    }
    const float to = top == -INFINITY ? 0.0f : top;
    Done<D, F::kKW> R;
    R.m = top;
    R.l = 0.0f;
#pragma unroll
    for (int i = 0; i < kMine; ++i) R.o[i] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
    for (int k = 0; k < F::kKW; ++k) {
      const float f = __builtin_amdgcn_exp2f((ml[k].x - to) * sl);
      R.l = fmaf(ml[k].y, f, R.l);
      const f32x4 *of = reinterpret_cast<const f32x4 *>(lds + (k * RW + rw) * F::kEach) + hf * 32 + n + kw * kMine * 64;
#pragma unroll
      for (int i = 0; i < kMine; ++i) R.o[i] += of[i * 64] * f;
    }
    const int side = QB == 1 ? rw : b;
    R.mine = J.row0 + side * 32 + n < rows;
    R.token = token[b];
    R.head = head[b];
    R.kw = kw;
    store(R, side, sees[b]);
  }
  if (!PAGED || !P.status) return false;
  __syncthreads();
  return flag != 0;
}

}  // namespace attn
}  // namespace specv
