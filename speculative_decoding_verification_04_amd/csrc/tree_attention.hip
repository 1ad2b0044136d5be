// Attention of drafted chains and trees over the cache (gfx950).
//
// The verify forward's N nodes of each sequence attend its n_b cached rows and,
// among the nodes' own rows n_b .. n_b + N - 1, those that the mask gives (a
// chain without a mask: node i sees nodes 0 .. i).  N = 1 is single-token
// decoding.
//
// Design.  Bound by HBM: each cache row is read once for the N * G query rows
// of its KV head, which fit one workgroup's tile (32, 64 or 128 rows) unless
// the tree and the group are large.  With one workgroup per (sequence, KV
// head, row tile) a batch does not fill the chip, so each such group's cache
// rows are cut into pieces of at most a common length, which the workgroups find
// on the device from the sequences' lengths (a group's own pieces differ by a
// tile at most; groups of other lengths have others: trees over 25k and 33k rows
// get pieces of 98 or 99 and of 129 tiles); the pieces' partial results
// go to the workspace and a second launch joins them, in the order of the
// pieces, one wave for each query row.  (Joining them in the first launch, by
// the workgroup that brings a group's last piece, took 19 us instead of 16 for
// one token over 1100 rows, and 40 instead of 23 for five tokens of eight
// sequences: one workgroup's loads of all pieces, past its L2, are slower than
// a launch.)
// Measured, both launches, bf16 heads of 128: 16-node trees over 32 sequences of
// 512 .. 4096 rows, 32 heads over 8: 71 us = 4.4 TB/s of cache rows; 255-node trees
// over 25k and 33k rows: 287 us = 840 TFLOP/s (there the matrix units bound, as in
// prompts); five tokens of 8 sequences of 64 .. 2048 rows in pages, 28 heads over
// 4: 18 us; one token over 1100 rows: 12 us, the latency of two launches.
#include "attention.h"

namespace specv {
namespace {
using namespace attn;

inline int dp_of(int D) { return D <= 64 ? 64 : D <= 128 ? 128 : 256; }

// Workgroups that join `rows` query rows: a wave each.
inline long long join_grid(long long rows) { return (rows + kThreads / kWave - 1) / (kThreads / kWave); }

// How a call is cut: waves side by side, row tiles, pieces aimed at.
struct Plan {
  int rw, kt, row_tiles, target;
  long long groups, tiles, slots;   // tiles, slots (pieces): the most that the cache can give
};

inline Plan plan_of(int B, int N, int H, int G, int D, long long max_rows, spec_dtype dt) {
  Plan p;
  const long long R = static_cast<long long>(N) * G;
  // two buffers of 128 / rw cache rows (K and V, padded to dp) have to fit LDS
  const int row = dp_of(D) * (dt == SPEC_BF16 ? 2 : 4), least = row <= 256 ? 1 : row <= 512 ? 2 : 4;
  p.rw = R > 64 || least == 4 ? 4 : R > 32 || least == 2 ? 2 : 1;
  p.kt = p.rw == 4 ? (dt == SPEC_BF16 ? 64 : 32) : 128 / p.rw;
  p.row_tiles = static_cast<int>((R + 32 * p.rw - 1) / (32 * p.rw));
  p.groups = static_cast<long long>(B) * H * p.row_tiles;
  p.tiles = p.groups * ((max_rows + p.kt - 1) / p.kt);
  // A piece for each workgroup that the chip holds at once, one a CU, or two where
  // a row takes up to 256 bytes and a workgroup more than 32 query rows.  (512 for
  // all: 66-node float32 trees, 28 heads of 128, took 46 us instead of 37.)  The
  // kernels of bf16 heads up to 64 would fit once more on a CU than this counts.
  p.target = p.rw > 1 && row <= 256 ? 512 : 256;
  p.slots = p.groups + (p.tiles < p.target ? p.tiles : p.target);
  if (p.slots > p.tiles) p.slots = p.tiles;
  return p;
}

// Both launches fit, and the kernel's sums of tiles (with a target added) stay below 2^31.
inline bool plan_fits(const Plan &p, long long rows) {
  return p.tiles <= INT32_MAX - p.target && launchable(p.slots, kThreads) && launchable(join_grid(rows), kThreads);
}

// Workspace: a slot for each piece, and each group's pieces.
struct Space {
  size_t o, ml, bad, pieces, end;   // offsets
};
inline Space space_of(const Plan &p, int D) {
  const size_t slots = static_cast<size_t>(p.slots), rows = slots * 32 * p.rw;
  Space s;
  s.o = 0;
  s.ml = s.o + rows * D * 4;
  s.bad = s.ml + rows * 8;
  s.pieces = round_up(s.bad + slots * 4, 8);              // pairs of 32 bits, read and written as one
  s.end = round_up(s.pieces + static_cast<size_t>(p.groups) * 8, 256);
  return s;
}

// A sequence's status, for its length n and the rectangle's end E (pages: 0); 0:
// its rows may be read.
__device__ inline int tree_status(const Params &P, int n, int E) {
  int st = n < 0 ? SPEC_ST_BAD_STATE : 0;
  const long long cap = cache_capacity(P.c);
  if (P.c.table) {
    if (static_cast<long long>(n) + P.N > cap) st |= SPEC_ST_CAPACITY;
  } else {
    if (E < 0 || static_cast<long long>(E) + P.N > cap) st |= SPEC_ST_CAPACITY;
    if (n > E) st |= SPEC_ST_BAD_STATE;
  }
  return st;
}

// Tiles of a sequence's rows (0: not to be read).
__device__ inline int tree_tiles(const Params &P, int n, int E, int kt) {
  return tree_status(P, n, E) ? 0 : static_cast<int>((static_cast<long long>(n) + P.N + kt - 1) / kt);
}

template <typename T, int DP, int RW, bool PAGED, bool ONCE>
__global__ __launch_bounds__(kThreads, DP <= 128 && sizeof(T) == 2 && RW > 1 ? 2 : 1) void tree_kernel(Params P) {
  using S = Shape<T, DP, RW>;
  __shared__ __attribute__((aligned(16))) char buf0[S::kLds];
  __shared__ __attribute__((aligned(16))) char buf1[S::kLds];
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), rw = wave % RW;
  const int H = P.c.H, each = H * P.row_tiles, E = PAGED ? 0 : *P.c.end_col;
  // all tiles of the call; the first 64 sequences' stay in the lanes
  const int n0 = lane < P.B ? P.c.kv_len[lane] : -1;
  const int tiles0 = tree_tiles(P, n0, E, S::kKT);
  int total = tiles0;                                     // the host has seen that it fits
  for (int b = lane + kWave; b < P.B; b += kWave) total += tree_tiles(P, P.c.kv_len[b], E, S::kKT);
  total = wave_reduce(total, [](int a, int c) { return a + c; }) * each;
  // Tiles of a piece, at most: so many that the pieces fit the chip at once.  A
  // few workgroups more than that would run alone behind all the others: 16-node
  // trees over 32 sequences of 512 .. 4096 rows took 74 us so and 84 us without
  // the second look, 255-node trees over 32k rows 324 and 410 us.  It is not taken
  // for more than 64 sequences, nor where the groups alone exceed the target.
  int per = max(1, (total + P.target - 1) / P.target);
  if (P.B <= kWave && each * P.B <= P.target)
    while (per > 1 && wave_reduce((tiles0 + per - 1) / per, [](int a, int c) { return a + c; }) * each > P.target)
      per += (per + 15) / 16;
  // this workgroup's sequence: the pieces are numbered in the order of sequence, head, row tile
  Job J;
  J.b = -1;
  int tiles = 0, pieces = 0, first = 0, n = 0;            // of the sequence; its first piece's number
  for (int b0 = 0; b0 < P.B; b0 += kWave) {
    const int b = b0 + lane;
    const int nb = b0 == 0 ? n0 : b < P.B ? P.c.kv_len[b] : -1;
    const int tb = b0 == 0 ? tiles0 : tree_tiles(P, nb, E, S::kKT), pb = (tb + per - 1) / per;
    const int upto = wave_incl_scan(pb * each);
    const uint64_t who = __ballot(first + upto > static_cast<int>(blockIdx.x));
    if (who) {
      const int l = __ffsll(static_cast<unsigned long long>(who)) - 1;
      J.b = b0 + l;
      n = read_lane(nb, l);
      tiles = read_lane(tb, l);
      pieces = read_lane(pb, l);
      first += read_lane(upto, l) - pieces * each;
      break;
    }
    first += read_lane(upto, kWave - 1);
  }
  J.tokens = P.N;
  if (J.b >= 0) {
    const int off = blockIdx.x - first, g = off / pieces, i = off - g * pieces;   // g = h * row_tiles + rt
    J.h = g / P.row_tiles;
    J.row0 = (g - J.h * P.row_tiles) * 32 * RW;
    J.token0 = static_cast<long long>(J.b) * P.N;
    J.limit0 = n + 1;
    J.total = n + P.N;
    J.start_col = PAGED ? 0 : E - n;
    const int size = tiles / pieces, more = tiles - size * pieces;   // the first `more` pieces are one tile longer
    J.t0 = i * size + min(i, more);
    J.t1 = J.t0 + size + (i < more ? 1 : 0);
    Done<DP, S::kKW> D;
    const bool bad = walk<T, DP, RW, PAGED, false, ONCE>(P, J, D, buf0, buf1);
    if (pieces == 1) {
      put_rows<T>(P, J, D, sees_any(P, J.b, D.token));
      if (P.status && J.h == 0 && J.row0 == 0 && threadIdx.x == 0) P.status[J.b] = bad ? SPEC_ST_BAD_STATE : 0;
    } else {
      if (D.mine) {
        const long long row = static_cast<long long>(blockIdx.x) * (32 * RW) + rw * 32 + (lane & 31);
        char *o = reinterpret_cast<char *>(P.part_o + row * P.c.D);
#pragma unroll
        for (int q = 0; q < DP / 8 / S::kKW; ++q) {
          const float x[4] = {D.o[q][0], D.o[q][1], D.o[q][2], D.o[q][3]};
          put4<float>(o, 8 * (D.kw * (DP / 8 / S::kKW) + q) + 4 * (lane >> 5), P.c.D, x);
        }
        if (lane < 32 && D.kw == 0) P.part_ml[row] = make_float2(D.m, D.l);
      }
      if (threadIdx.x == 0) P.part_bad[blockIdx.x] = bad;
    }
    if (i == 0 && threadIdx.x == 0)
      reinterpret_cast<int2 *>(P.pieces)[static_cast<long long>(J.b) * each + g] = make_int2(blockIdx.x, pieces);
  }
  // sequences that are not read: zeros
  for (int b = blockIdx.x; b < P.B; b += gridDim.x) {
    const int st = tree_status(P, P.c.kv_len[b], E);
    if (!st) continue;
    J.token0 = static_cast<long long>(b) * P.N;
    J.row0 = 0;
    for (J.h = 0; J.h < H; ++J.h) put_zeros<T>(P, J, P.N * P.G);
    if (P.status && threadIdx.x == 0) P.status[b] = st;
    for (int x = threadIdx.x; x < each; x += kThreads)
      reinterpret_cast<int2 *>(P.pieces)[static_cast<long long>(b) * each + x] = make_int2(0, 0);
  }
}

// Joins the pieces of the groups that were cut, one wave for each query row,
// in the order of the pieces.  DP / 4 lanes read a piece's row, 16 bytes each,
// so a wave reads 256 / DP pieces at once.
template <typename T, int DP>
__global__ __launch_bounds__(kThreads) void join_kernel(Params P, int tile_rows) {
  constexpr int kLanes = DP / 4, kSide = kWave / kLanes, kAhead = 4;
  const int lane = threadIdx.x & (kWave - 1), side = lane / kLanes, d0 = lane % kLanes * 4;
  const int R = P.N * P.G, D = P.c.D;
  const int x = blockIdx.x * (kThreads / kWave) + threadIdx.x / kWave;   // (b * H + h) * R + row
  if (x >= P.B * P.c.H * R) return;
  const int row = x % R, bh = x / R, b = bh / P.c.H, h = bh - b * P.c.H;
  const int rt = row / tile_rows, at_row = row - rt * tile_rows;
  const int2 cut = reinterpret_cast<const int2 *>(P.pieces)[static_cast<long long>(bh) * P.row_tiles + rt];
  const int pieces = cut.y;
  if (pieces <= 1) return;
  auto slot = [&](int i) { return static_cast<long long>(cut.x) + i; };
  const int token = row / P.G;
  uint32_t word = 1;
  if (P.mask) word = lane < P.words ? P.mask[(static_cast<long long>(b) * P.N + token) * P.words + lane] : 0u;
  // up to eight pieces' rows (DP = 128), asked for before their weights are known
  f32x4 v[kAhead];
  auto fetch = [&](int s, int end) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < kAhead; ++u) {
      if (s + u * kSide >= end) break;
      const int i = min(s + u * kSide + side, end - 1);
      v[u] = d0 < D ? *reinterpret_cast<const f32x4 *>(P.part_o + (slot(i) * tile_rows + at_row) * D + d0)
                    : f32x4{0.0f, 0.0f, 0.0f, 0.0f};
    }
  };
  float top = -INFINITY, sum = 0.0f;
  f32x4 acc = {0.0f, 0.0f, 0.0f, 0.0f};
  bool bad = false;
  for (int s0 = 0; s0 < pieces; s0 += kWave) {
    const int count = min(kWave, pieces - s0);
    fetch(s0, s0 + count);
    float m = -INFINITY, l = 0.0f;
    if (lane < count) {
      const float2 x = P.part_ml[slot(s0 + lane) * tile_rows + at_row];
      m = x.x;
      l = x.y;
      if (P.status) bad |= P.part_bad[slot(s0 + lane)] != 0;
    }
    const float high = fmaxf(top, wave_max_dpp(m)), base = high == -INFINITY ? 0.0f : high;
    const float a = __builtin_amdgcn_exp2f((top - base) * P.sl), f = __builtin_amdgcn_exp2f((m - base) * P.sl);
    top = high;
    sum = fmaf(sum, a, wave_reduce(l * f, [](float p, float q) { return p + q; }));
    acc *= a;
    for (int s = 0; s < count; s += kSide * kAhead) {
      if (s > 0) fetch(s0 + s, s0 + count);
#pragma unroll
      for (int u = 0; u < kAhead; ++u) {
        if (s + u * kSide >= count) break;
        const int i = s + u * kSide + side;
        const float w = __shfl(f, min(i, count - 1));     // every lane takes part
        if (i < count) acc += v[u] * w;
      }
    }
  }
#pragma unroll
  for (int d = kLanes; d < kWave; d <<= 1)
#pragma unroll
    for (int j = 0; j < 4; ++j) acc[j] += __shfl_xor(acc[j], d);
  const bool none = !__any(word != 0) || sum == 0.0f;
  const float f = none ? 0.0f : 1.0f / sum;
  const long long at = (static_cast<long long>(b) * P.N + token) * P.c.H * P.G + h * P.G + (row - token * P.G);
  if (side == 0) {
    const float o[4] = {none ? 0.0f : acc[0] * f, none ? 0.0f : acc[1] * f, none ? 0.0f : acc[2] * f,
                        none ? 0.0f : acc[3] * f};
    put4<T>(P.out + at * D * sizeof(T), d0, D, o);
  }
  if (P.lse && lane == 0) P.lse[at] = none ? -INFINITY : top * P.scale + logf(sum);
  if (P.status && h == 0 && row == 0) {
    const bool any = __any(bad);
    if (lane == 0) P.status[b] = any ? SPEC_ST_BAD_STATE : 0;
  }
}

template <typename T, int DP, int RW, bool ONCE>
void launch_once(const Params &P, unsigned grid, hipStream_t s) {
  if (P.c.table)
    hipLaunchKernelGGL((tree_kernel<T, DP, RW, true, ONCE>), dim3(grid), dim3(kThreads), 0, s, P);
  else
    hipLaunchKernelGGL((tree_kernel<T, DP, RW, false, ONCE>), dim3(grid), dim3(kThreads), 0, s, P);
}

// Rows that one workgroup reads, of a layer too large to be found in the
// Infinity Cache (256 MB) again, are read non-temporally: 75 us instead of 83
// for 16-node trees over 32 sequences of 512 .. 4096 rows (300 MB) that rotate
// over four caches.  Smaller layers lose by it (18 MB: 20.0 -> 21.3 us), and so do
// rows that several row tiles share (294 -> 320 us).
template <typename T, int DP, int RW>
void launch_rows(const Params &P, unsigned grid, hipStream_t s) {
  if constexpr (sizeof(T) == 2) {
    const long long planes = P.c.table ? P.c.planes : P.B;
    if (P.row_tiles == 1 && planes * P.c.H * P.c.cols * P.c.D * 4 > (256ll << 20))
      return launch_once<T, DP, RW, true>(P, grid, s);
  }
  launch_once<T, DP, RW, false>(P, grid, s);
}

template <typename T, int DP>
void launch_tree(const Params &P, const Plan &p, hipStream_t s) {
  const unsigned grid = static_cast<unsigned>(p.slots);
  if (p.rw == 4) return launch_rows<T, DP, 4>(P, grid, s);
  if constexpr (sizeof(T) * DP <= 512) {
    if (p.rw == 2) return launch_rows<T, DP, 2>(P, grid, s);
  }
  if constexpr (sizeof(T) * DP <= 256) launch_rows<T, DP, 1>(P, grid, s);
}

template <typename T, int DP>
int launch_both(const Params &P, const Plan &p, hipStream_t s) {
  (void)hipGetLastError();
  launch_tree<T, DP>(P, p, s);
  const int st = launch_status();
  if (st != SPEC_OK) return st;
  const unsigned joins = static_cast<unsigned>(join_grid(static_cast<long long>(P.B) * P.c.H * P.N * P.G));
  hipLaunchKernelGGL((join_kernel<T, DP>), dim3(joins), dim3(kThreads), 0, s, P, 32 * p.rw);
  return launch_status();
}

template <typename T>
int launch_all(const Params &P, const Plan &p, hipStream_t s) {
  if (P.c.D <= 64) return launch_both<T, 64>(P, p, s);
  return P.c.D <= 128 ? launch_both<T, 128>(P, p, s) : launch_both<T, 256>(P, p, s);
}

int tree_call(const void *q, int64_t q_stride, const void *kv, spec_dtype dt, int L, int planes, int B, int H,
              int cols, int D, int layer, int N, int G, const int32_t *table, int max_pages, bool paged,
              const int32_t *end_col, const int32_t *kv_len, const uint32_t *mask, float scale, void *out, float *lse,
              int32_t *status, void *ws, size_t ws_bytes, spec_stream_t stream) {
  Params P;
  const int err = fill(P, q, q_stride, kv, dt, L, planes, B, H, cols, D, layer, G, table, max_pages, paged, end_col,
                       kv_len, scale, out, lse, status);
  if (err) return err;
  if (N < 1) return SPEC_EINVAL;
  if (N > SPEC_TREE_MAX_N) return SPEC_ECAPACITY;
  if (!aligned(mask, 4)) return SPEC_EINVAL;
  const long long tokens = static_cast<long long>(B) * N, rows = tokens * H * G;
  if (rows >= INT32_MAX) return SPEC_EINVAL;
  const Plan p = plan_of(B, N, H, G, D, cache_capacity(P.c), dt);
  if (!plan_fits(p, rows)) return SPEC_EINVAL;
  const size_t elt = dt == SPEC_BF16 ? 2 : 4, hd = static_cast<size_t>(H) * G * D, b4 = static_cast<size_t>(B) * 4;
  const int words = (N + 31) / 32;
  const Space sp = space_of(p, D);
  const size_t need = sp.end;
  const void *ins[] = {q, kv, table, end_col, kv_len, mask};
  const size_t in_n[] = {((tokens - 1) * static_cast<size_t>(q_stride) + hd) * elt,
                         cache_bytes(dt, L, planes, H, cols, D), paged ? b4 * max_pages : 0, paged ? 0u : 4u, b4,
                         static_cast<size_t>(tokens) * words * 4};
  const void *outs[] = {out, lse, status, ws};
  const size_t out_n[] = {tokens * hd * elt, static_cast<size_t>(tokens) * H * G * 4, b4, need};
  for (int o = 0; o < 4; ++o) {
    for (int j = 0; j < 6; ++j)
      if (overlaps(outs[o], out_n[o], ins[j], in_n[j])) return SPEC_EINVAL;
    for (int j = o + 1; j < 4; ++j)
      if (overlaps(outs[o], out_n[o], outs[j], out_n[j])) return SPEC_EINVAL;
  }
  if (!ws || ws_bytes < need || !aligned(ws, 256)) return SPEC_EWORKSPACE;
  P.N = N;
  P.words = words;
  P.mask = mask;
  P.target = p.target;
  P.row_tiles = p.row_tiles;
  char *w = static_cast<char *>(ws);
  P.part_o = reinterpret_cast<float *>(w + sp.o);
  P.part_ml = reinterpret_cast<float2 *>(w + sp.ml);
  P.part_bad = reinterpret_cast<int32_t *>(w + sp.bad);
  P.pieces = reinterpret_cast<int32_t *>(w + sp.pieces);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return dt == SPEC_BF16 ? launch_all<__bf16>(P, p, s) : launch_all<float>(P, p, s);
}

}  // namespace
}  // namespace specv

using namespace specv;

extern "C" size_t spec_tree_attention_workspace_bytes(int B, int N, int H, int G, int D, int max_rows,
                                                      spec_dtype dt) {
  if (B < 1 || N < 1 || N > SPEC_TREE_MAX_N || H < 1 || G < 1 || D < 1 || D > SPEC_ATTN_MAX_D || max_rows < 1) return 0;
  if (dt != SPEC_F32 && dt != SPEC_BF16) return 0;
  if (static_cast<long long>(H) * G >= INT32_MAX / SPEC_ATTN_MAX_D) return 0;
  const long long rows = static_cast<long long>(B) * N * H * G;
  if (rows >= INT32_MAX) return 0;
  const Plan p = plan_of(B, N, H, G, D, max_rows, dt);
  return plan_fits(p, rows) ? space_of(p, D).end : 0;
}

extern "C" int spec_tree_attention(const void *q, int64_t q_stride, const void *kv, spec_dtype dt, int L, int B, int H,
                                   int C, int D, int layer, int N, int G, const int32_t *end_col,
                                   const int32_t *kv_len, const uint32_t *mask, float scale, void *out, float *lse,
                                   int32_t *status, void *ws, size_t ws_bytes, spec_stream_t stream) {
  return tree_call(q, q_stride, kv, dt, L, B, B, H, C, D, layer, N, G, nullptr, 0, false, end_col, kv_len, mask, scale,
                   out, lse, status, ws, ws_bytes, stream);
}

extern "C" int spec_tree_attention_paged(const void *q, int64_t q_stride, const void *pool, spec_dtype dt, int L,
                                         int pages, int H, int page_size, int D, int layer, int B, int N, int G,
                                         const int32_t *block_table, int max_pages, const int32_t *kv_len,
                                         const uint32_t *mask, float scale, void *out, float *lse, int32_t *status,
                                         void *ws, size_t ws_bytes, spec_stream_t stream) {
  return tree_call(q, q_stride, pool, dt, L, pages, B, H, page_size, D, layer, N, G, block_table, max_pages, true,
                   nullptr, kv_len, mask, scale, out, lse, status, ws, ws_bytes, stream);
}
