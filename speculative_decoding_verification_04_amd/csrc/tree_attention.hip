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
// head) a batch does not fill the chip, so the cache rows are split over
// workgroups and a second launch joins their partial results in split order.
#include "attention.h"

namespace specv {
namespace {
using namespace attn;

// How a call is cut: waves side by side, row tiles, splits of the cache rows.
struct Plan {
  int rw, tile_rows, row_tiles, splits;
  long long slots;
};

inline Plan plan_of(int B, int N, int H, int G, int D, long long max_rows, spec_dtype dt) {
  Plan p;
  const long long R = static_cast<long long>(N) * G;
  // two buffers of a tile fit LDS: 32 * 4 / rw cache rows of K and V (64 for bf16 and rw = 4)
  const int least = (dt == SPEC_F32 ? 2 : 1) * (D > 128 ? 2 : 1);
  p.rw = R > 64 || least == 4 ? 4 : R > 32 || least == 2 ? 2 : 1;
  p.tile_rows = 32 * p.rw;
  p.row_tiles = static_cast<int>((R + p.tile_rows - 1) / p.tile_rows);
  const long long groups = static_cast<long long>(B) * H * p.row_tiles;
  const long long tiles = (max_rows + 63) / 64;
  long long want = (1024 + groups - 1) / groups;
  if (want > tiles / 2) want = tiles / 2;
  if (want > 64) want = 64;
  p.splits = want < 1 ? 1 : static_cast<int>(want);
  p.slots = groups * p.splits;
  return p;
}

inline size_t part_bytes(const Plan &p, int D) {
  if (p.splits == 1) return 0;
  return round_up(static_cast<size_t>(p.slots) * p.tile_rows * D * 4, 256) +
         round_up(static_cast<size_t>(p.slots) * p.tile_rows * 8, 256) + round_up(static_cast<size_t>(p.slots) * 4, 256);
}

// A sequence's status; 0: its rows may be read.
__device__ inline int tree_status(const Params &P, int b) {
  const int n = P.c.kv_len[b];
  int st = n < 0 ? SPEC_ST_BAD_STATE : 0;
  const long long cap = cache_capacity(P.c);
  if (P.c.table) {
    if (static_cast<long long>(n) + P.N > cap) st |= SPEC_ST_CAPACITY;
  } else {
    const int E = *P.c.end_col;
    if (E < 0 || static_cast<long long>(E) + P.N > cap) st |= SPEC_ST_CAPACITY;
    if (n > E) st |= SPEC_ST_BAD_STATE;
  }
  return st;
}

template <typename T, int DP, int RW, bool PAGED>
__global__ __launch_bounds__(kThreads, DP <= 128 && sizeof(T) == 2 ? 2 : 1) void tree_kernel(Params P) {
  using S = Shape<T, DP, RW>;
  __shared__ __attribute__((aligned(16))) char buf0[S::kLds];
  __shared__ __attribute__((aligned(16))) char buf1[S::kLds];
  const int x = blockIdx.x;                               // ((b * H + h) * row_tiles + rt) * splits + s
  const int s = x % P.splits, y = x / P.splits, rt = y % P.row_tiles, bh = y / P.row_tiles;
  Job J;
  J.b = bh / P.c.H;
  J.h = bh - J.b * P.c.H;
  J.row0 = rt * 32 * RW;
  J.tokens = P.N;
  J.token0 = static_cast<long long>(J.b) * P.N;
  const int st = tree_status(P, J.b), n = P.c.kv_len[J.b];
  const bool reports = P.status && J.h == 0 && rt == 0;
  if (st) {
    if (s == 0) {
      put_zeros<T>(P, J, 32 * RW);
      if (reports && threadIdx.x == 0) P.status[J.b] = st;
    }
    return;
  }
  J.limit0 = n + 1;
  J.total = n + P.N;
  J.start_col = PAGED ? 0 : *P.c.end_col - n;
  const int tiles = (J.total + S::kKT - 1) / S::kKT;
  J.t0 = static_cast<int>(static_cast<long long>(tiles) * s / P.splits);
  J.t1 = static_cast<int>(static_cast<long long>(tiles) * (s + 1) / P.splits);
  const int bad = walk<T, DP, RW, PAGED, false>(P, J, P.splits > 1 ? x : -1, buf0, buf1);
  if (threadIdx.x == 0) {
    if (P.splits > 1)
      P.part_bad[x] = bad;
    else if (reports)
      P.status[J.b] = bad;
  }
}

// Joins the splits of one query row per wave, in split order.
template <typename T>
__global__ __launch_bounds__(kThreads) void tree_join_kernel(Params P, int tile_rows) {
  const int lane = threadIdx.x & (kWave - 1);
  const int R = P.N * P.G, D = P.c.D;
  const long long x = static_cast<long long>(blockIdx.x) * (kThreads / kWave) + threadIdx.x / kWave;
  if (x >= static_cast<long long>(P.B) * P.c.H * R) return;
  const int row = static_cast<int>(x % R), bh = static_cast<int>(x / R), b = bh / P.c.H, h = bh - b * P.c.H;
  if (tree_status(P, b)) return;                          // the first launch wrote its zeros
  const int token = row / P.G;
  const long long slot0 = (static_cast<long long>(bh) * P.row_tiles + row / tile_rows) * P.splits;
  const int at_row = row % tile_rows;
  const float2 *ml = reinterpret_cast<const float2 *>(P.part_ml);
  float m = -INFINITY, l = 0.0f;
  int bad = 0;
  if (lane < P.splits) {                                  // at most 64 splits
    const float2 v = ml[(slot0 + lane) * tile_rows + at_row];
    m = v.x;
    l = v.y;
    bad = P.part_bad[slot0 + lane];
  }
  const float top = wave_max_dpp(m), base = top == -INFINITY ? 0.0f : top;
  const float f = __builtin_amdgcn_exp2f((m - base) * P.sl);
  const float sum = wave_reduce(l * f, [](float a, float c) { return a + c; });
  bool sees = true;
  if (P.mask) {
    const uint32_t w = lane < P.words ? P.mask[(static_cast<long long>(b) * P.N + token) * P.words + lane] : 0u;
    sees = __any(w != 0);
  }
  const bool none = !sees || sum == 0.0f;
  const float inv = none ? 0.0f : 1.0f / sum;
  float o[4] = {};
  const int d0 = lane * 4;
  for (int s = 0; s < P.splits; ++s) {
    const float w = __shfl(f, s);                         // every lane takes part: lane s may hold no elements
    if (d0 < D) {
      const f32x4 v = *reinterpret_cast<const f32x4 *>(P.part_o + ((slot0 + s) * tile_rows + at_row) * D + d0);
#pragma unroll
      for (int j = 0; j < 4; ++j) o[j] = fmaf(v[j], w, o[j]);
    }
  }
  if (d0 < D) {
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = none ? 0.0f : o[j] * inv;
    const long long at = (static_cast<long long>(b) * P.N + token) * P.c.H * P.G + h * P.G + (row - token * P.G);
    put4<T>(P.out + at * D * sizeof(T), d0, D, o);
    if (P.lse && lane == 0) P.lse[at] = none ? -INFINITY : top * P.scale + logf(sum);
  }
  const bool any = __any(bad != 0);
  if (P.status && h == 0 && row == 0 && lane == 0) P.status[b] = any ? SPEC_ST_BAD_STATE : 0;
}

template <typename T, int DP, int RW>
void launch_rows(const Params &P, unsigned grid, hipStream_t s) {
  if (P.c.table)
    hipLaunchKernelGGL((tree_kernel<T, DP, RW, true>), dim3(grid), dim3(kThreads), 0, s, P);
  else
    hipLaunchKernelGGL((tree_kernel<T, DP, RW, false>), dim3(grid), dim3(kThreads), 0, s, P);
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

template <typename T>
int launch_all(const Params &P, const Plan &p, hipStream_t s) {
  (void)hipGetLastError();
  if (P.c.D <= 64)
    launch_tree<T, 64>(P, p, s);
  else if (P.c.D <= 128)
    launch_tree<T, 128>(P, p, s);
  else
    launch_tree<T, 256>(P, p, s);
  const int st = launch_status();
  if (st != SPEC_OK || p.splits == 1) return st;
  const long long rows = static_cast<long long>(P.B) * P.c.H * P.N * P.G;
  const unsigned grid = static_cast<unsigned>((rows + kThreads / kWave - 1) / (kThreads / kWave));
  hipLaunchKernelGGL(tree_join_kernel<T>, dim3(grid), dim3(kThreads), 0, s, P, p.tile_rows);
  return launch_status();
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
  const long long tokens = static_cast<long long>(B) * N;
  if (tokens * H * G >= INT32_MAX) return SPEC_EINVAL;
  const Plan p = plan_of(B, N, H, G, D, cache_capacity(P.c), dt);
  if (p.slots >= INT32_MAX) return SPEC_EINVAL;
  const size_t elt = dt == SPEC_BF16 ? 2 : 4, hd = static_cast<size_t>(H) * G * D, b4 = static_cast<size_t>(B) * 4;
  const int words = (N + 31) / 32;
  const size_t need = part_bytes(p, D);
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
  if (need && (!ws || ws_bytes < need || !aligned(ws, 256))) return SPEC_EWORKSPACE;
  P.N = N;
  P.words = words;
  P.mask = mask;
  P.splits = p.splits;
  P.row_tiles = p.row_tiles;
  if (need) {
    char *w = static_cast<char *>(ws);
    P.part_o = reinterpret_cast<float *>(w);
    w += round_up(static_cast<size_t>(p.slots) * p.tile_rows * D * 4, 256);
    P.part_ml = reinterpret_cast<float *>(w);
    w += round_up(static_cast<size_t>(p.slots) * p.tile_rows * 8, 256);
    P.part_bad = reinterpret_cast<int32_t *>(w);
  }
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
  if (static_cast<long long>(B) * N * H * G >= INT32_MAX) return 0;
  return part_bytes(plan_of(B, N, H, G, D, max_rows, dt), D);
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
