// Commit of a tree over pages: the accepted path's slots moved together (gfx950).
//
// The forward over a candidate tree wrote node i's K and V at row n + i of its
// sequence, which lies in pages.  The slots path[0 .. e-1] are kept (node indices that
// rise, from the root 0) and have to be rows n .. n + e - 1 before the lengths are
// committed: row n + path[j] becomes row n + j, in every layer, K/V and head.
//
// As in the rectangle's compaction, path[j] >= j with equality on a prefix, so the
// slots that move are a tail j0 .. e - 1, slot j takes from a larger one that no later
// slot takes from again, and every pass reads all its sources before it writes.
//
// Design.  A copy of a few rows, bound by latency for one tree and by memory for
// many.  One workgroup per (sequence, layer and K/V, group of heads): it checks the
// path and its pages in one round of loads with a lane per slot, leaves the slots'
// offsets in LDS, and moves units of up to 16 bytes.
// Measured: 32 trees of 63 nodes with 2 .. 24 kept, 28 layers of 4 heads of 128 in bf16
// (45 MB read and written) 12.6 us = 3.6 TB/s, two dependent rounds of loads before the
// first row moves; one tree of 16 nodes, 32 layers of 8 heads, 3.6 us.
#include <algorithm>

#include "cache_view.h"

namespace specv {
namespace {

constexpr int kThreads = 256;
constexpr int kU = 4;        // units in flight per lane
static_assert(kThreads >= SPEC_TREE_MAX_N, "a lane for each tree node");

struct PagedCompactParams {
  CacheView c;               // layer 0's K; the layers' K and V follow each other
  int B, N, R;               // R: bytes of a row
  int hpb, hsplit;           // heads of a workgroup, workgroups of a (sequence, layer, K/V)
  long long half;            // bytes of one layer's K
  const int32_t *path, *emit_count;
  int32_t *status;
};

template <int VB>
__global__ __launch_bounds__(kThreads) void paged_compact_kernel(PagedCompactParams P) {
  using VT = typename VecOf<VB>::T;
  __shared__ long long src[SPEC_TREE_MAX_N], dst[SPEC_TREE_MAX_N];   // of moved slots, in rows
  const int t = threadIdx.x;
  const int b = blockIdx.x % P.B, rest = blockIdx.x / P.B;           // consecutive workgroups: consecutive sequences
  const int hs = rest % P.hsplit, lk = rest / P.hsplit;              // lk: layer * 2 + (K or V)
  const int32_t *pb = P.path + static_cast<long long>(b) * P.N;
  const int node = t < P.N ? pb[t] : -1, prev = t > 0 && t < P.N ? pb[t - 1] : -1;
  const int e = P.emit_count[b], n = P.c.kv_len[b];
  int st = n < 0 || e < 0 || e > P.N ? SPEC_ST_BAD_STATE : 0;
  if (n >= 0 && static_cast<long long>(n) + P.N > cache_capacity(P.c)) st |= SPEC_ST_CAPACITY;
  bool ok = true, moves = false;
  long long from = 0, to = 0;
  if (!st && t < e) {
    ok = node > prev && node < P.N && (t > 0 || node == 0);
    if (ok) {
      moves = node != t;
      const int32_t *table = P.c.table + static_cast<long long>(b) * P.c.max_pages;
      const int rf = n + node, rt = n + t, pf = cache_page(P.c, rf), pt = cache_page(P.c, rt);
      const int of = table[pf], at = table[pt];
      ok = of >= 0 && of < P.c.planes && at >= 0 && at < P.c.planes;
      from = static_cast<long long>(of) * P.c.H * P.c.cols + (rf - pf * P.c.cols);
      to = static_cast<long long>(at) * P.c.H * P.c.cols + (rt - pt * P.c.cols);
    }
  }
  if (!__syncthreads_and(ok)) st |= SPEC_ST_BAD_STATE;
  if (P.status && lk == 0 && hs == 0 && t == 0) P.status[b] = st;
  if (st) return;                                         // the same for all of the sequence's workgroups
  if (moves) {
    src[t] = from;
    dst[t] = to;
  }
  const int moved = __syncthreads_count(moves), j0 = e - moved;      // barrier: the offsets are visible
  const int h0 = hs * P.hpb, nh = min(P.hpb, P.c.H - h0);
  if (moved <= 0 || nh <= 0) return;
  const int per_row = P.R / VB, per_head = moved * per_row, units = nh * per_head;
  char *base = P.c.k + lk * P.half + static_cast<long long>(h0) * P.c.cols * P.R;
  for (int u0 = 0; u0 < units; u0 += kThreads * kU) {
    VT x[kU];
    VT *out[kU];
#pragma unroll
    for (int q = 0; q < kU; ++q) {
      const int u = u0 + q * kThreads + t;
      out[q] = nullptr;
      if (u < units) {
        const int h = u / per_head, r = u - h * per_head, m = r / per_row, v = r - m * per_row;
        char *head = base + static_cast<long long>(h) * P.c.cols * P.R + v * VB;
        x[q] = *reinterpret_cast<const VT *>(head + src[j0 + m] * P.R);
        out[q] = reinterpret_cast<VT *>(head + dst[j0 + m] * P.R);
      }
    }
#pragma unroll
    for (int q = 0; q < kU; ++q)
      if (out[q]) hold(x[q]);
    __syncthreads();                                      // every source of the pass is read
#pragma unroll
    for (int q = 0; q < kU; ++q)
      if (out[q]) *out[q] = x[q];
  }
}

}  // namespace
}  // namespace specv

using namespace specv;

extern "C" int spec_compact_tree_paged(void *pool, spec_dtype dt, int L, int pages, int H, int page_size, int D, int B,
                                       int N, const int32_t *block_table, int max_pages, const int32_t *kv_len,
                                       const int32_t *path, const int32_t *emit_count, int32_t *status,
                                       spec_stream_t stream) {
  if (!path || !emit_count) return SPEC_EINVAL;
  PagedCompactParams P;
  const int err = cache_view(P.c, pool, dt, L, pages, H, page_size, D, 0, block_table, max_pages, true, nullptr, kv_len);
  if (err) return err;
  if (B < 1 || N < 1) return SPEC_EINVAL;
  if (N > SPEC_TREE_MAX_N) return SPEC_ECAPACITY;
  const int elt = dt == SPEC_BF16 ? 2 : 4;
  if (!aligned(pool, elt) || !aligned(status, 4)) return SPEC_EINVAL;
  const long long R = static_cast<long long>(D) * elt;
  // units of a workgroup and a row's bytes in 31 bits
  if (R > INT32_MAX / SPEC_TREE_MAX_N || static_cast<long long>(H) * N * R >= INT32_MAX) return SPEC_EINVAL;
  if (static_cast<long long>(L) * B >= INT32_MAX / 2) return SPEC_EINVAL;
  // four workgroups a CU: each sequence's heads are split where its layers alone are too
  // few (32 trees, 28 layers: 1792 workgroups of 4 heads take 13.3 us, twice as many of 2
  // heads 14.1, since each has the path to look up first)
  const long long groups = static_cast<long long>(B) * 2 * L;
  const int split = static_cast<int>(std::min<long long>(H, std::max<long long>(1, (1024 + groups - 1) / groups)));
  P.hpb = (H + split - 1) / split;
  P.hsplit = (H + P.hpb - 1) / P.hpb;
  if (!launchable(groups * P.hsplit, kThreads)) return SPEC_EINVAL;
  const size_t b4 = static_cast<size_t>(B) * 4, bytes = cache_bytes(dt, L, pages, H, page_size, D);
  const void *ins[] = {block_table, kv_len, path, emit_count};
  const size_t in_n[] = {b4 * max_pages, b4, b4 * N, b4};
  for (int j = 0; j < 4; ++j)
    if (overlaps(pool, bytes, ins[j], in_n[j]) || overlaps(status, b4, ins[j], in_n[j])) return SPEC_EINVAL;
  if (overlaps(status, b4, pool, bytes)) return SPEC_EINVAL;
  P.B = B;
  P.N = N;
  P.R = static_cast<int>(R);
  P.half = static_cast<long long>(pages) * H * page_size * R;
  P.path = path;
  P.emit_count = emit_count;
  P.status = status;
  const dim3 grid(static_cast<unsigned>(groups * P.hsplit)), block(kThreads);
  const hipStream_t s = static_cast<hipStream_t>(stream);
  (void)hipGetLastError();
  if (R % 16 == 0 && aligned(pool, 16))
    hipLaunchKernelGGL(paged_compact_kernel<16>, grid, block, 0, s, P);
  else if (R % 8 == 0 && aligned(pool, 8))
    hipLaunchKernelGGL(paged_compact_kernel<8>, grid, block, 0, s, P);
  else if (R % 4 == 0 && aligned(pool, 4))
    hipLaunchKernelGGL(paged_compact_kernel<4>, grid, block, 0, s, P);
  else
    hipLaunchKernelGGL(paged_compact_kernel<2>, grid, block, 0, s, P);
  return launch_status();
}
