// How the attention half of the verify forward finds a sequence's rows in a
// KV cache (gfx950), shared by the cache write and the attention kernels.
//
// One layer of a cache is two arrays (K and V) of planes [planes][H][cols][D].
// In the left-padded rectangle a plane is a sequence and row r of sequence b
// lies at column E - n + r of plane b; in a page pool a plane is a page and
// row r lies at column r % cols of plane table[b][r / cols].
#pragma once

#include "common.h"

namespace specv {

struct CacheView {
  char *k, *v;              // the layer's K and V planes
  int H, cols, D, planes;   // cols: C of the rectangle, or the page size
  const int32_t *table;     // block table [B][max_pages], or NULL: a rectangle
  int max_pages;
  uint32_t div_m;           // r / cols = (r * div_m) >> (31 + div_s) for 0 <= r < 2^31
  int div_s;
  const int32_t *end_col;   // rectangle: device scalar E
  const int32_t *kv_len;    // [B]
};

// Whether a launch's work-items fit the 32 bits that a grid's x has for them:
// past that a launch fails, and calls refuse before they enqueue anything.
inline bool launchable(long long workgroups, int threads) { return workgroups * threads <= UINT32_MAX; }

// Division of a 31-bit number by d >= 1: with s = ceil(log2 d) and
// m = ceil(2^(31+s) / d) < 2^32 the product's error r * (m d - 2^(31+s)) / d is
// below 2^(31+s) / d for r < 2^31, so (r * m) >> (31 + s) is exact.
inline void cache_divisor(CacheView &c) {
  int s = 0;
  while ((1ll << s) < c.cols) ++s;
  c.div_s = s;
  c.div_m = static_cast<uint32_t>(((1ull << (31 + s)) + c.cols - 1) / c.cols);
}

__device__ inline int cache_page(const CacheView &c, int r) {
  return static_cast<int>((static_cast<uint64_t>(static_cast<uint32_t>(r)) * c.div_m) >> (31 + c.div_s));
}

// Bytes from a layer's K (or V) base to column col of (plane, head).
__device__ inline long long cache_offset(const CacheView &c, int plane, int h, int col, int elt) {
  return ((static_cast<long long>(plane) * c.H + h) * c.cols + col) * c.D * elt;
}

// Rows a sequence may have, whatever its state.
__host__ __device__ inline long long cache_capacity(const CacheView &c) {
  return c.table ? static_cast<long long>(c.max_pages) * c.cols : c.cols;
}

// Host checks shared by the calls that take a cache; fills the view of one
// layer.  Returns SPEC_OK or SPEC_EINVAL.
inline int cache_view(CacheView &c, const void *kv, spec_dtype dt, int L, int planes, int H, int cols, int D,
                      int layer, const int32_t *table, int max_pages, bool paged, const int32_t *end_col,
                      const int32_t *kv_len) {
  if (!kv || !kv_len || (paged ? !table : !end_col)) return SPEC_EINVAL;
  if (dt != SPEC_F32 && dt != SPEC_BF16) return SPEC_EINVAL;
  if (L < 1 || planes < 1 || H < 1 || cols < 1 || D < 1 || layer < 0 || layer >= L) return SPEC_EINVAL;
  // row numbers, rounded up to whole tiles, stay below 2^31
  if (paged && max_pages < 1) return SPEC_EINVAL;
  if ((paged ? static_cast<long long>(max_pages) : 1ll) * cols > INT32_MAX - 512) return SPEC_EINVAL;
  const long long elt = dt == SPEC_BF16 ? 2 : 4;
  const long long half = static_cast<long long>(planes) * H * cols * D * elt;  // one layer's K
  c.k = static_cast<char *>(const_cast<void *>(kv)) + 2 * half * layer;
  c.v = c.k + half;
  c.H = H;
  c.cols = cols;
  c.D = D;
  c.planes = planes;
  c.table = paged ? table : nullptr;
  c.max_pages = paged ? max_pages : 0;
  c.end_col = paged ? nullptr : end_col;
  c.kv_len = kv_len;
  cache_divisor(c);
  return SPEC_OK;
}

inline size_t cache_bytes(spec_dtype dt, int L, int planes, int H, int cols, int D) {
  return static_cast<size_t>(L) * 2 * planes * H * cols * D * (dt == SPEC_BF16 ? 2 : 4);
}

}  // namespace specv
