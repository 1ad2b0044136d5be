// Per-head norms of queries and keys and the position rotation (gfx950): what the
// kernels that write caches of a type and of 4-bit numbers share.
//
// For a head x of D elements at position p:
//   y = x * w / sqrt(mean(x^2) + eps)            (w given; else y = x)
//   (y_a, y_b) -> (y_a cos t - y_b sin t, y_b cos t + y_a sin t),
//   t = p * inv_freq[i], pair i: (i, i + rot/2), or (2i, 2i + 1); the elements
//   from rot on are not rotated.
#pragma once

#include "mx.h"
#include "token_rows.h"

namespace specv {
namespace {

constexpr int kMaxThreads = 256;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

struct RopeParams : TokenRows {
  const char *q, *k, *v;
  long long q_stride, k_stride, v_stride;   // bytes from token to token
  char *q_out;
  int Hq, half, lanes;       // lanes: per head
  const int32_t *positions;
  const void *q_weight, *k_weight;
  float eps;
  const float *inv_freq;
};

template <typename T> struct Vec;
template <> struct Vec<float> { static constexpr int n = 4; };
template <> struct Vec<__bf16> { static constexpr int n = 8; };

template <typename T>
__device__ inline void widen(u32x4 p, float (&x)[Vec<T>::n]) {
  typedef T V __attribute__((ext_vector_type(Vec<T>::n)));
  const V v = __builtin_bit_cast(V, p);
#pragma unroll
  for (int j = 0; j < Vec<T>::n; ++j) x[j] = static_cast<float>(v[j]);
}

template <typename T>
__device__ inline u32x4 narrow(const float (&x)[Vec<T>::n]) {
  typedef T V __attribute__((ext_vector_type(Vec<T>::n)));
  V v;
#pragma unroll
  for (int j = 0; j < Vec<T>::n; ++j) v[j] = static_cast<T>(x[j]);
  return __builtin_bit_cast(u32x4, v);
}

// Sum over the lanes of a head's group (a power of two, aligned): lane moves
// within 16 lanes, exchanges beyond.
template <typename F>
__device__ inline F group_sum(F x, int lanes) {
  if (lanes > 1) x += dpp_move<kDppQuadXor1>(x, x);
  if (lanes > 2) x += dpp_move<kDppQuadXor2>(x, x);
  if (lanes > 4) x += dpp_move<kDppRowHalfMirror>(x, x);
  if (lanes > 8) x += dpp_move<kDppRowMirror>(x, x);
  if (lanes > 16) x += __shfl_xor(x, 16);
  if (lanes > 32) x += __shfl_xor(x, 32);
  return x;
}

// Where a pair's partner lies: the neighbouring element, a power of two of
// chunks away, or anywhere.
enum Pairs { kNext, kChunksApart, kAny };

// Workgroups of a token each, and those that write the status, a wave for each sequence.
inline long long rope_grid(int tokens, int B, const void *status, int waves) {
  return static_cast<long long>(tokens) + (status ? (static_cast<long long>(B) + waves - 1) / waves : 0);
}

// Host checks of a call, into a cache of dt's elements or of 4-bit numbers, but for its
// launch; fills P.  threads: one token's heads, in whole waves.
struct RopeShape {
  Pairs pairs;
  int threads;
};

inline int rope_params(RopeParams &P, RopeShape &shape, bool mx, const void *q, int64_t q_stride, const void *k,
                       int64_t k_stride, const void *v, int64_t v_stride, void *kv, void *scales, spec_dtype dt, int L,
                       int planes, int H, int cols, int D, int layer, int T, int B, int N, int G,
                       const int32_t *table, int max_pages, bool paged, const int32_t *end_col, const int32_t *kv_len,
                       const int32_t *cu, const int32_t *positions, const void *q_weight, const void *k_weight,
                       float eps, const float *inv_freq, int rot, int interleaved, void *q_out, int32_t *status) {
  if (!q || !k || !v || !q_out || (rot && !inv_freq)) return SPEC_EINVAL;
  if (dt != SPEC_F32 && dt != SPEC_BF16) return SPEC_EINVAL;
  const int err =
      mx ? mx_view(P.c, kv, scales, L, planes, H, cols, D, layer, table, max_pages, paged, end_col, kv_len)
         : cache_view(P.c, kv, dt, L, planes, H, cols, D, layer, table, max_pages, paged, end_col, kv_len);
  if (err) return err;
  if (T < 1 || B < 1 || G < 1 || (!paged && planes != B)) return SPEC_EINVAL;
  if (cu ? N != 0 : N < 1 || static_cast<long long>(B) * N != T) return SPEC_EINVAL;
  if (rot < 0 || rot > D || rot % 2 || !(eps >= 0.0f) || eps > 3.4e38f) return SPEC_EINVAL;
  if (D > SPEC_ATTN_MAX_D) return SPEC_ECAPACITY;
  const int elt = dt == SPEC_BF16 ? 2 : 4, Hq = H * G;
  if (static_cast<long long>(H) * (G + 2) >= INT32_MAX / D || static_cast<long long>(T) + B >= INT32_MAX)
    return SPEC_EINVAL;
  P.lanes = 1;
  while (P.lanes * (16 / elt) < D) P.lanes *= 2;
  // one token's heads, in whole waves
  const long long lanes = static_cast<long long>(H) * (G + 2) * P.lanes;
  const int threads = static_cast<int>(lanes < kMaxThreads ? round_up(lanes, kWave) : kMaxThreads);
  const long long qh = static_cast<long long>(Hq) * D, kh = static_cast<long long>(H) * D;
  if (D * elt % 16 || q_stride < qh || k_stride < kh || v_stride < kh) return SPEC_EINVAL;
  if (q_stride * elt % 16 || k_stride * elt % 16 || v_stride * elt % 16) return SPEC_EINVAL;
  const void *wide[] = {q, k, v, kv, q_out};
  for (const void *p : wide)
    if (!aligned(p, 16)) return SPEC_EINVAL;
  if (!aligned(q_weight, elt) || !aligned(k_weight, elt) || !aligned(inv_freq, 4)) return SPEC_EINVAL;
  const size_t b4 = static_cast<size_t>(B) * 4, d = static_cast<size_t>(D) * elt;
  const void *ins[] = {q, k, v, table, end_col, kv_len, cu, positions, q_weight, k_weight, inv_freq};
  const size_t in_n[] = {((T - 1) * static_cast<size_t>(q_stride) + qh) * elt,
                         ((T - 1) * static_cast<size_t>(k_stride) + kh) * elt,
                         ((T - 1) * static_cast<size_t>(v_stride) + kh) * elt,
                         paged ? b4 * max_pages : 0, paged ? 0u : 4u, b4, b4 + 4, static_cast<size_t>(T) * 4, d, d,
                         static_cast<size_t>(rot) * 2};
  const size_t rows = mx_rows(L, planes, H, cols);
  const void *outs[] = {kv, scales, q_out, status};
  const size_t out_n[] = {mx ? rows * (D / 2) : cache_bytes(dt, L, planes, H, cols, D), rows * (D / kMxBlock),
                          static_cast<size_t>(T) * qh * elt, b4};
  for (int o = 0; o < 4; ++o) {
    for (int j = 0; j < 11; ++j)
      if (overlaps(outs[o], out_n[o], ins[j], in_n[j])) return SPEC_EINVAL;
    for (int j = o + 1; j < 4; ++j)
      if (overlaps(outs[o], out_n[o], outs[j], out_n[j])) return SPEC_EINVAL;
  }
  P.q = static_cast<const char *>(q);
  P.k = static_cast<const char *>(k);
  P.v = static_cast<const char *>(v);
  P.q_stride = q_stride * elt;
  P.k_stride = k_stride * elt;
  P.v_stride = v_stride * elt;
  P.q_out = static_cast<char *>(q_out);
  P.T = T;
  P.B = B;
  P.N = N;
  P.Hq = Hq;
  P.half = rot / 2;
  P.cu = cu;
  P.positions = positions;
  P.q_weight = q_weight;
  P.k_weight = k_weight;
  P.eps = eps;
  P.inv_freq = inv_freq;
  P.status = status;
  const int n = 16 / elt, apart = P.half / n;
  shape.pairs = interleaved ? kNext : P.half % n == 0 && (apart & (apart - 1)) == 0 ? kChunksApart : kAny;
  shape.threads = threads;
  return SPEC_OK;
}

}  // namespace
}  // namespace specv
