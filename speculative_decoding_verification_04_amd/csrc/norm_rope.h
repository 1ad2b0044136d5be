// Per-head norms of queries and keys, the position rotation, and the write of
// K and V into the cache, in one pass (gfx950): a cache of the inputs' type, or of
// 4-bit numbers.
//
// For a head x of D elements at position p:
//   y = x * w / sqrt(mean(x^2) + eps)            (w given; else y = x)
//   (y_a, y_b) -> (y_a cos t - y_b sin t, y_b cos t + y_a sin t),
//   t = p * inv_freq[i], pair i: (i, i + rot/2), or (2i, 2i + 1); the elements
//   from rot on are not rotated.
// V is copied.  Everything between the load and the one rounding at the store
// is float32; the norm's result is not rounded before the rotation.  The angle
// is reduced in float64 (p * inv_freq / 2 pi minus its nearest whole number),
// since in float32 a position of 10^5 would leave 2^-7 of a radian.
//
// Design.  Bound by HBM: each element is read once and written once.  One
// workgroup per token; a group of lanes takes one head, 16 bytes a lane, and
// every lane issues all loads that wait for nothing before it uses any.  The token's
// cosines and sines are computed once, by one lane each, and shared through LDS
// with the weights.  Partners (i, i + rot / 2) are a lane exchange apart where
// the distance is a power of two of chunks; else they are loaded again, one by
// one.  20.9k prompt tokens of 32 + 16 heads of 128 in bf16 (514 MB read and
// written) into four caches in turn: 90 us, 5.7 TB/s, where a large copy reaches
// 4.74 TB/s on the same card.
#pragma once

#include "mx.h"
#include "token_rows.h"

namespace specv {
namespace {

// Keys for 4-bit numbers are computed in float64: in float32 an element within
// 2^-22 of the border between two codes takes the wrong one (40 of the 21 million
// of 20.9k tokens of 8 heads of 128), and with it is off by half of itself.  Sine and
// cosine of t turns of the circle, t within [-1/2, 1/2]: their series on an eighth of the
// circle, within 2^-52.
__device__ inline void turn_of(double t, double &s, double &c) {
  const double quarter = rint(4.0 * t);
  const double x = (t - 0.25 * quarter) * 6.283185307179586477, y = x * x;   // |x| <= pi / 4
  // 1 / k! for odd and even k, alternating
  const double a = x + x * y * (-1.0 / 6 + y * (1.0 / 120 + y * (-1.0 / 5040 + y * (1.0 / 362880 +
                   y * (-1.0 / 39916800 + y * (1.0 / 6227020800.0 + y * (-1.0 / 1307674368000.0)))))));
  const double b = 1.0 + y * (-0.5 + y * (1.0 / 24 + y * (-1.0 / 720 + y * (1.0 / 40320 + y * (-1.0 / 3628800 +
                   y * (1.0 / 479001600 + y * (-1.0 / 87178291200.0 + y * (1.0 / 20922789888000.0))))))));
  const int q = static_cast<int>(quarter) & 3;            // 4 t is within [-2, 2]
  s = q == 0 ? a : q == 1 ? b : q == 2 ? -a : -b;
  c = q == 0 ? b : q == 1 ? -a : q == 2 ? -b : a;
}

constexpr int kMaxThreads = 256;
constexpr int kU = 3;      // heads in flight per lane (with 2 or 4, 20.9k tokens of 48 heads of 128 take 1 to 2% longer)

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

template <typename T, typename F>
__device__ inline void widen(u32x4 p, F (&x)[Vec<T>::n]) {
  typedef T V __attribute__((ext_vector_type(Vec<T>::n)));
  const V v = __builtin_bit_cast(V, p);
#pragma unroll
  for (int j = 0; j < Vec<T>::n; ++j) x[j] = static_cast<F>(static_cast<float>(v[j]));
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

__device__ inline float fma_of(float a, float b, float c) { return fmaf(a, b, c); }
__device__ inline double fma_of(double a, double b, double c) { return fma(a, b, c); }
__device__ inline float root_of(float x) { return sqrtf(x); }
__device__ inline double root_of(double x) { return sqrt(x); }

// A lane's elements of a head after norm and rotation, computed in F.  x: as
// loaded; src: the head; w: its weights or NULL, the same for a head's lanes; c, sn:
// cosines, and sines with the sign that the element's side takes.
template <typename T, Pairs PAIRS, typename F>
__device__ inline void turned(const RopeParams &P, u32x4 x, const T *src, const float *w, int e0, bool active,
                              const F (&c)[Vec<T>::n], const F (&sn)[Vec<T>::n], F (&a)[Vec<T>::n]) {
  constexpr int kN = Vec<T>::n;
  const int D = P.c.D, half = P.half, apart = half / kN;  // apart: chunks between partners
  // Element e turns with mate(e): e ^ 1, or e + half, or e - half.
  auto mate = [&](int e) {
    if (e >= 2 * half) return e;
    return PAIRS == kNext ? e ^ 1 : e < half ? e + half : e - half;
  };
  F m[kN];
  widen<T>(x, a);
  if constexpr (PAIRS == kChunksApart) {
    u32x4 y;
#pragma unroll
    for (int j = 0; j < 4; ++j) y[j] = __shfl_xor(x[j], apart);
    widen<T>(y, m);
  }
  if constexpr (PAIRS == kAny) {
#pragma unroll
    for (int j = 0; j < kN; ++j) m[j] = active ? static_cast<F>(static_cast<float>(src[mate(e0 + j)])) : F(0);
  }
  if (w) {
    F ss = 0;
#pragma unroll
    for (int j = 0; j < kN; ++j) ss = fma_of(a[j], a[j], ss);
    const F r = F(1) / root_of(group_sum(ss, P.lanes) / static_cast<F>(D) + static_cast<F>(P.eps));
#pragma unroll
    for (int j = 0; j < kN; ++j) a[j] = a[j] * r * static_cast<F>(w[e0 + j]);
    if constexpr (PAIRS == kChunksApart) {
      const float *wm = w + (e0 < 2 * half ? e0 ^ (apart * kN) : e0);
#pragma unroll
      for (int j = 0; j < kN; ++j) m[j] = m[j] * r * static_cast<F>(wm[j]);
    }
    if constexpr (PAIRS == kAny) {
#pragma unroll
      for (int j = 0; j < kN; ++j) m[j] = active ? m[j] * r * static_cast<F>(w[mate(e0 + j)]) : F(0);
    }
  }
  if constexpr (PAIRS == kNext) {
#pragma unroll
    for (int j = 0; j < kN; ++j) m[j] = a[j ^ 1];
  }
#pragma unroll
  for (int j = 0; j < kN; ++j) a[j] = e0 + j < 2 * half ? fma_of(m[j], sn[j], a[j] * c[j]) : a[j];
}

// A lane's elements of a head into a row of 4-bit numbers; `row`: the row's number
// in the layer's K or V.  A block's 32 elements are those of neighbouring lanes.
template <typename T>
__device__ inline void put_mx(const float (&x)[Vec<T>::n], char *codes, char *scales, long long row, int D, int e0,
                              bool store) {
  constexpr int kN = Vec<T>::n;
  uint32_t top = 0;
#pragma unroll
  for (int j = 0; j < kN; ++j) top = max(top, __float_as_uint(x[j]) & 0x7fffffffu);
  top = max(top, dpp_move<kDppQuadXor1>(top, top));
  top = max(top, dpp_move<kDppQuadXor2>(top, top));
  if constexpr (kN == 4) top = max(top, dpp_move<kDppRowHalfMirror>(top, top));
  const int byte = mx_scale_byte(top);
  const uint32_t c = mx_codes<kN>(x, byte);
  if (!store) return;
  char *to = codes + row * (D / 2) + e0 / 2;
  if constexpr (kN == 8) *reinterpret_cast<uint32_t *>(to) = c;
  else *reinterpret_cast<uint16_t *>(to) = static_cast<uint16_t>(c);
  if (e0 % kMxBlock == 0) scales[row * (D / kMxBlock) + e0 / kMxBlock] = static_cast<char>(byte);
}

template <typename T, Pairs PAIRS, bool MX>
__global__ __launch_bounds__(kMaxThreads, 4) void norm_rope_kernel(RopeParams P) {
  constexpr int kN = Vec<T>::n;
  __shared__ __attribute__((aligned(16))) float cosine[SPEC_ATTN_MAX_D / 2], sine[SPEC_ATTN_MAX_D / 2];
  __shared__ __attribute__((aligned(16))) float weight[2][SPEC_ATTN_MAX_D];
  __shared__ __attribute__((aligned(16))) double fine[2][MX ? SPEC_ATTN_MAX_D / 2 : 1];   // sines and cosines for keys
  const int lane = threadIdx.x & (kWave - 1);
  if (blockIdx.x >= static_cast<unsigned>(P.T)) {
    write_status(P, (blockIdx.x - P.T) * (blockDim.x / kWave) + threadIdx.x / kWave);
    return;
  }
  const int t = blockIdx.x;
  const int D = P.c.D, half = P.half;
  const int lph = P.lanes, g = threadIdx.x / lph, e0 = (threadIdx.x & (lph - 1)) * kN;
  const bool active = e0 < D;
  const int heads = P.Hq + 2 * P.c.H, step = blockDim.x / lph;
  // Head h of q, k and v in a row.  Sums of distances: from a choice between
  // pointers the compiler makes a choice between the addresses of arguments, and
  // each lane loads its pointer before it can ask for the data.
  const char *const rows_q = P.q + t * P.q_stride;
  const long long to_k = P.k + t * P.k_stride - rows_q - static_cast<long long>(P.Hq) * D * sizeof(T);
  const long long k_to_v = P.v + t * P.v_stride - (P.k + t * P.k_stride) - static_cast<long long>(P.c.H) * D * sizeof(T);
  const long long cache_k_to_v = P.c.v - P.c.k;
  auto source = [&](int h) {
    return rows_q + static_cast<long long>(h) * D * sizeof(T) + (h >= P.Hq ? to_k : 0) +
           (h >= P.Hq + P.c.H ? k_to_v : 0);
  };
  u32x4 x[kU];
  auto fetch = [&](int h0) __attribute__((always_inline)) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int h = h0 + u * step;
      x[u] = u32x4{0, 0, 0, 0};
      if (h < heads && active) x[u] = *reinterpret_cast<const u32x4 *>(source(h) + e0 * sizeof(T));
    }
  };
  // Everything that waits for nothing is asked for at once, the small things first
  // (loads come back in order): the first 64 sequences' state, the angles'
  // factors and the weights, then the heads.  What is absent is read from where
  // something is, since a branch around a load would end in a wait.  20.9k prompt
  // tokens of 48 heads of 128, replayed over four caches in turn, take 94 us so,
  // 104 with the heads first and a branch around each of the others.
  const int32_t *any = P.c.kv_len;
  const int own = t / max(P.N, 1), i0 = min(lane, P.B - 1);
  const int E0 = *(P.c.table ? any : P.c.end_col);
  const int pos_given = *(P.positions ? P.positions + t : any);
  const int lo0 = *(P.cu ? P.cu + i0 : any), hi0 = *(P.cu ? P.cu + i0 + 1 : any);
  const int n0 = P.c.kv_len[P.cu ? i0 : own];
  const float freq = *(half ? P.inv_freq + min(static_cast<int>(threadIdx.x), half - 1)
                            : reinterpret_cast<const float *>(any));
  const int iw = min(static_cast<int>(threadIdx.x), D - 1);
  const T wq = *(static_cast<const T *>(P.q_weight ? P.q_weight : any) + (P.q_weight ? iw : 0));
  const T wk = *(static_cast<const T *>(P.k_weight ? P.k_weight : any) + (P.k_weight ? iw : 0));
  fetch(g);
  const int E = P.c.table ? 0 : E0;
  int b = -1, t0 = 0, t1 = 0, n = n0;
  if (P.cu) {
    // the first sequence that holds token t, with no fall before it
    for (int b0 = 0; b0 < P.B; b0 += kWave) {
      const bool is = b0 + lane < P.B;
      const int i = min(b0 + lane, P.B - 1);
      const int lo = b0 ? P.cu[i] : lo0, hi = b0 ? P.cu[i + 1] : hi0, ni = b0 ? P.c.kv_len[i] : n0;
      const uint64_t who = __ballot(is && lo <= t && t < hi), falls = __ballot(is && lo > hi);
      if (who | falls) {
        const int l = __ffsll(static_cast<unsigned long long>(who | falls)) - 1;
        if (who >> l & 1) {
          b = b0 + l;
          t0 = read_lane(lo, l);
          t1 = read_lane(hi, l);
          n = read_lane(ni, l);
        }
        break;
      }
    }
    if (b < 0) return;                                    // a token of no sequence
  } else {
    b = own;
  }
  const Span s = span_of(P, b, t0, t1, n, E);
  const int row = s.row0 + (t - s.t0);
  bool write = s.st == 0;
  long long slot = 0;                                     // K's and V's offset of head 0
  if (write) {
    int plane = b, col = E - n + row;
    if (P.c.table) {
      const int i = cache_page(P.c, row);
      plane = P.c.table[static_cast<long long>(b) * P.c.max_pages + i];
      col = row - i * P.c.cols;
      write = plane >= 0 && plane < P.c.planes;
    }
    slot = cache_offset(P.c, write ? plane : 0, 0, col, MX ? 1 : sizeof(T));
    if (MX) slot /= D;                                    // the row's number
  }
  const long long head_step = MX ? P.c.cols : static_cast<long long>(P.c.cols) * D * sizeof(T);
  const int pos = P.positions ? pos_given : row;
  if (P.q_weight || P.k_weight) {
    for (int i = threadIdx.x; i < D; i += blockDim.x) {
      const bool first = i < static_cast<int>(blockDim.x);
      if (P.q_weight) weight[0][i] = static_cast<float>(first ? wq : static_cast<const T *>(P.q_weight)[i]);
      if (P.k_weight) weight[1][i] = static_cast<float>(first ? wk : static_cast<const T *>(P.k_weight)[i]);
    }
  }
  if (static_cast<int>(threadIdx.x) < half) {             // half <= 128; one wave may hold a token's few heads
    for (int i = threadIdx.x; i < half; i += blockDim.x) {
      const double angle = static_cast<double>(pos) * (i < static_cast<int>(blockDim.x) ? freq : P.inv_freq[i]);
      const double turn = angle * 0.15915494309189533577;
      if constexpr (MX) {
        // 1 / (2 pi) in two parts, and the product's own rounding: far positions keep 2^-52 of a turn
        const double rest = fma(angle, 0.15915494309189533577, -turn) + angle * -9.839338337591243e-18;
        turn_of(turn - rint(turn) + rest, fine[0][i], fine[1][i]);
        sine[i] = static_cast<float>(fine[0][i]);
        cosine[i] = static_cast<float>(fine[1][i]);
      } else {
        sincospif(2.0f * static_cast<float>(turn - rint(turn)), &sine[i], &cosine[i]);
      }
    }
  }
  __syncthreads();
  // a lane's cosines and sines from LDS, in F
  auto angles = [&](auto &c, auto &sn, const auto *cosines, const auto *sines) __attribute__((always_inline)) {
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      const int e = e0 + j;
      c[j] = 1;
      sn[j] = 0;
      if (e < 2 * half) {
        const int i = PAIRS == kNext ? e >> 1 : e < half ? e : e - half;
        c[j] = cosines[i];
        sn[j] = (PAIRS == kNext ? !(e & 1) : e < half) ? -sines[i] : sines[i];
      }
    }
  };
  float c[kN], sn[kN];
  angles(c, sn, cosine, sine);
  for (int h0 = g;; h0 += kU * step) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int h = h0 + u * step;
      if (h >= heads) break;
      const bool is_q = h < P.Hq, is_k = !is_q && h < P.Hq + P.c.H;
      const int hh = is_q ? h : is_k ? h - P.Hq : h - P.Hq - P.c.H;
      const bool store = active && (is_q || write);
      const T *src = reinterpret_cast<const T *>(source(h));
      float a[kN];
      if constexpr (MX) {
        if (!is_q) {
          if (is_k) {
            double cd[kN], sd[kN], y[kN];
            angles(cd, sd, fine[1], fine[0]);
            turned<T, PAIRS, double>(P, x[u], src, P.k_weight ? weight[1] : nullptr, e0, active, cd, sd, y);
#pragma unroll
            for (int j = 0; j < kN; ++j) a[j] = mx_sided(y[j]);
          } else {
            widen<T>(x[u], a);
          }
          put_mx<T>(a, is_k ? P.c.k : P.c.v, is_k ? P.c.ks : P.c.vs, slot + hh * head_step, D, e0, store);
          continue;
        }
      }
      char *to = is_q ? P.q_out + (static_cast<long long>(t) * P.Hq + hh) * D * sizeof(T) + e0 * sizeof(T)
                      : P.c.k + (is_k ? 0 : cache_k_to_v) + slot + hh * head_step + e0 * sizeof(T);
      if (!is_q && !is_k) {
        if (store) *reinterpret_cast<u32x4 *>(to) = x[u];
        continue;
      }
      turned<T, PAIRS, float>(P, x[u], src, is_q ? P.q_weight ? weight[0] : nullptr : P.k_weight ? weight[1] : nullptr,
                              e0, active, c, sn, a);
      if (store) *reinterpret_cast<u32x4 *>(to) = narrow<T>(a);
    }
    if (h0 + kU * step >= heads) break;
    fetch(h0 + kU * step);
  }
}

template <typename T, bool MX>
int launch_rope(const RopeParams &P, Pairs pairs, unsigned grid, int threads, hipStream_t s) {
  switch (pairs) {
    case kNext: hipLaunchKernelGGL((norm_rope_kernel<T, kNext, MX>), dim3(grid), dim3(threads), 0, s, P); break;
    case kChunksApart: hipLaunchKernelGGL((norm_rope_kernel<T, kChunksApart, MX>), dim3(grid), dim3(threads), 0, s, P); break;
    default: hipLaunchKernelGGL((norm_rope_kernel<T, kAny, MX>), dim3(grid), dim3(threads), 0, s, P); break;
  }
  return launch_status();
}

template <bool MX>
int norm_rope_call(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                   int64_t v_stride, void *kv, void *scales, spec_dtype dt, int L, int planes, int H, int cols, int D, int layer,
                   int T, int B, int N, int G, const int32_t *table, int max_pages, bool paged,
                   const int32_t *end_col, const int32_t *kv_len, const int32_t *cu, const int32_t *positions,
                   const void *q_weight, const void *k_weight, float eps, const float *inv_freq, int rot,
                   int interleaved, void *q_out, int32_t *status, spec_stream_t stream) {
  if (!q || !k || !v || !q_out || (rot && !inv_freq)) return SPEC_EINVAL;
  RopeParams P;
  if (dt != SPEC_F32 && dt != SPEC_BF16) return SPEC_EINVAL;
  const int err =
      MX ? mx_view(P.c, kv, scales, L, planes, H, cols, D, layer, table, max_pages, paged, end_col, kv_len)
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
  const int waves = threads / kWave;
  const unsigned grid = static_cast<unsigned>(T) + (status ? (static_cast<long long>(B) + waves - 1) / waves : 0);
  if (!launchable(grid, threads)) return SPEC_EINVAL;
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
  const size_t out_n[] = {MX ? rows * (D / 2) : cache_bytes(dt, L, planes, H, cols, D), rows * (D / kMxBlock),
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
  (void)hipGetLastError();
  const hipStream_t s = static_cast<hipStream_t>(stream);
  const int n = 16 / elt, apart = P.half / n;
  const Pairs pairs = interleaved ? kNext : P.half % n == 0 && (apart & (apart - 1)) == 0 ? kChunksApart : kAny;
  return dt == SPEC_BF16 ? launch_rope<__bf16, MX>(P, pairs, grid, threads, s)
                        : launch_rope<float, MX>(P, pairs, grid, threads, s);
}

}  // namespace
}  // namespace specv
