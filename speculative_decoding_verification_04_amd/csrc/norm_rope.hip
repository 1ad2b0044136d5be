// Per-head norms of queries and keys, the position rotation, and the write of
// K and V into the cache, in one pass (gfx950).
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
#include "cache_view.h"

namespace specv {
namespace {

constexpr int kMaxThreads = 256;
constexpr int kU = 3;      // heads in flight per lane (with 2 or 4, 20.9k tokens of 48 heads of 128 take 1 to 2% longer)

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

struct RopeParams {
  CacheView c;
  const char *q, *k, *v;
  long long q_stride, k_stride, v_stride;   // bytes from token to token
  char *q_out;
  int T, B, N, Hq, half, lanes;  // N 0: packed; lanes: per head
  const int32_t *cu, *positions;
  const void *q_weight, *k_weight;
  float eps;
  const float *inv_freq;
  int32_t *status;
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

// A sequence's new tokens and where their rows start.
struct Span {
  int t0, len, row0;   // first token, tokens, first row
  int st;              // status bits; nonzero: nothing is written to the cache
};

// t0, t1: the sequence's token range (packed calls); n: its length; E: the
// rectangle's end (pages: 0).
__device__ inline Span span_of(const RopeParams &P, int b, int t0, int t1, int n, int E) {
  Span s;
  s.st = 0;
  if (P.cu) {
    // no difference is taken before its operands are known to be in range
    const bool in = t0 >= 0 && t0 <= t1 && t1 <= P.T;
    s.t0 = in ? t0 : 0;
    s.len = in ? t1 - t0 : 0;
    if (!in || n < s.len) s.st = SPEC_ST_BAD_STATE;
    s.row0 = s.st ? 0 : n - s.len;
  } else {
    s.t0 = b * P.N;
    s.len = P.N;
    s.row0 = n;
    if (n < 0) s.st = SPEC_ST_BAD_STATE;
  }
  const long long cap = cache_capacity(P.c), end = static_cast<long long>(n) + (P.cu ? 0 : P.N);
  if (P.c.table) {
    if (end > cap) s.st |= SPEC_ST_CAPACITY;
  } else {
    if (E < 0 || static_cast<long long>(E) + (P.cu ? 0 : P.N) > cap) s.st |= SPEC_ST_CAPACITY;
    if (n > E) s.st |= SPEC_ST_BAD_STATE;
  }
  return s;
}

// The status of one sequence per wave: its span and the pages of its new rows.
__device__ inline void write_status(const RopeParams &P, int b) {
  const int lane = threadIdx.x & (kWave - 1);
  if (b >= P.B) return;
  const Span s = span_of(P, b, P.cu ? P.cu[b] : 0, P.cu ? P.cu[b + 1] : 0, P.c.kv_len[b], P.c.table ? 0 : *P.c.end_col);
  int st = s.st;
  if (P.cu) {
    bool falls = false;                                   // before the sequence
    for (int i = lane; i < b; i += kWave) falls |= P.cu[i] > P.cu[i + 1];
    if (__any(falls)) st |= SPEC_ST_BAD_STATE;
  }
  if (!st && P.c.table && s.len > 0) {
    bool bad = false;
    const int last = cache_page(P.c, s.row0 + s.len - 1);
    for (int i = cache_page(P.c, s.row0) + lane; i <= last; i += kWave) {
      const int page = P.c.table[static_cast<long long>(b) * P.c.max_pages + i];
      bad |= page < 0 || page >= P.c.planes;
    }
    if (__any(bad)) st = SPEC_ST_BAD_STATE;
  }
  if (lane == 0) P.status[b] = st;
}

// Sum over the lanes of a head's group (a power of two, aligned): lane moves
// within 16 lanes, exchanges beyond.
__device__ inline float group_sum(float x, int lanes) {
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

template <typename T, Pairs PAIRS>
__global__ __launch_bounds__(kMaxThreads, 4) void norm_rope_kernel(RopeParams P) {
  constexpr int kN = Vec<T>::n;
  __shared__ __attribute__((aligned(16))) float cosine[SPEC_ATTN_MAX_D / 2], sine[SPEC_ATTN_MAX_D / 2];
  __shared__ __attribute__((aligned(16))) float weight[2][SPEC_ATTN_MAX_D];
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
    slot = cache_offset(P.c, write ? plane : 0, 0, col, sizeof(T));
  }
  const long long head_step = static_cast<long long>(P.c.cols) * D * sizeof(T);
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
      const double turn =
          static_cast<double>(pos) * (i < static_cast<int>(blockDim.x) ? freq : P.inv_freq[i]) * 0.15915494309189533577;
      sincospif(2.0f * static_cast<float>(turn - rint(turn)), &sine[i], &cosine[i]);
    }
  }
  __syncthreads();
  // Element e turns with mate(e): e ^ 1, or e + half, or e - half.
  auto mate = [&](int e) {
    if (e >= 2 * half) return e;
    return PAIRS == kNext ? e ^ 1 : e < half ? e + half : e - half;
  };
  float c[kN], sn[kN];                                    // sn: the sine with the sign that the element's side takes
#pragma unroll
  for (int j = 0; j < kN; ++j) {
    const int e = e0 + j;
    c[j] = 1.0f;
    sn[j] = 0.0f;
    if (e < 2 * half) {
      const int i = PAIRS == kNext ? e >> 1 : e < half ? e : e - half;
      c[j] = cosine[i];
      sn[j] = (PAIRS == kNext ? !(e & 1) : e < half) ? -sine[i] : sine[i];
    }
  }
  const int apart = half / kN;                            // chunks between partners
  for (int h0 = g;; h0 += kU * step) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int h = h0 + u * step;
      if (h >= heads) break;
      const bool is_q = h < P.Hq, is_k = !is_q && h < P.Hq + P.c.H;
      const int hh = is_q ? h : is_k ? h - P.Hq : h - P.Hq - P.c.H;
      char *to = is_q ? P.q_out + (static_cast<long long>(t) * P.Hq + hh) * D * sizeof(T) + e0 * sizeof(T)
                      : P.c.k + (is_k ? 0 : cache_k_to_v) + slot + hh * head_step + e0 * sizeof(T);
      const bool store = active && (is_q || write);
      if (!is_q && !is_k) {
        if (store) *reinterpret_cast<u32x4 *>(to) = x[u];
        continue;
      }
      float a[kN], m[kN];
      widen<T>(x[u], a);
      if constexpr (PAIRS == kChunksApart) {
        u32x4 y;
#pragma unroll
        for (int j = 0; j < 4; ++j) y[j] = __shfl_xor(x[u][j], apart);
        widen<T>(y, m);
      }
      if constexpr (PAIRS == kAny) {
        const T *src = reinterpret_cast<const T *>(source(h));
#pragma unroll
        for (int j = 0; j < kN; ++j) m[j] = active ? static_cast<float>(src[mate(e0 + j)]) : 0.0f;
      }
      if (is_q ? P.q_weight : P.k_weight) {               // the same for a head's lanes
        float ss = 0.0f;
#pragma unroll
        for (int j = 0; j < kN; ++j) ss = fmaf(a[j], a[j], ss);
        const float r = 1.0f / sqrtf(group_sum(ss, lph) / static_cast<float>(D) + P.eps);
        const float *w = weight[is_q ? 0 : 1];
#pragma unroll
        for (int j = 0; j < kN; ++j) a[j] = a[j] * r * w[e0 + j];
        if constexpr (PAIRS == kChunksApart) {
          const float *wm = w + (e0 < 2 * half ? e0 ^ (apart * kN) : e0);
#pragma unroll
          for (int j = 0; j < kN; ++j) m[j] = m[j] * r * wm[j];
        }
        if constexpr (PAIRS == kAny) {
#pragma unroll
          for (int j = 0; j < kN; ++j) m[j] = active ? m[j] * r * w[mate(e0 + j)] : 0.0f;
        }
      }
      if constexpr (PAIRS == kNext) {
#pragma unroll
        for (int j = 0; j < kN; ++j) m[j] = a[j ^ 1];
      }
#pragma unroll
      for (int j = 0; j < kN; ++j) a[j] = e0 + j < 2 * half ? fmaf(m[j], sn[j], a[j] * c[j]) : a[j];
      if (store) *reinterpret_cast<u32x4 *>(to) = narrow<T>(a);
    }
    if (h0 + kU * step >= heads) break;
    fetch(h0 + kU * step);
  }
}

template <typename T>
int launch_rope(const RopeParams &P, Pairs pairs, unsigned grid, int threads, hipStream_t s) {
  switch (pairs) {
    case kNext: hipLaunchKernelGGL((norm_rope_kernel<T, kNext>), dim3(grid), dim3(threads), 0, s, P); break;
    case kChunksApart: hipLaunchKernelGGL((norm_rope_kernel<T, kChunksApart>), dim3(grid), dim3(threads), 0, s, P); break;
    default: hipLaunchKernelGGL((norm_rope_kernel<T, kAny>), dim3(grid), dim3(threads), 0, s, P); break;
  }
  return launch_status();
}

int norm_rope_call(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                   int64_t v_stride, void *kv, spec_dtype dt, int L, int planes, int H, int cols, int D, int layer,
                   int T, int B, int N, int G, const int32_t *table, int max_pages, bool paged,
                   const int32_t *end_col, const int32_t *kv_len, const int32_t *cu, const int32_t *positions,
                   const void *q_weight, const void *k_weight, float eps, const float *inv_freq, int rot,
                   int interleaved, void *q_out, int32_t *status, spec_stream_t stream) {
  if (!q || !k || !v || !q_out || (rot && !inv_freq)) return SPEC_EINVAL;
  RopeParams P;
  const int err = cache_view(P.c, kv, dt, L, planes, H, cols, D, layer, table, max_pages, paged, end_col, kv_len);
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
  const void *outs[] = {kv, q_out, status};
  const size_t out_n[] = {cache_bytes(dt, L, planes, H, cols, D), static_cast<size_t>(T) * qh * elt, b4};
  for (int o = 0; o < 3; ++o) {
    for (int j = 0; j < 11; ++j)
      if (overlaps(outs[o], out_n[o], ins[j], in_n[j])) return SPEC_EINVAL;
    for (int j = o + 1; j < 3; ++j)
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
  return dt == SPEC_BF16 ? launch_rope<__bf16>(P, pairs, grid, threads, s) : launch_rope<float>(P, pairs, grid, threads, s);
}

}  // namespace
}  // namespace specv

using namespace specv;

extern "C" int spec_norm_rope_kv(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                                 int64_t v_stride, void *kv, spec_dtype dt, int L, int B, int H, int C, int D,
                                 int layer, int T, int N, int G, const int32_t *end_col, const int32_t *kv_len,
                                 const int32_t *cu_seqlens, const int32_t *positions, const void *q_weight,
                                 const void *k_weight, float eps, const float *inv_freq, int rot, int interleaved,
                                 void *q_out, int32_t *status, spec_stream_t stream) {
  return norm_rope_call(q, q_stride, k, k_stride, v, v_stride, kv, dt, L, B, H, C, D, layer, T, B, N, G, nullptr, 0,
                        false, end_col, kv_len, cu_seqlens, positions, q_weight, k_weight, eps, inv_freq, rot,
                        interleaved, q_out, status, stream);
}

extern "C" int spec_norm_rope_kv_paged(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                                       const void *v, int64_t v_stride, void *pool, spec_dtype dt, int L, int pages,
                                       int H, int page_size, int D, int layer, int T, int B, int N, int G,
                                       const int32_t *block_table, int max_pages, const int32_t *kv_len,
                                       const int32_t *cu_seqlens, const int32_t *positions, const void *q_weight,
                                       const void *k_weight, float eps, const float *inv_freq, int rot,
                                       int interleaved, void *q_out, int32_t *status, spec_stream_t stream) {
  return norm_rope_call(q, q_stride, k, k_stride, v, v_stride, pool, dt, L, pages, H, page_size, D, layer, T, B, N,
                        G, block_table, max_pages, true, nullptr, kv_len, cu_seqlens, positions, q_weight, k_weight,
                        eps, inv_freq, rot, interleaved, q_out, status, stream);
}
