// Norm, rotation and the write into caches of 4-bit numbers (gfx950).
//
// Queries as in spec_norm_rope_kv.  A key's code has to be the nearest one to its
// value: next to the border between two codes a rounding of float32 would decide
// otherwise (40 elements of the 21 million of 20.9k tokens of 8 heads of 128), and the
// element would be off by up to half of itself.  So keys are computed in float64,
// their angles too, and leave it as floats that no border separates from them.
//
// Design.  Bound by the vector units as much as by HBM.  One wave takes a token (where
// tokens are few: two or four waves share its heads), with no barrier: it finds the
// token's place and angles, a lane for each pair, and keeps for its elements what turns
// and weighs them, the same for all query heads: a head then costs a product, a sum and
// a scaling an element.  Values go from bf16 to codes in one instruction a pair.
// Measured, heads of 128, 32 over 8: 20.9k tokens (450 MB in and out) 113 us = 4.0 TB/s,
// vector instructions issuing in three quarters of the cycles, in float32 (881 MB) 187 us;
// 512 tokens into pages 10.6 us (as bf16 rows 7.5: here each of a token's two waves finds the
// place and computes the angles); one token 6 us, the latency of three dependent loads and
// the float64 angles.
#include "norm_rope.h"

namespace specv {
namespace {

constexpr int kWaves = kMaxThreads / kWave;
constexpr int kU = 4;          // blocks of query heads in flight

// pos * freq in turns of the circle, less the nearest whole number of them: off by the
// rounding of the last sum, 2^-54 of a turn, at any position.  The product's rounding and
// 1 / (2 pi)'s second half are carried along, and nothing may be contracted: turn -
// rint(turn) as one fma would hold the rounding of turn, which rest adds (so contracted,
// position 2000 was off by 2^-46 of a turn and 2^31 - 1 by 2^-26).
__device__ inline double turns_of(int pos, float freq) {
#pragma clang fp contract(off)
  const double p = pos, f = freq, angle = p * f, low = fma(p, f, -angle);
  const double turn = angle * 0.15915494309189533577;
  const double rest = fma(angle, 0.15915494309189533577, -turn) +
                      (angle * -9.839338337591243e-18 + low * 0.15915494309189533577);
  return (turn - rint(turn)) + rest;
}

// Sine and cosine of t turns of the circle, t within [-1/2, 1/2]: their series on an
// eighth of the circle, within 2^-52.
__device__ inline double2 turn_of(double t) {
  const double quarter = rint(4.0 * t);
  const double x = (t - 0.25 * quarter) * 6.283185307179586477, y = x * x;   // |x| <= pi / 4
  // 1 / k! for odd and even k, alternating
  const double a = x + x * y * (-1.0 / 6 + y * (1.0 / 120 + y * (-1.0 / 5040 + y * (1.0 / 362880 +
                   y * (-1.0 / 39916800 + y * (1.0 / 6227020800.0 + y * (-1.0 / 1307674368000.0)))))));
  const double b = 1.0 + y * (-0.5 + y * (1.0 / 24 + y * (-1.0 / 720 + y * (1.0 / 40320 + y * (-1.0 / 3628800 +
                   y * (1.0 / 479001600 + y * (-1.0 / 87178291200.0 + y * (1.0 / 20922789888000.0))))))));
  const int q = static_cast<int>(quarter) & 3;            // 4 t is within [-2, 2]
  return make_double2(q == 0 ? a : q == 1 ? b : q == 2 ? -a : -b, q == 0 ? b : q == 1 ? -a : q == 2 ? -b : a);
}

// How element e0 + j of a head turns: its pair, its partner, and whether it is the
// pair's first.  Elements that keep theirs (not `in`) are their own partners.
struct Turn {
  int pair, mate;
  bool in, low;
};
template <Pairs PAIRS>
__device__ inline Turn turn_at(int half, int e0, int j) {
  Turn t;
  const int e = e0 + j;
  if constexpr (PAIRS == kNext) {
    t.in = e < 2 * half;
    t.low = !(j & 1);
    t.pair = t.in ? e >> 1 : 0;
    t.mate = t.in ? e ^ 1 : e;
  } else {
    const int of = PAIRS == kChunksApart ? e0 : e;        // whole chunks turn alike
    t.in = of < 2 * half;
    t.low = of < half;
    t.pair = t.in ? (t.low ? of : of - half) + (e - of) : 0;
    t.mate = t.in ? (t.low ? of + half : of - half) + (e - of) : e;
  }
  return t;
}

// A lane's elements of a head and their partners.  x: as loaded; src: the head.
template <typename T, Pairs PAIRS>
__device__ inline void with_mates(u32x4 x, const T *src, int half, int e0, bool active, float (&a)[Vec<T>::n],
                                  float (&m)[Vec<T>::n]) {
  constexpr int kN = Vec<T>::n;
  widen<T>(x, a);
  if constexpr (PAIRS == kChunksApart) {
    u32x4 o;
#pragma unroll
    for (int j = 0; j < 4; ++j) o[j] = __shfl_xor(x[j], half / kN);
    widen<T>(o, m);
  } else if constexpr (PAIRS == kNext) {
#pragma unroll
    for (int j = 0; j < kN; ++j) m[j] = a[j ^ 1];
  } else {
#pragma unroll
    for (int j = 0; j < kN; ++j) m[j] = active ? static_cast<float>(src[turn_at<PAIRS>(half, e0, j).mate]) : 0.0f;
  }
}

// The weights of a lane's elements and of their partners; 1 without any.
template <typename T, Pairs PAIRS>
__device__ inline void weights_of(const void *weights, int half, int e0, bool active, float (&own)[Vec<T>::n],
                                  float (&mate)[Vec<T>::n]) {
  constexpr int kN = Vec<T>::n;
  if (weights) {                                          // of the call, not of the lane
    const T *w = static_cast<const T *>(weights);
    u32x4 x = {0, 0, 0, 0}, y = {0, 0, 0, 0};
    if (active) __builtin_memcpy(&x, w + e0, 16);
    widen<T>(x, own);
    if constexpr (PAIRS == kChunksApart) {
      if (active) __builtin_memcpy(&y, w + turn_at<PAIRS>(half, e0, 0).mate, 16);
      widen<T>(y, mate);
    } else if constexpr (PAIRS == kNext) {
#pragma unroll
      for (int j = 0; j < kN; ++j) mate[j] = own[j ^ 1];
    } else {
#pragma unroll
      for (int j = 0; j < kN; ++j) mate[j] = active ? static_cast<float>(w[turn_at<PAIRS>(half, e0, j).mate]) : 0.0f;
    }
  } else {
#pragma unroll
    for (int j = 0; j < kN; ++j) own[j] = mate[j] = 1.0f;
  }
}

// A lane's elements of a query after norm and rotation: r a c + r m s, with c and s the
// cosine and the signed sine times the weights.  The norm comes first: an element times
// its weight may leave float32 where the result does not.
template <typename T, Pairs PAIRS>
__device__ inline void query_turned(const RopeParams &P, u32x4 x, const T *src, int e0, bool active,
                                    const float (&c)[Vec<T>::n], const float (&s)[Vec<T>::n], float (&y)[Vec<T>::n]) {
  constexpr int kN = Vec<T>::n;
  float a[kN], m[kN];
  with_mates<T, PAIRS>(x, src, P.half, e0, active, a, m);
  if (P.q_weight) {
    float squares = 0.0f;
#pragma unroll
    for (int j = 0; j < kN; ++j) squares = fmaf(a[j], a[j], squares);
    const float of = group_sum(squares, P.lanes) / static_cast<float>(P.c.D) + P.eps;
    const bool low = of < 0x1p-100f;                      // the instruction takes what is no normal number for 0
    const float r = __builtin_amdgcn_rsqf(low ? of * 0x1p64f : of) * (low ? 0x1p32f : 1.0f);
#pragma unroll
    for (int j = 0; j < kN; ++j) {
      a[j] *= r;
      m[j] *= r;
    }
  }
#pragma unroll
  for (int j = 0; j < kN; ++j) {
    const float z = a[j] * c[j];
    y[j] = turn_at<PAIRS>(P.half, e0, j).in ? fmaf(m[j], s[j], z) : z;
  }
}

// A key's, from float64, as floats on the right side of every border.  w: the weights
// of the elements and of their partners; angles: the token's sines and cosines.
template <typename T, Pairs PAIRS>
__device__ inline void key_turned(const RopeParams &P, u32x4 x, const T *src, int e0, bool active,
                                  const float (&w)[2][Vec<T>::n], const double2 *angles, float (&y)[Vec<T>::n]) {
  constexpr int kN = Vec<T>::n;
  float a[kN], m[kN];
  with_mates<T, PAIRS>(x, src, P.half, e0, active, a, m);
  double r = 1.0;
  if (P.k_weight) {
    double squares = 0.0;
#pragma unroll
    for (int j = 0; j < kN; ++j) squares = fma(static_cast<double>(a[j]), static_cast<double>(a[j]), squares);
    const double of = group_sum(squares, P.lanes) / P.c.D + P.eps;
    // the instruction gives 24 bits and each step twice as many (of 0 and infinity it is what it is)
    r = __builtin_amdgcn_rsq(of);
    if (of > 0.0 && of < INFINITY) {
      r = r * fma(-0.5 * of * r, r, 1.5);
      r = r * fma(-0.5 * of * r, r, 1.5);
    }
  }
#pragma unroll
  for (int j = 0; j < kN; ++j) {
    const Turn t = turn_at<PAIRS>(P.half, e0, j);
    const double2 angle = angles[t.pair];
    // in float64: the fraction of a product of bf16 would fit float32, its exponent need not (2^100 times
    // 2^30, while the normed key is 2^30); 20.9k tokens of 32 + 16 heads of 128 take 115 us so, 110 otherwise
    const double p = static_cast<double>(a[j]) * w[0][j], o = static_cast<double>(m[j]) * w[1][j];
    y[j] = mx_sided((t.in ? fma(o, t.low ? -angle.x : angle.x, p * angle.y) : p) * r);
  }
}

// Of a lane's elements as loaded: the largest, as bits without sign, and the codes.
template <typename T>
__device__ inline uint32_t raw_top(u32x4 x) {
  if constexpr (sizeof(T) == 2) {
    typedef uint16_t u16x2 __attribute__((ext_vector_type(2)));
    const auto size = [&](int j) { return __builtin_bit_cast(u16x2, x[j] & 0x7fff7fffu); };
    const u16x2 y = __builtin_elementwise_max(__builtin_elementwise_max(size(0), size(1)),
                                              __builtin_elementwise_max(size(2), size(3)));
    return static_cast<uint32_t>(max(y[0], y[1])) << 16;
  } else {
    return max(max(x[0] & 0x7fffffffu, x[1] & 0x7fffffffu), max(x[2] & 0x7fffffffu, x[3] & 0x7fffffffu));
  }
}
template <typename T>
__device__ inline uint32_t raw_codes(u32x4 x, int byte) {
  if constexpr (sizeof(T) == 2) {
    return mx_codes_bf16({x[0], x[1], x[2], x[3]}, byte);
  } else {
    float y[4];
    widen<T>(x, y);
    return mx_codes<4>(y, byte);
  }
}

// The largest of the 32 elements of a lane's block (as bits without sign), which
// neighbouring lanes hold.
template <typename T>
__device__ inline uint32_t block_top(uint32_t top) {
  top = max(top, dpp_move<kDppQuadXor1>(top, top));
  top = max(top, dpp_move<kDppQuadXor2>(top, top));
  if constexpr (Vec<T>::n == 4) top = max(top, dpp_move<kDppRowHalfMirror>(top, top));
  return top;
}

// A lane's codes and its block's scale into a row of 4-bit numbers; `row`: the row's
// number in the layer's K or V.  Two blocks' scales are written as one.
template <typename T>
__device__ inline void put_mx(uint32_t codes, int byte, char *to, char *scales, long long row, int D, int e0, bool store) {
  uint32_t both = e0 & kMxBlock ? byte << 8 : byte;
  both |= Vec<T>::n == 8 ? dpp_move<kDppRowHalfMirror>(both, both) : dpp_move<kDppRowMirror>(both, both);
  if (!store) return;
  to += row * (D / 2) + e0 / 2;
  if constexpr (Vec<T>::n == 8) *reinterpret_cast<uint32_t *>(to) = codes;
  else *reinterpret_cast<uint16_t *>(to) = static_cast<uint16_t>(codes);
  if (e0 % (2 * kMxBlock) == 0)
    *reinterpret_cast<uint16_t *>(scales + row * (D / kMxBlock) + e0 / kMxBlock) = static_cast<uint16_t>(both);
}

// ONCE: the rows are too many to be found in a cache: read non-temporally.
template <typename T, Pairs PAIRS, bool ONCE>
__global__ __launch_bounds__(kMaxThreads, 4) void norm_rope_mx_kernel(RopeParams P, int split, int groups) {
  constexpr int kN = Vec<T>::n;
  __shared__ double2 all_angles[kWaves][SPEC_ATTN_MAX_D / 2];   // sines and cosines, a wave's own
  const int lane = threadIdx.x & (kWave - 1), wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  if (blockIdx.x >= static_cast<unsigned>(groups)) {
    write_status(P, (blockIdx.x - groups) * kWaves + wave);
    return;
  }
  const int part = wave % split;                          // of the token's waves
  const int t = blockIdx.x * (kWaves / split) + wave / split;
  if (t >= P.T) return;                                   // no barrier follows
  double2 *const angles = all_angles[wave];
  const int D = P.c.D, half = P.half, H = P.c.H;
  const int lph = P.lanes, g = lane / lph, e0 = (lane & (lph - 1)) * kN, each = kWave / lph;   // each: heads at once
  const bool active = e0 < D;
  // the lane's heads; the last of a token's waves take the first values, since the first take the first keys
  const int first = part * each + g, first_v = (split - 1 - part) * each + g, step = split * each;
  const char *const q = P.q + t * P.q_stride + e0 * sizeof(T), *const k = P.k + t * P.k_stride + e0 * sizeof(T);
  const char *const v = P.v + t * P.v_stride + e0 * sizeof(T);
  const long long head = static_cast<long long>(D) * sizeof(T);
  auto load = [&](const char *rows, int h, int count) __attribute__((always_inline)) {
    u32x4 x = {0, 0, 0, 0};
    const u32x4 *from = reinterpret_cast<const u32x4 *>(rows + h * head);
    if (h < count && active) x = ONCE ? __builtin_nontemporal_load(from) : *from;
    return x;
  };
  // What waits for nothing, the small things first: loads come back in order.
  const Early early = early_of(P, t);
  const int given = *(P.positions ? P.positions + t : P.c.kv_len);
  const float freq = *(half ? P.inv_freq + min(lane, half - 1) : reinterpret_cast<const float *>(P.c.kv_len));
  u32x4 flight[kU];
#pragma unroll
  for (int u = 0; u < kU; ++u) flight[u] = load(q, first + u * step, P.Hq);
  u32x4 key = load(k, first, H), value = load(v, first_v, H);
  float c[kN], s[kN], w[2][kN];                           // of queries; of keys
  weights_of<T, PAIRS>(P.q_weight, half, e0, active, c, s);
  weights_of<T, PAIRS>(P.k_weight, half, e0, active, w[0], w[1]);
  const Place place = place_of(P, t, early);
  if (place.at == kNoSequence) return;
  const int pos = P.positions ? given : place.row;
  for (int i = lane; i < half; i += kWave) {
    angles[i] = turn_of(turns_of(pos, i < kWave ? freq : P.inv_freq[i]));
  }
  __builtin_amdgcn_wave_barrier();                        // the wave's own LDS, in order
#pragma unroll
  for (int j = 0; j < kN; ++j) {
    const Turn z = turn_at<PAIRS>(half, e0, j);
    const double2 angle = angles[z.pair];
    c[j] *= z.in ? static_cast<float>(angle.y) : 1.0f;
    s[j] *= static_cast<float>(z.low ? -angle.x : angle.x);
  }
  char *const out = P.q_out + (static_cast<long long>(t) * P.Hq * D + e0) * sizeof(T);
  for (int h0 = first; h0 - g < P.Hq; h0 += kU * step) {
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int h = h0 + u * step;
      if (h - g >= P.Hq) break;
      const u32x4 x = flight[u];
      flight[u] = load(q, h + kU * step, P.Hq);
      float y[kN];
      query_turned<T, PAIRS>(P, x, reinterpret_cast<const T *>(P.q + t * P.q_stride + min(h, P.Hq - 1) * head), e0, active, c, s, y);
      if (h < P.Hq && active) *reinterpret_cast<u32x4 *>(out + h * head) = narrow<T>(y);
    }
  }
  const bool held = active && place.at >= 0;
#pragma unroll 1
  for (int h = first; h - g < H; h += step) {
    const u32x4 x = key;
    key = load(k, h + step, H);
    float y[kN];
    key_turned<T, PAIRS>(P, x, reinterpret_cast<const T *>(P.k + t * P.k_stride + min(h, H - 1) * head), e0, active, w, angles, y);
    uint32_t top = 0;
#pragma unroll
    for (int j = 0; j < kN; ++j) top = max(top, __float_as_uint(y[j]) & 0x7fffffffu);
    const int byte = mx_scale_byte(block_top<T>(top));
    put_mx<T>(mx_codes<kN>(y, byte), byte, P.c.k, P.c.ks, place.at + static_cast<long long>(h) * P.c.cols, D, e0, held && h < H);
  }
#pragma unroll 1
  for (int h = first_v; h - g < H; h += step) {
    const u32x4 x = value;
    value = load(v, h + step, H);
    const int byte = mx_scale_byte(block_top<T>(raw_top<T>(x)));
    put_mx<T>(raw_codes<T>(x, byte), byte, P.c.v, P.c.vs, place.at + static_cast<long long>(h) * P.c.cols, D, e0, held && h < H);
  }
}

template <typename T, Pairs PAIRS>
void launch_pairs(const RopeParams &P, int split, int groups, unsigned grid, hipStream_t s) {
  // What a call reads and writes beyond the Infinity Cache (256 MB) is not found again:
  // 20.9k tokens of 32 + 16 heads of 128 (451 MB) take 119 us so and 125 without.
  const long long bytes = static_cast<long long>(P.T) * (2 * P.Hq + 2 * P.c.H) * P.c.D * sizeof(T);
  if (bytes > (256ll << 20))
    hipLaunchKernelGGL((norm_rope_mx_kernel<T, PAIRS, true>), dim3(grid), dim3(kMaxThreads), 0, s, P, split, groups);
  else
    hipLaunchKernelGGL((norm_rope_mx_kernel<T, PAIRS, false>), dim3(grid), dim3(kMaxThreads), 0, s, P, split, groups);
}

template <typename T>
int launch_rope_mx(const RopeParams &P, Pairs pairs, int split, int groups, unsigned grid, hipStream_t s) {
  switch (pairs) {
    case kNext: launch_pairs<T, kNext>(P, split, groups, grid, s); break;
    case kChunksApart: launch_pairs<T, kChunksApart>(P, split, groups, grid, s); break;
    default: launch_pairs<T, kAny>(P, split, groups, grid, s); break;
  }
  return launch_status();
}

int norm_rope_mx_call(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v, int64_t v_stride,
                      uint8_t *codes, uint8_t *scales, spec_dtype dt, int L, int planes, int H, int cols, int D,
                      int layer, int T, int B, int N, int G, const int32_t *table, int max_pages, bool paged,
                      const int32_t *end_col, const int32_t *kv_len, const int32_t *cu, const int32_t *positions,
                      const void *q_weight, const void *k_weight, float eps, const float *inv_freq, int rot,
                      int interleaved, void *q_out, int32_t *status, spec_stream_t stream) {
  RopeParams P;
  RopeShape shape;
  const int err = rope_params(P, shape, true, q, q_stride, k, k_stride, v, v_stride, codes, scales, dt, L, planes, H,
                              cols, D, layer, T, B, N, G, table, max_pages, paged, end_col, kv_len, cu, positions,
                              q_weight, k_weight, eps, inv_freq, rot, interleaved, q_out, status);
  if (err) return err;
  // Few tokens leave waves to spare.  bf16, 32 heads of 128 over 8, captured calls with one /
  // two / four waves a token: 1 token 9.8 / 7.3 / 6.4 us; 256: 11.5 / 8.6 / 7.7; 512: 12.0 / 9.4
  // / 9.5; 1024: 12.8 / 11.3 / 12.6; 2048: 16.5 / 17.8 / 21.3; 4096: 26.0 / 30.3 / 37.3.  Fewer
  // heads leave less to share, which the rule does not look at (2 heads over 2: 256 tokens
  // 7.0 / 6.7 / 6.8; 1024: 7.7 / 8.3 / 10.2; 2048: 9.4 / 10.9 / 15.7), and in float32 it is
  // within 1 us of the best for 32 heads over 8 but for 256 tokens (19.7 / 18.0 / 20.5) and
  // loses up to 8 us for 2 over 2 there (11.0 / 13.5 / 18.9).
  const int split = T <= 256 ? 4 : T <= 2048 ? 2 : 1, per = kWaves / split, groups = (T + per - 1) / per;
  const long long grid = rope_grid(groups, B, status, kWaves);
  if (!launchable(grid, kMaxThreads)) return SPEC_EINVAL;
  (void)hipGetLastError();
  const hipStream_t s = static_cast<hipStream_t>(stream);
  return dt == SPEC_BF16 ? launch_rope_mx<__bf16>(P, shape.pairs, split, groups, static_cast<unsigned>(grid), s)
                         : launch_rope_mx<float>(P, shape.pairs, split, groups, static_cast<unsigned>(grid), s);
}

}  // namespace
}  // namespace specv

using namespace specv;

extern "C" int spec_norm_rope_kv_mx(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                                 int64_t v_stride, uint8_t *codes, uint8_t *scales, spec_dtype dt, int L, int B,
                                 int H, int C, int D, int layer, int T, int N, int G, const int32_t *end_col,
                                 const int32_t *kv_len, const int32_t *cu_seqlens, const int32_t *positions,
                                 const void *q_weight, const void *k_weight, float eps, const float *inv_freq,
                                 int rot, int interleaved, void *q_out, int32_t *status, spec_stream_t stream) {
  return norm_rope_mx_call(q, q_stride, k, k_stride, v, v_stride, codes, scales, dt, L, B, H, C, D, layer, T, B, N,
                           G, nullptr, 0, false, end_col, kv_len, cu_seqlens, positions, q_weight, k_weight, eps,
                           inv_freq, rot, interleaved, q_out, status, stream);
}

extern "C" int spec_norm_rope_kv_mx_paged(const void *q, int64_t q_stride, const void *k, int64_t k_stride,
                                       const void *v, int64_t v_stride, uint8_t *codes, uint8_t *scales,
                                       spec_dtype dt, int L, int pages, int H, int page_size, int D, int layer,
                                       int T, int B, int N, int G, const int32_t *block_table, int max_pages,
                                       const int32_t *kv_len, const int32_t *cu_seqlens, const int32_t *positions,
                                       const void *q_weight, const void *k_weight, float eps,
                                       const float *inv_freq, int rot, int interleaved, void *q_out,
                                       int32_t *status, spec_stream_t stream) {
  return norm_rope_mx_call(q, q_stride, k, k_stride, v, v_stride, codes, scales, dt, L, pages, H, page_size, D,
                           layer, T, B, N, G, block_table, max_pages, true, nullptr, kv_len, cu_seqlens, positions,
                           q_weight, k_weight, eps, inv_freq, rot, interleaved, q_out, status, stream);
}
