// KV caches of 4-bit numbers (gfx950): the format, its view and its conversions.
//
// 32 elements of a row share a scale, a power of two held as its exponent + 127
// in a byte; an element is a code of four bits (E2M1: a sign, and one of 0, 0.5,
// 1, 1.5, 2, 3, 4, 6), the even element of a pair in the low half of a byte.  The
// value is the code's times the scale: exact in bf16 and in float32.  A scale byte
// above 252 (6 * 2^126 would pass the largest finite number) stands for NaN in
// all 32 elements.
//
// Writing: with a the largest magnitude of the 32, the scale 2^e is the one with
// which a, rounded to two bits, becomes 4 or 6: e = floor(log2 a) - 2, and one more
// from 1.75 * 2^floor(log2 a) on.  So no element is off by more than half a step
// of the codes around it (with the floor alone, elements between 7 and 8 units
// would be cut to 6).  e is kept within -125 .. 125, where scales, codes' values and
// products stay normal numbers.  Elements go to the nearest code, ties to the even
// one.  A block with an infinity or a NaN gets the scale byte 255 and codes of 0.
#pragma once

#include "cache_view.h"

namespace specv {

constexpr int kMxBlock = 32, kMxNan = 255, kMxTop = 252;   // elements to a scale; the bytes for NaN and the largest scale

typedef float f32x2 __attribute__((ext_vector_type(2)));

// Host checks of a cache of 4-bit numbers: as cache_view(); D a multiple of 64.
inline int mx_view(CacheView &c, const void *codes, const void *scales, int L, int planes, int H, int cols, int D,
                   int layer, const int32_t *table, int max_pages, bool paged, const int32_t *end_col,
                   const int32_t *kv_len) {
  if (!codes || !scales) return SPEC_EINVAL;
  const int err = cache_shape(c, L, planes, H, cols, D, layer, table, max_pages, paged, end_col, kv_len);
  if (err) return err;
  if (D % 64 || !aligned(codes, 16) || !aligned(scales, 16)) return SPEC_EINVAL;
  const long long rows = static_cast<long long>(planes) * H * cols;            // one layer's K
  c.k = static_cast<char *>(const_cast<void *>(codes)) + 2 * rows * (D / 2) * layer;
  c.v = c.k + rows * (D / 2);
  c.ks = static_cast<char *>(const_cast<void *>(scales)) + 2 * rows * (D / kMxBlock) * layer;
  c.vs = c.ks + rows * (D / kMxBlock);
  return SPEC_OK;
}

inline size_t mx_rows(int L, int planes, int H, int cols) { return static_cast<size_t>(L) * 2 * planes * H * cols; }

// The scale as a float; byte 0 (2^-127, no normal number) counts as 1.
__device__ inline float mx_scale(int byte) { return __uint_as_float(static_cast<uint32_t>(max(byte, 1)) << 23); }

// The values of eight codes.
template <typename T>
__device__ inline void mx_widen(uint32_t codes, float scale, T (&x)[8]) {
  if constexpr (sizeof(T) == 2) {
    typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
    const bf16x2 a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 0);
    const bf16x2 b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 1);
    const bf16x2 c = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 2);
    const bf16x2 d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(codes, scale, 3);
    x[0] = a[0], x[1] = a[1], x[2] = b[0], x[3] = b[1], x[4] = c[0], x[5] = c[1], x[6] = d[0], x[7] = d[1];
  } else {
    const f32x2 a = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 0);
    const f32x2 b = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 1);
    const f32x2 c = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 2);
    const f32x2 d = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(codes, scale, 3);
    x[0] = a[0], x[1] = a[1], x[2] = b[0], x[3] = b[1], x[4] = c[0], x[5] = c[1], x[6] = d[0], x[7] = d[1];
  }
}

// The scale byte of a block whose largest magnitude has the float32 bits `top`
// (sign clear).  A quarter of the leading bit added to it carries into the
// exponent from 1.75 on.
__device__ inline int mx_scale_byte(uint32_t top) {
  if (top >= 0x7f800000u) return kMxNan;
  return min(max(static_cast<int>((top + 0x200000u) >> 23) - 2, 2), kMxTop);
}

// Codes of N (4 or 8) elements, for a scale byte of mx_scale_byte().
template <int N>
__device__ inline uint32_t mx_codes(const float (&x)[N], int byte) {
  if (byte == kMxNan) return 0u;
  const float scale = mx_scale(byte), most = 6.0f * scale;
  float y[N];
#pragma unroll
  for (int j = 0; j < N; ++j) y[j] = fminf(fmaxf(x[j], -most), most);
  uint32_t c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, y[0], y[1], scale, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[2], y[3], scale, 1);
  if constexpr (N == 8) {
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[4], y[5], scale, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, y[6], y[7], scale, 3);
  }
  return c;
}

// A double as the float on its way to a code: rounded so that no border between
// codes or scales is reached or passed that the double itself does not reach or
// pass.  Borders are floats with few bits, so their last bit is 0: where the
// nearest float is not the double itself and its last bit is 0, the neighbour on
// the double's side is taken.
__device__ inline float mx_sided(double x) {
  const float f = static_cast<float>(x);
  const double off = x - static_cast<double>(f);
  const uint32_t u = __float_as_uint(f);
  if (off == 0.0 || (u & 1u) || (u & 0x7fffffffu) >= 0x7f800000u) return f;
  if ((u & 0x7fffffffu) == 0u) return __uint_as_float((x < 0.0 ? 0x80000000u : 0u) | 1u);   // below the smallest float
  return __uint_as_float((off > 0.0) == (f > 0.0f) ? u + 1u : u - 1u);
}

}  // namespace specv
