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

inline size_t mx_rows(int L, int planes, int H, int cols) { return static_cast<size_t>(L) * 2 * planes * H * cols; }

// Host checks of a cache of 4-bit numbers: as cache_view(); D a multiple of 64; codes and
// scales apart.
inline int mx_view(CacheView &c, const void *codes, const void *scales, int L, int planes, int H, int cols, int D,
                   int layer, const int32_t *table, int max_pages, bool paged, const int32_t *end_col,
                   const int32_t *kv_len) {
  if (!codes || !scales) return SPEC_EINVAL;
  const int err = cache_shape(c, L, planes, H, cols, D, layer, table, max_pages, paged, end_col, kv_len);
  if (err) return err;
  if (D % 64 || !aligned(codes, 16) || !aligned(scales, 16)) return SPEC_EINVAL;
  const size_t all = mx_rows(L, planes, H, cols);
  if (overlaps(codes, all * (D / 2), scales, all * (D / kMxBlock))) return SPEC_EINVAL;
  const long long rows = static_cast<long long>(planes) * H * cols;            // one layer's K
  c.k = static_cast<char *>(const_cast<void *>(codes)) + 2 * rows * (D / 2) * layer;
  c.v = c.k + rows * (D / 2);
  c.ks = static_cast<char *>(const_cast<void *>(scales)) + 2 * rows * (D / kMxBlock) * layer;
  c.vs = c.ks + rows * (D / kMxBlock);
  return SPEC_OK;
}

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

// Codes of N (4 or 8) elements, for a scale byte of mx_scale_byte().  The instruction
// rounds to the nearest code, ties to the even one, and gives 6 for more.
template <int N>
__device__ inline uint32_t mx_codes(const float (&x)[N], int byte) {
  if (byte == kMxNan) return 0u;
  const float scale = mx_scale(byte);
  uint32_t c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(0u, x[0], x[1], scale, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[2], x[3], scale, 1);
  if constexpr (N == 8) {
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[4], x[5], scale, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, x[6], x[7], scale, 3);
  }
  return c;
}

// The same of eight elements of bf16, in pairs.
__device__ inline uint32_t mx_codes_bf16(const uint32_t (&x)[4], int byte) {
  typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
  if (byte == kMxNan) return 0u;
  const float scale = mx_scale(byte);
  uint32_t c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(0u, __builtin_bit_cast(bf16x2, x[0]), scale, 0);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, x[1]), scale, 1);
  c = __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, x[2]), scale, 2);
  return __builtin_amdgcn_cvt_scalef32_pk_fp4_bf16(c, __builtin_bit_cast(bf16x2, x[3]), scale, 3);
}

// A double as the float on its way to a code: cut to 20 bits of its fraction, with the
// last of them set where anything was cut off, so that it is on the double's side of
// every border (borders have few bits).  What float32 would round to infinity, from
// 2^128 - 2^103 on: infinity; between half and all of the smallest normal number, three
// quarters of it, and 0 below.
__device__ inline float mx_sided(double x) {
  const uint64_t u = __builtin_bit_cast(uint64_t, x);
  const uint32_t high = static_cast<uint32_t>(u >> 32), size = (high & 0x7fffffffu) | (static_cast<uint32_t>(u) ? 1u : 0u);
  const uint32_t base = 896u << 20;                       // what exponents differ by
  uint32_t bits = (size - base) << 3;
  if (size < base + (1u << 20)) bits = size > base ? 0x00600000u : 0u;
  if (!(fabs(x) < 0x1.ffffffp127)) bits = size > 0x7ff00000u ? 0x7fc00000u : 0x7f800000u;
  return __uint_as_float(bits | (high & 0x80000000u));
}

}  // namespace specv
