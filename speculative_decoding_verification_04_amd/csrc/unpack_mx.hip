// Rows of a cache of 4-bit numbers as the values that they stand for (gfx950).
//
// value = code * 2^e, e the exponent of the 32 elements' scale: exact in bf16 and
// in float32.
//
// Design.  Bound by the writes: 16 or 32 bits an element out for 4.25 in.  A
// workgroup takes some tokens, finds where their rows lie (a wave for each token),
// and then its lanes take eight elements each.
// Measured: 20.9k tokens of 8 heads of 128 in bf16 (109 MB) 25 us = 4.4 TB/s; 512 tokens
// from pages 5 us and one token 2.3 us, latency.
#include "mx.h"
#include "token_rows.h"

namespace specv {
namespace {

constexpr int kThreads = 256, kWaves = kThreads / kWave;
constexpr int kU = 4;        // items in flight per lane
constexpr int kMaxTokens = 64;

typedef uint32_t u32x4 __attribute__((ext_vector_type(4)));

struct UnpackParams : TokenRows {
  char *k_out, *v_out;       // [T][H][D]
  int per, groups;           // tokens of a workgroup; workgroups that have tokens
};

template <typename T>
__global__ __launch_bounds__(kThreads) void unpack_kernel(UnpackParams P) {
  __shared__ long long at[kMaxTokens];                   // each token's Place::at
  const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
  if (blockIdx.x >= static_cast<unsigned>(P.groups)) {
    write_status(P, (blockIdx.x - P.groups) * kWaves + wave);
    return;
  }
  const int first = blockIdx.x * P.per, count = min(P.per, P.T - first);
  for (int i = wave; i < count; i += kWaves) {
    const Place p = place_of(P, first + i, early_of(P, first + i));
    if ((threadIdx.x & (kWave - 1)) == 0) at[i] = p.at;
  }
  __syncthreads();
  const int D = P.c.D, row_items = D / 8, half = P.c.H * row_items, items = 2 * half;   // of a token
  for (int x0 = threadIdx.x; x0 < count * items; x0 += kU * kThreads) {
    uint32_t codes[kU];
    int byte[kU];
    char *to[kU];
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      const int x = x0 + u * kThreads;
      to[u] = nullptr;
      codes[u] = 0;
      byte[u] = 1;
      if (x >= count * items) continue;
      const int i = x / items, y = x - i * items;
      const bool is_v = y >= half;
      const int z = is_v ? y - half : y, h = z / row_items, d = (z - h * row_items) * 8;
      const long long r0 = at[i];
      if (r0 == kNoSequence) continue;
      to[u] = (is_v ? P.v_out : P.k_out) + (static_cast<long long>(first + i) * half * 8 + z * 8) * sizeof(T);
      if (r0 < 0) continue;
      const long long row = r0 + static_cast<long long>(h) * P.c.cols;
      codes[u] = *reinterpret_cast<const uint32_t *>((is_v ? P.c.v : P.c.k) + row * (D / 2) + d / 2);
      byte[u] = static_cast<uint8_t>((is_v ? P.c.vs : P.c.ks)[row * (D / kMxBlock) + d / kMxBlock]);
    }
#pragma unroll
    for (int u = 0; u < kU; ++u) {
      if (!to[u]) continue;
      T y[8];
      mx_widen<T>(codes[u], mx_scale(byte[u]), y);
      if (byte[u] > kMxTop) {
#pragma unroll
        for (int j = 0; j < 8; ++j) y[j] = static_cast<T>(NAN);
      }
      u32x4 z[sizeof(T) / 2];
      __builtin_memcpy(z, y, sizeof(z));
#pragma unroll
      for (unsigned j = 0; j < sizeof(T) / 2; ++j) reinterpret_cast<u32x4 *>(to[u])[j] = z[j];
    }
  }
}

int unpack_call(const uint8_t *codes, const uint8_t *scales, spec_dtype dt, int L, int planes, int H, int cols, int D,
                int layer, int T, int B, int N, const int32_t *table, int max_pages, bool paged,
                const int32_t *end_col, const int32_t *kv_len, const int32_t *cu, void *k_out, void *v_out,
                int32_t *status, spec_stream_t stream) {
  if (!k_out || !v_out || (dt != SPEC_F32 && dt != SPEC_BF16)) return SPEC_EINVAL;
  UnpackParams P;
  const int err = mx_view(P.c, codes, scales, L, planes, H, cols, D, layer, table, max_pages, paged, end_col, kv_len);
  if (err) return err;
  if (T < 1 || B < 1 || (!paged && planes != B)) return SPEC_EINVAL;
  if (cu ? N != 0 : N < 1 || static_cast<long long>(B) * N != T) return SPEC_EINVAL;
  if (D > SPEC_ATTN_MAX_D) return SPEC_ECAPACITY;
  // a workgroup's items, up to 64 tokens of 2 H D / 8, stay far below 2^31
  if (H >= INT32_MAX / (16 * SPEC_ATTN_MAX_D) || static_cast<long long>(T) + B >= INT32_MAX) return SPEC_EINVAL;
  if (!aligned(k_out, 16) || !aligned(v_out, 16) || !aligned(status, 4)) return SPEC_EINVAL;
  const int items = 2 * H * (D / 8);
  P.per = 1;
  while (P.per < kMaxTokens && P.per * items < kU * kThreads) P.per *= 2;
  P.groups = (T + P.per - 1) / P.per;
  const long long grid = P.groups + (status ? (static_cast<long long>(B) + kWaves - 1) / kWaves : 0);
  if (!launchable(grid, kThreads)) return SPEC_EINVAL;
  const size_t b4 = static_cast<size_t>(B) * 4, rows = mx_rows(L, planes, H, cols);
  const size_t out = static_cast<size_t>(T) * H * D * (dt == SPEC_BF16 ? 2 : 4);
  const void *ins[] = {codes, scales, table, end_col, kv_len, cu};
  const size_t in_n[] = {rows * (D / 2), rows * (D / kMxBlock), paged ? b4 * max_pages : 0, paged ? 0u : 4u, b4, b4 + 4};
  const void *outs[] = {k_out, v_out, status};
  const size_t out_n[] = {out, out, b4};
  for (int o = 0; o < 3; ++o) {
    for (int j = 0; j < 6; ++j)
      if (overlaps(outs[o], out_n[o], ins[j], in_n[j])) return SPEC_EINVAL;
    for (int j = o + 1; j < 3; ++j)
      if (overlaps(outs[o], out_n[o], outs[j], out_n[j])) return SPEC_EINVAL;
  }
  P.T = T;
  P.B = B;
  P.N = N;
  P.cu = cu;
  P.status = status;
  P.k_out = static_cast<char *>(k_out);
  P.v_out = static_cast<char *>(v_out);
  (void)hipGetLastError();
  const hipStream_t s = static_cast<hipStream_t>(stream);
  if (dt == SPEC_BF16)
    hipLaunchKernelGGL((unpack_kernel<__bf16>), dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, s, P);
  else
    hipLaunchKernelGGL((unpack_kernel<float>), dim3(static_cast<unsigned>(grid)), dim3(kThreads), 0, s, P);
  return launch_status();
}

}  // namespace
}  // namespace specv

using namespace specv;

extern "C" int spec_unpack_kv_mx(const uint8_t *codes, const uint8_t *scales, spec_dtype dt, int L, int B, int H, int C,
                                 int D, int layer, int T, int N, const int32_t *end_col, const int32_t *kv_len,
                                 const int32_t *cu_seqlens, void *k_out, void *v_out, int32_t *status,
                                 spec_stream_t stream) {
  return unpack_call(codes, scales, dt, L, B, H, C, D, layer, T, B, N, nullptr, 0, false, end_col, kv_len, cu_seqlens,
                     k_out, v_out, status, stream);
}

extern "C" int spec_unpack_kv_mx_paged(const uint8_t *codes, const uint8_t *scales, spec_dtype dt, int L, int pages,
                                       int H, int page_size, int D, int layer, int T, int B, int N,
                                       const int32_t *block_table, int max_pages, const int32_t *kv_len,
                                       const int32_t *cu_seqlens, void *k_out, void *v_out, int32_t *status,
                                       spec_stream_t stream) {
  return unpack_call(codes, scales, dt, L, pages, H, page_size, D, layer, T, B, N, block_table, max_pages, true,
                     nullptr, kv_len, cu_seqlens, k_out, v_out, status, stream);
}
