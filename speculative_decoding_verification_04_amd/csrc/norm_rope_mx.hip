// Norm, rotation and the write into caches of 4-bit numbers (gfx950).
#include "norm_rope.h"

using namespace specv;

extern "C" int spec_norm_rope_kv_mx(const void *q, int64_t q_stride, const void *k, int64_t k_stride, const void *v,
                                    int64_t v_stride, uint8_t *codes, uint8_t *scales, spec_dtype dt, int L, int B,
                                    int H, int C, int D, int layer, int T, int N, int G, const int32_t *end_col,
                                    const int32_t *kv_len, const int32_t *cu_seqlens, const int32_t *positions,
                                    const void *q_weight, const void *k_weight, float eps, const float *inv_freq,
                                    int rot, int interleaved, void *q_out, int32_t *status, spec_stream_t stream) {
  return norm_rope_call<true>(q, q_stride, k, k_stride, v, v_stride, codes, scales, dt, L, B, H, C, D, layer, T, B, N,
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
  return norm_rope_call<true>(q, q_stride, k, k_stride, v, v_stride, codes, scales, dt, L, pages, H, page_size, D,
                              layer, T, B, N, G, block_table, max_pages, true, nullptr, kv_len, cu_seqlens, positions,
                              q_weight, k_weight, eps, inv_freq, rot, interleaved, q_out, status, stream);
}
