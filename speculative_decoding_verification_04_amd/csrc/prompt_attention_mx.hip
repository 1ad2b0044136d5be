// The prompt attention calls over caches of 4-bit numbers (gfx950).
#include "prompt_attention.h"

using namespace specv;

extern "C" int spec_prompt_attention_mx(const void *q, int64_t q_stride, const uint8_t *codes, const uint8_t *scales,
                                        spec_dtype dt, int L, int B, int H, int C, int D, int layer, int T, int G,
                                        const int32_t *end_col, const int32_t *kv_len, const int32_t *cu_seqlens,
                                        float scale, void *out, float *lse, int32_t *status, spec_stream_t stream) {
  return prompt_call<true>(q, q_stride, Given{codes, scales, true}, dt, L, B, B, H, C, D, layer, T, G, nullptr, 0,
                           false, end_col, kv_len, cu_seqlens, scale, out, lse, status, stream);
}

extern "C" int spec_prompt_attention_mx_paged(const void *q, int64_t q_stride, const uint8_t *codes,
                                              const uint8_t *scales, spec_dtype dt, int L, int pages, int H,
                                              int page_size, int D, int layer, int B, int T, int G,
                                              const int32_t *block_table, int max_pages, const int32_t *kv_len,
                                              const int32_t *cu_seqlens, float scale, void *out, float *lse,
                                              int32_t *status, spec_stream_t stream) {
  return prompt_call<true>(q, q_stride, Given{codes, scales, true}, dt, L, pages, B, H, page_size, D, layer, T, G,
                           block_table, max_pages, true, nullptr, kv_len, cu_seqlens, scale, out, lse, status, stream);
}
