// The tree attention calls over caches of bf16 and float32 (gfx950).
#include "tree_attention.h"

using namespace specv;

extern "C" size_t spec_tree_attention_workspace_bytes(int B, int N, int H, int G, int D, int max_rows,
                                                      spec_dtype dt) {
  return tree_workspace_bytes(B, N, H, G, D, max_rows, dt, false);
}

extern "C" int spec_tree_attention(const void *q, int64_t q_stride, const void *kv, spec_dtype dt, int L, int B, int H,
                                   int C, int D, int layer, int N, int G, const int32_t *end_col,
                                   const int32_t *kv_len, const uint32_t *mask, float scale, void *out, float *lse,
                                   int32_t *status, void *ws, size_t ws_bytes, spec_stream_t stream) {
  return tree_call<false>(q, q_stride, Given{kv, nullptr, false}, dt, L, B, B, H, C, D, layer, N, G, nullptr, 0, false,
                          end_col, kv_len, mask, scale, out, lse, status, ws, ws_bytes, stream);
}

extern "C" int spec_tree_attention_paged(const void *q, int64_t q_stride, const void *pool, spec_dtype dt, int L,
                                         int pages, int H, int page_size, int D, int layer, int B, int N, int G,
                                         const int32_t *block_table, int max_pages, const int32_t *kv_len,
                                         const uint32_t *mask, float scale, void *out, float *lse, int32_t *status,
                                         void *ws, size_t ws_bytes, spec_stream_t stream) {
  return tree_call<false>(q, q_stride, Given{pool, nullptr, false}, dt, L, pages, B, H, page_size, D, layer, N, G,
                          block_table, max_pages, true, nullptr, kv_len, mask, scale, out, lse, status, ws, ws_bytes,
                          stream);
}
