// Entry points of the paged serving operators: validation and dispatch.
// Declared and documented in include/sgqa.h.
#include <cmath>

#include "paged.h"

namespace sgqa {

int derive_paged(const sgqa_paged_params* p, PagedDims* pd) {
  if (p == nullptr || pd == nullptr) return SGQA_ERR_INVALID_ARG;
  if (p->n_seqs < 0 || p->max_tokens < 0 || p->n_pages < 1 || p->max_pages < 1 ||
      p->page_size < 1)
    return SGQA_ERR_INVALID_ARG;
  if (p->n_kv_heads < 1 || p->n_q_heads < 1 || p->n_q_heads % p->n_kv_heads)
    return SGQA_ERR_INVALID_ARG;
  if (p->dtype < 0 || p->dtype > 1 || p->causal < 0 || p->causal > 1 || p->window < 0 ||
      (p->window > 0 && !p->causal))
    return SGQA_ERR_INVALID_ARG;
  if (!(p->softmax_scale >= 0.0f) || !std::isfinite(p->softmax_scale * 1.4426950408889634f))
    return SGQA_ERR_INVALID_ARG;
  const int64_t hd = (int64_t)p->n_q_heads * p->head_dim;
  const int64_t kd = (int64_t)p->n_kv_heads * p->head_dim;
  if (p->head_dim != 64 && p->head_dim != 128) return SGQA_ERR_UNSUPPORTED;
  if ((p->q_stride != 0 && p->q_stride < hd) || (p->kv_stride != 0 && p->kv_stride < kd))
    return SGQA_ERR_INVALID_ARG;
  if (p->page_size % 8 || p->n_q_heads / p->n_kv_heads > 128 || p->max_tokens > (1 << 24) ||
      (int64_t)p->max_pages * p->page_size > (int64_t(1) << 25) ||
      (int64_t)p->max_tokens * p->n_q_heads > 0x7fffffffll ||
      (double)p->n_pages * p->n_kv_heads * p->page_size > 2147483647.0)
    return SGQA_ERR_UNSUPPORTED;
  pd->N = p->n_seqs;
  pd->T = p->max_tokens;
  pd->H = p->n_q_heads;
  pd->Hkv = p->n_kv_heads;
  pd->G = p->n_q_heads / p->n_kv_heads;
  pd->d = p->head_dim;
  pd->ps = p->page_size;
  pd->n_pages = p->n_pages;
  pd->max_pages = p->max_pages;
  pd->cap = p->max_pages * p->page_size;
  pd->dtype = p->dtype;
  pd->elem = p->dtype == SGQA_BF16 ? 2 : 4;
  pd->causal = p->causal;
  pd->window = p->window;
  pd->scale = p->softmax_scale > 0.0f ? p->softmax_scale : 1.0f / std::sqrt((float)p->head_dim);
  pd->qs = p->q_stride ? p->q_stride : hd;
  pd->kvs = p->kv_stride ? p->kv_stride : kd;
  if (pd->qs * pd->elem % 16 || pd->kvs * pd->elem % 16) return SGQA_ERR_ALIGNMENT;
  return SGQA_OK;
}

namespace {
inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
}  // namespace
}  // namespace sgqa

using namespace sgqa;

extern "C" {

SGQA_API int sgqa_page_plan(const sgqa_paged_params* p, const int32_t* q_len,
                            const int32_t* kv_len, const int32_t* free_pages,
                            const int32_t* n_free, int32_t* page_table, int32_t* q_start,
                            int64_t* slot_map, int32_t* positions, int32_t* n_free_out,
                            int32_t* status, sgqa_stream_t stream) {
  PagedDims pd;
  const int rc = derive_paged(p, &pd);
  if (rc != SGQA_OK) return rc;
  if ((pd.N > 0 && (q_len == nullptr || kv_len == nullptr || page_table == nullptr)) ||
      free_pages == nullptr || n_free == nullptr || q_start == nullptr ||
      n_free_out == nullptr || n_free_out == n_free ||
      (pd.T > 0 && (slot_map == nullptr || positions == nullptr)))
    return SGQA_ERR_INVALID_ARG;
  return launch_page_plan(pd, q_len, kv_len, free_pages, n_free, page_table, q_start, slot_map,
                          positions, n_free_out, status, reinterpret_cast<cudaStream_t>(stream));
}

SGQA_API int sgqa_page_release(const sgqa_paged_params* p, const int32_t* kv_len,
                               const int32_t* keep_len, const int32_t* page_table,
                               int32_t* free_pages, const int32_t* n_free, int32_t* n_free_out,
                               int32_t* status, sgqa_stream_t stream) {
  PagedDims pd;
  const int rc = derive_paged(p, &pd);
  if (rc != SGQA_OK) return rc;
  if ((pd.N > 0 && (kv_len == nullptr || keep_len == nullptr || page_table == nullptr)) ||
      free_pages == nullptr || n_free == nullptr || n_free_out == nullptr || n_free_out == n_free)
    return SGQA_ERR_INVALID_ARG;
  return launch_page_release(pd, kv_len, keep_len, page_table, free_pages, n_free, n_free_out,
                             status, reinterpret_cast<cudaStream_t>(stream));
}

SGQA_API int sgqa_paged_append(const sgqa_paged_params* p, const void* K, const void* V,
                               const int64_t* slot_map, void* K_pages, void* V_pages,
                               int32_t* status, sgqa_stream_t stream) {
  PagedDims pd;
  const int rc = derive_paged(p, &pd);
  if (rc != SGQA_OK) return rc;
  if (K_pages == nullptr || V_pages == nullptr ||
      (pd.T > 0 && (K == nullptr || V == nullptr || slot_map == nullptr)))
    return SGQA_ERR_INVALID_ARG;
  if (!aligned16(K) || !aligned16(V) || !aligned16(K_pages) || !aligned16(V_pages))
    return SGQA_ERR_ALIGNMENT;
  if (pd.T == 0) return SGQA_OK;
  return launch_paged_append(pd, K, V, slot_map, K_pages, V_pages, status,
                             reinterpret_cast<cudaStream_t>(stream));
}

SGQA_API size_t sgqa_paged_workspace_bytes(const sgqa_paged_params* p) {
  PagedDims pd;
  if (derive_paged(p, &pd) != SGQA_OK) return 0;
  return (pd.dtype == SGQA_BF16 ? paged_tc_ws_bytes(pd) : paged_simt_ws_bytes(pd)) +
         256;  // slack to align the caller's base
}

SGQA_API int sgqa_paged_attn(const sgqa_paged_params* p, const void* Q, const void* K_pages,
                             const void* V_pages, const int32_t* page_table,
                             const int32_t* q_start, const int32_t* kv_len, void* O, float* lse,
                             void* ws, size_t ws_bytes, int32_t* status, sgqa_stream_t stream) {
  PagedDims pd;
  const int rc = derive_paged(p, &pd);
  if (rc != SGQA_OK) return rc;
  if (pd.N == 0 || pd.T == 0) return SGQA_OK;
  if (Q == nullptr || K_pages == nullptr || V_pages == nullptr || page_table == nullptr ||
      q_start == nullptr || kv_len == nullptr || O == nullptr || lse == nullptr)
    return SGQA_ERR_INVALID_ARG;
  if (!aligned16(Q) || !aligned16(K_pages) || !aligned16(V_pages) || !aligned16(O))
    return SGQA_ERR_ALIGNMENT;
  if (ws == nullptr || ws_bytes < sgqa_paged_workspace_bytes(p)) return SGQA_ERR_WORKSPACE;
  void* base = reinterpret_cast<void*>((reinterpret_cast<uintptr_t>(ws) + 255) &
                                       ~static_cast<uintptr_t>(255));
  const PagedAttnArgs a{Q, K_pages, V_pages, page_table, q_start, kv_len, O, lse, status};
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return pd.dtype == SGQA_BF16 ? launch_paged_tc(pd, a, base, st)
                               : launch_paged_simt(pd, a, base, st);
}

}  // extern "C"
