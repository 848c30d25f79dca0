// Definitions shared by the paged serving operators (page tables, K/V append,
// ragged attention over the paged pool).
#pragma once

#include "common.cuh"
#include "internal.h"

namespace sgqa {

// A validated sgqa_paged_params in kernel-argument form.
struct PagedDims {
  int N, T;            // requests; token rows
  int H, Hkv, G, d;
  int ps, n_pages, max_pages;
  int cap;             // max_pages * ps: most positions of a request
  int dtype, elem;
  int causal, window;
  float scale;
  int64_t qs, kvs;     // row strides of Q and of K, V (elements)
};

int derive_paged(const sgqa_paged_params* p, PagedDims* pd);

int launch_page_plan(const PagedDims& pd, const int32_t* q_len, const int32_t* kv_len,
                     const int32_t* free_pages, const int32_t* n_free, int32_t* page_table,
                     int32_t* q_start, int64_t* slot_map, int32_t* positions,
                     int32_t* n_free_out, int32_t* status, cudaStream_t st);
int launch_page_release(const PagedDims& pd, const int32_t* kv_len, const int32_t* keep_len,
                        const int32_t* page_table, int32_t* free_pages, const int32_t* n_free,
                        int32_t* n_free_out, int32_t* status, cudaStream_t st);
int launch_paged_append(const PagedDims& pd, const void* K, const void* V,
                        const int64_t* slot_map, void* Kp, void* Vp, int32_t* status,
                        cudaStream_t st);

struct PagedAttnArgs {
  const void *Q, *K, *V;  // rows of stride qs; the pool
  const int32_t *page_table, *q_start, *kv_len;
  void* O;
  float* lse;
  int32_t* status;
};

// CUDA-core attention
size_t paged_simt_ws_bytes(const PagedDims& pd);
int launch_paged_simt(const PagedDims& pd, const PagedAttnArgs& a, void* ws, cudaStream_t st);

// tensor-core attention (bf16)
size_t paged_tc_ws_bytes(const PagedDims& pd);
int launch_paged_tc(const PagedDims& pd, const PagedAttnArgs& a, void* ws, cudaStream_t st);

// Whether two buffers share a byte (a NULL or empty one shares none).
inline bool overlap(const void* a, size_t na, const void* b, size_t nb) {
  const uintptr_t x = reinterpret_cast<uintptr_t>(a), y = reinterpret_cast<uintptr_t>(b);
  return a != nullptr && b != nullptr && na > 0 && nb > 0 && (x < y ? y - x < na : x - y < nb);
}

// Launches in a row: each kernel lets the next one be scheduled from its start on
// (pdl_next) and, before it touches memory that another kernel may still read or write,
// waits until the one before it is complete (pdl_wait).  The next launch's latency and
// set-up then lie beside the end of this one's work.  No pointer of such a kernel is
// __restrict__: what it points to may be written until the wait returns, and the
// qualifier would allow loads through the non-coherent path, or ahead of the wait,
// whose memory clobber need not order them.
__device__ __forceinline__ void pdl_next() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
__device__ __forceinline__ void pdl_wait() { asm volatile("griddepcontrol.wait;" ::: "memory"); }

template <typename... P, typename... A>
inline cudaError_t launch_pdl(void (*kernel)(P...), int64_t grid, int threads, size_t smem,
                              cudaStream_t st, const A&... args) {
  cudaLaunchAttribute attr;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)grid);
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kernel, args...);
}

// Lengths of request s as the kernels use them: rows [q0, q0 + ql) and kv
// cached positions; ql = 0 and a report where they do not fit the call.
struct SeqLen {
  int q0, ql, kv;
};
__device__ __forceinline__ SeqLen seq_len_of(const PagedDims& pd, const int32_t* q_start,
                                             const int32_t* kv_len, int s, int32_t* status,
                                             bool tell) {
  SeqLen r;
  const int a = q_start[s], b = q_start[s + 1];
  r.kv = kv_len[s];
  r.q0 = a;
  r.ql = b - a;
  if (a < 0 || b < a || b > pd.T || r.kv < 0 || r.kv > pd.cap) {
    if (tell) report(status, SGQA_ERR_BOUNDS, 301);
    r.q0 = r.ql = r.kv = 0;
  }
  return r;
}

}  // namespace sgqa
