// New K and V rows into the paged pool through the slot map: a copy, bound by
// memory.  131072 rows of 8 heads of 128 in bf16: 160 us, 6.7 TB/s read and written
// together, the rate of a plain copy; 256 rows: 2.1 us in a row of such calls.
#include "paged.h"

namespace sgqa {
namespace {

// One warp per token: its K row and its V row, Hkv * d values each, move as
// 16-byte units (2^log_up of them per head), kBatch of each row a lane at a time
// with their loads before their stores.
constexpr int kBatch = 4;
__global__ void __launch_bounds__(256)
    k_paged_append(PagedDims pd, const uint4* K, const uint4* V, const int64_t* slot_map,
                   uint4* Kp, uint4* Vp, int log_up, int64_t row_units, int32_t* status) {
  pdl_next();
  pdl_wait();
  const int64_t t = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (t >= pd.T) return;
  const int lane = threadIdx.x & 31;
  const int64_t slot = slot_map[t];
  if (slot < 0) return;
  if (slot >= (int64_t)pd.n_pages * pd.ps) {
    if (lane == 0) report(status, SGQA_ERR_BOUNDS, 321);
    return;
  }
  const uint32_t page = (uint32_t)slot / (uint32_t)pd.ps, off = (uint32_t)slot % (uint32_t)pd.ps;
  const int units = pd.Hkv << log_up;
  const uint4* k = K + t * row_units;
  const uint4* v = V + t * row_units;
  const int64_t base = (int64_t)page * pd.Hkv * pd.ps + off;  // row of head 0
  for (int u0 = lane; u0 < units; u0 += 32 * kBatch) {
    uint4 x[kBatch], y[kBatch];
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int u = u0 + 32 * b;
      if (u >= units) break;
      x[b] = k[u];
      y[b] = v[u];
    }
#pragma unroll
    for (int b = 0; b < kBatch; ++b) {
      const int u = u0 + 32 * b;
      if (u >= units) break;
      const int g = u >> log_up, c = u & ((1 << log_up) - 1);
      const int64_t at = ((base + (int64_t)g * pd.ps) << log_up) + c;
      Kp[at] = x[b];
      Vp[at] = y[b];
    }
  }
}

}  // namespace

int launch_paged_append(const PagedDims& pd, const void* K, const void* V,
                        const int64_t* slot_map, void* Kp, void* Vp, int32_t* status,
                        cudaStream_t st) {
  const int up = pd.d * pd.elem / 16;  // 8, 16 or 32
  const int log_up = up == 8 ? 3 : up == 16 ? 4 : 5;
  log_begin(SGQA_K_APPEND, st);
  const cudaError_t e = launch_pdl(
      k_paged_append, ((int64_t)pd.T + 7) / 8, 256, 0, st, pd, static_cast<const uint4*>(K),
      static_cast<const uint4*>(V), slot_map, static_cast<uint4*>(Kp), static_cast<uint4*>(Vp),
      log_up, pd.kvs * pd.elem / 16, status);
  log_end(st);
  return e == cudaSuccess ? SGQA_OK : SGQA_ERR_CUDA;
}

}  // namespace sgqa
