// Ragged attention over the paged pool on the CUDA cores, in fp32 throughout.
//
// One pass over a request's keys, 64 at a time, with the running maximum m and
// sum l of an online softmax: for each tile S = Q K^T (scaled to base 2), the
// new maximum m', P = 2^(S - m'), l = l 2^(m - m') + rowsum P, O = O 2^(m -
// m') + P V; at the end O / l and lse = ln 2 (m + log2 l).  The rows of a tile
// are a request's (token, head of the KV group) pairs in that order, so every
// key read serves the whole group.  256 threads as 16 x 16: thread (ty, tx)
// holds rows RPT ty .. RPT ty + RPT - 1 and of each 64 keys tx + 16 j, and of
// each row of O the columns 4 tx + 64 c.
#include "paged.h"

namespace sgqa {
namespace {

constexpr int KT = 64;  // keys per tile
constexpr int NT = 256;

template <int D, int RPT>
struct Cfg {
  static constexpr int R = 16 * RPT;
  static constexpr int QS = D + 4;   // row strides in shared memory (floats): the
  static constexpr int KS = D + 4;   // 16-byte reads of 8 neighbouring rows fall in
  static constexpr int PS = KT + 4;  // different banks
  static constexpr int SMEM = (R * QS + KT * KS + KT * D + R * PS) * 4;
};

// 4 consecutive values as fp32
__device__ __forceinline__ float4 load4(const float* p) {
  return *reinterpret_cast<const float4*>(p);
}
__device__ __forceinline__ float4 load4(const __nv_bfloat16* p) {
  const uint2 u = *reinterpret_cast<const uint2*>(p);
  return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xffff0000u),
                     __uint_as_float(u.y << 16), __uint_as_float(u.y & 0xffff0000u));
}
__device__ __forceinline__ void store4(float* p, float4 v) { *reinterpret_cast<float4*>(p) = v; }
__device__ __forceinline__ void store4(__nv_bfloat16* p, float4 v) {
  *reinterpret_cast<uint2*>(p) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
}

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// grid: (row tiles of all requests at most, KV groups, splits of the keys)
template <typename E, int D, int RPT>
__global__ void __launch_bounds__(NT)
    k_paged_simt(PagedDims pd, PagedAttnArgs a, int nsplit, float* __restrict__ opart,
                 float* __restrict__ lpart) {
  using C = Cfg<D, RPT>;
  constexpr int R = C::R, DC = D / 64;
  extern __shared__ __align__(16) float sm[];
  float* sQ = sm;
  float* sK = sQ + R * C::QS;
  float* sV = sK + KT * C::KS;
  float* sP = sV + KT * D;
  __shared__ int where[3];

  // this CTA's request: row tile blockIdx.x of the batch
  const int tid = threadIdx.x;
  if (tid < 32) {
    int base = 0, found = -1, tile = 0;
    for (int s0 = 0; s0 < pd.N && found < 0; s0 += 32) {
      const int s = s0 + tid;
      int n = 0;
      if (s < pd.N)
        n = (seq_len_of(pd, a.q_start, a.kv_len, s, a.status, blockIdx.x == 0 && blockIdx.y == 0 &&
                        blockIdx.z == 0).ql * pd.G + R - 1) / R;
      int inc = n;
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, inc, o);
        if (tid >= o) inc += x;
      }
      const unsigned in = __ballot_sync(0xffffffffu, base + inc > (int)blockIdx.x);
      if (in) {
        const int l = __ffs(in) - 1;
        found = s0 + l;
        tile = (int)blockIdx.x - base - __shfl_sync(0xffffffffu, inc - n, l);
      }
      base += __shfl_sync(0xffffffffu, inc, 31);
    }
    if (tid == 0) {
      where[0] = found;
      where[1] = tile;
    }
  }
  __syncthreads();
  const int s = where[0];
  if (s < 0) return;
  const SeqLen sl = seq_len_of(pd, a.q_start, a.kv_len, s, nullptr, false);
  const int g = blockIdx.y, sp = blockIdx.z;
  const int r0 = where[1] * R, rows = min(R, sl.ql * pd.G - r0);
  const int tok0 = r0 / pd.G, tok1 = (r0 + rows - 1) / pd.G;  // first and last token
  const int pos0 = sl.kv - sl.ql;                              // position of token 0
  // keys some row of the tile sees, and this split's share of them
  int hi = pd.causal ? max(0, min(sl.kv, pos0 + tok1 + 1)) : sl.kv;
  int lo = pd.window ? max(0, pos0 + tok0 + 1 - pd.window) : 0;
  if (nsplit > 1) {
    const int tiles = hi > lo ? (hi - lo + KT - 1) / KT : 0;
    const int from = (int)((int64_t)tiles * sp / nsplit);
    const int to = (int)((int64_t)tiles * (sp + 1) / nsplit);
    hi = min(hi, lo + to * KT);
    lo += from * KT;
  }

  const E* Q = static_cast<const E*>(a.Q);
  const E* Kp = static_cast<const E*>(a.K);
  const E* Vp = static_cast<const E*>(a.V);
  const float sl2 = pd.scale * 1.4426950408889634f;
  for (int i = tid; i < R * (D / 4); i += NT) {
    const int r = i / (D / 4), c = i % (D / 4) * 4;
    float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
    if (r < rows) {
      const int t = sl.q0 + (r0 + r) / pd.G, h = g * pd.G + (r0 + r) % pd.G;
      x = load4(Q + t * pd.qs + (int64_t)h * D + c);
    }
    *reinterpret_cast<float4*>(sQ + r * C::QS + c) = x;
  }

  const int ty = tid >> 4, tx = tid & 15;
  const float ninf = -__int_as_float(0x7f800000);
  float m[RPT], l[RPT], o[RPT][DC][4];
  int end[RPT], beg[RPT];  // keys row i sees
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    m[i] = ninf;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < DC; ++c)
#pragma unroll
      for (int e = 0; e < 4; ++e) o[i][c][e] = 0.f;
    const int pos = pos0 + (r0 + ty * RPT + i) / pd.G;
    end[i] = pd.causal ? min(hi, pos + 1) : hi;
    beg[i] = pd.window ? max(lo, pos + 1 - pd.window) : lo;
  }

  for (int k0 = lo; k0 < hi; k0 += KT) {
    __syncthreads();  // Q is there; the last tile's V has been read
    for (int i = tid; i < KT * (D / 4); i += NT) {
      const int r = i / (D / 4), c = i % (D / 4) * 4;
      const int key = k0 + r;
      float4 x = make_float4(0.f, 0.f, 0.f, 0.f), y = x;
      if (key < hi) {
        const int page = a.page_table[(int64_t)s * pd.max_pages + key / pd.ps];
        if (page >= 0 && page < pd.n_pages) {
          const int64_t at = (((int64_t)page * pd.Hkv + g) * pd.ps + key % pd.ps) * D + c;
          x = load4(Kp + at);
          y = load4(Vp + at);
        } else if (c == 0) {
          report(a.status, SGQA_ERR_BOUNDS, 302);
        }
      }
      *reinterpret_cast<float4*>(sK + r * C::KS + c) = x;
      *reinterpret_cast<float4*>(sV + r * D + c) = y;
    }
    __syncthreads();
    float p[RPT][4];
#pragma unroll
    for (int i = 0; i < RPT; ++i)
#pragma unroll
      for (int j = 0; j < 4; ++j) p[i][j] = 0.f;
#pragma unroll 4
    for (int c = 0; c < D; c += 4) {
      float4 kk[4];
#pragma unroll
      for (int j = 0; j < 4; ++j)
        kk[j] = *reinterpret_cast<const float4*>(sK + (tx + 16 * j) * C::KS + c);
#pragma unroll
      for (int i = 0; i < RPT; ++i) {
        const float4 q = *reinterpret_cast<const float4*>(sQ + (ty * RPT + i) * C::QS + c);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          p[i][j] = fmaf(q.x, kk[j].x, p[i][j]);
          p[i][j] = fmaf(q.y, kk[j].y, p[i][j]);
          p[i][j] = fmaf(q.z, kk[j].z, p[i][j]);
          p[i][j] = fmaf(q.w, kk[j].w, p[i][j]);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      float mx = ninf;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int key = k0 + tx + 16 * j;
        p[i][j] = key >= beg[i] && key < end[i] ? p[i][j] * sl2 : ninf;
        mx = fmaxf(mx, p[i][j]);
      }
#pragma unroll
      for (int x = 8; x > 0; x >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, x));
      const float mn = fmaxf(m[i], mx);
      const float base = mn == ninf ? 0.f : mn;  // nothing seen so far: all P are 0
      const float f = ex2(m[i] - base);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        p[i][j] = ex2(p[i][j] - base);
        sum += p[i][j];
        sP[(ty * RPT + i) * C::PS + tx + 16 * j] = p[i][j];
      }
      l[i] = l[i] * f + sum;  // this thread's keys; summed over tx at the end
      m[i] = mn;
#pragma unroll
      for (int c = 0; c < DC; ++c)
#pragma unroll
        for (int e = 0; e < 4; ++e) o[i][c][e] *= f;
    }
    __syncwarp();  // a row's P is written and read by the same half warp
#pragma unroll 2
    for (int k = 0; k < KT; k += 4) {
      float4 pr[RPT];
#pragma unroll
      for (int i = 0; i < RPT; ++i)
        pr[i] = *reinterpret_cast<const float4*>(sP + (ty * RPT + i) * C::PS + k);
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
#pragma unroll
        for (int c = 0; c < DC; ++c) {
          const float4 v = *reinterpret_cast<const float4*>(sV + (k + kk) * D + c * 64 + tx * 4);
#pragma unroll
          for (int i = 0; i < RPT; ++i) {
            const float pv = kk == 0 ? pr[i].x : kk == 1 ? pr[i].y : kk == 2 ? pr[i].z : pr[i].w;
            o[i][c][0] = fmaf(pv, v.x, o[i][c][0]);
            o[i][c][1] = fmaf(pv, v.y, o[i][c][1]);
            o[i][c][2] = fmaf(pv, v.z, o[i][c][2]);
            o[i][c][3] = fmaf(pv, v.w, o[i][c][3]);
          }
        }
      }
    }
  }

#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    const int r = ty * RPT + i;
    float lt = l[i];
#pragma unroll
    for (int x = 8; x > 0; x >>= 1) lt += __shfl_xor_sync(0xffffffffu, lt, x);
    if (r >= rows) continue;
    const int64_t t = sl.q0 + (r0 + r) / pd.G;
    const int h = g * pd.G + (r0 + r) % pd.G;
    const float inv = lt > 0.f ? 1.f / lt : 0.f;
    const float lse = lt > 0.f ? (m[i] + log2f(lt)) * 0.69314718055994531f : ninf;
    const int64_t at = t * pd.H + h;
#pragma unroll
    for (int c = 0; c < DC; ++c) {
      const float4 v = make_float4(o[i][c][0] * inv, o[i][c][1] * inv, o[i][c][2] * inv,
                                   o[i][c][3] * inv);
      if (nsplit > 1)
        store4(opart + ((int64_t)sp * pd.T * pd.H + at) * D + c * 64 + tx * 4, v);
      else
        store4(static_cast<E*>(a.O) + at * D + c * 64 + tx * 4, v);
    }
    if (tx == 0) {
      if (nsplit > 1)
        lpart[(int64_t)sp * pd.T * pd.H + at] = lse;
      else
        a.lse[h * (int64_t)pd.T + t] = lse;
    }
  }
}

// Merge of the splits in split order: lse = ln sum_s e^(lse_s), O = sum_s
// e^(lse_s - lse) O_s.  A warp per (token, head); padding rows are left alone.
template <typename E, int D>
__global__ void __launch_bounds__(256)
    k_paged_simt_merge(PagedDims pd, PagedAttnArgs a, int nsplit,
                       const float* __restrict__ opart, const float* __restrict__ lpart) {
  const int64_t row = (int64_t)blockIdx.x * 8 + (threadIdx.x >> 5);
  if (row >= (int64_t)pd.T * pd.H) return;
  const int lane = threadIdx.x & 31;
  const int64_t t = row / pd.H;
  const int h = (int)(row % pd.H);
  // the row belongs to a request that was computed
  bool mine = false;
  for (int s0 = 0; s0 < pd.N && !mine; s0 += 32) {
    bool in = false;
    if (s0 + lane < pd.N) {
      const SeqLen sl = seq_len_of(pd, a.q_start, a.kv_len, s0 + lane, nullptr, false);
      in = t >= sl.q0 && t < sl.q0 + sl.ql;
    }
    mine = __any_sync(0xffffffffu, in);
  }
  if (!mine) return;
  const float ninf = -__int_as_float(0x7f800000);
  const int64_t n = (int64_t)pd.T * pd.H;
  float mx = ninf;
  for (int s = 0; s < nsplit; ++s) mx = fmaxf(mx, lpart[s * n + row]);
  float acc[D / 32], sw = 0.f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) acc[i] = 0.f;
  for (int s = 0; s < nsplit; ++s) {
    const float ls = lpart[s * n + row];
    if (ls == ninf) continue;
    const float w = expf(ls - mx);
    sw += w;
#pragma unroll
    for (int i = 0; i < D / 32; ++i)
      acc[i] = fmaf(w, opart[(s * n + row) * D + lane + 32 * i], acc[i]);
  }
  const float inv = sw > 0.f ? 1.f / sw : 0.f;
#pragma unroll
  for (int i = 0; i < D / 32; ++i) {
    const float v = acc[i] * inv;
    if constexpr (sizeof(E) == 4)
      static_cast<E*>(a.O)[row * D + lane + 32 * i] = v;
    else
      static_cast<E*>(a.O)[row * D + lane + 32 * i] = __float2bfloat16_rn(v);
  }
  if (lane == 0) a.lse[h * (int64_t)pd.T + t] = sw > 0.f ? mx + logf(sw) : ninf;
}

// Rows per tile: 16 when the requests have on average at most that many (one
// token each, a group of up to 16 heads), else 64.
int rows_per_tile(const PagedDims& pd) {
  return (int64_t)pd.T * pd.G <= (int64_t)16 * pd.N ? 16 : 64;
}
// Most row tiles the batch can have.
int64_t most_tiles(const PagedDims& pd) {
  const int R = rows_per_tile(pd);
  return (int64_t)pd.T * pd.G / R + pd.N;
}
// Splits of the keys: enough CTAs for two per SM, at least 256 keys in each.
int splits(const PagedDims& pd) {
  const int64_t ctas = most_tiles(pd) * pd.Hkv;
  const int64_t want = (2 * 152 + ctas - 1) / ctas;
  const int64_t most = pd.cap / 256;
  return (int)(want < most ? (want < 64 ? want : 64) : most < 1 ? 1 : most < 64 ? most : 64);
}

template <typename E, int D, int RPT>
int launch(const PagedDims& pd, const PagedAttnArgs& a, int nsplit, float* opart, float* lpart,
           cudaStream_t st) {
  using C = Cfg<D, RPT>;
  if (cudaFuncSetAttribute(k_paged_simt<E, D, RPT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           C::SMEM) != cudaSuccess)
    return SGQA_ERR_CUDA;
  const int64_t tiles = most_tiles(pd);
  if (tiles > 0x7fffffffll || pd.Hkv > 65535) return SGQA_ERR_UNSUPPORTED;
  log_begin(SGQA_K_PAGED_ATTN, st);
  k_paged_simt<E, D, RPT><<<dim3((unsigned)tiles, pd.Hkv, nsplit), NT, C::SMEM, st>>>(
      pd, a, nsplit, opart, lpart);
  log_end(st);
  if (cudaGetLastError() != cudaSuccess) return SGQA_ERR_CUDA;
  if (nsplit > 1) {
    const int64_t rows = (int64_t)pd.T * pd.H;
    log_begin(SGQA_K_PAGED_ATTN, st);
    k_paged_simt_merge<E, D><<<(unsigned)((rows + 7) / 8), 256, 0, st>>>(pd, a, nsplit, opart,
                                                                        lpart);
    log_end(st);
  }
  return cudaGetLastError() == cudaSuccess ? SGQA_OK : SGQA_ERR_CUDA;
}

template <typename E>
int launch_e(const PagedDims& pd, const PagedAttnArgs& a, int nsplit, float* opart, float* lpart,
             cudaStream_t st) {
  const int R = rows_per_tile(pd);
  if (pd.d == 128)
    return R == 16 ? launch<E, 128, 1>(pd, a, nsplit, opart, lpart, st)
                   : launch<E, 128, 4>(pd, a, nsplit, opart, lpart, st);
  return R == 16 ? launch<E, 64, 1>(pd, a, nsplit, opart, lpart, st)
                 : launch<E, 64, 4>(pd, a, nsplit, opart, lpart, st);
}

}  // namespace

size_t paged_simt_ws_bytes(const PagedDims& pd) {
  if (pd.N == 0 || pd.T == 0) return 0;
  const int n = splits(pd);
  return n > 1 ? (size_t)n * pd.T * pd.H * (pd.d + 1) * 4 : 0;
}

int launch_paged_simt(const PagedDims& pd, const PagedAttnArgs& a, void* ws, cudaStream_t st) {
  const int n = splits(pd);
  float* opart = static_cast<float*>(ws);
  float* lpart = opart + (size_t)n * pd.T * pd.H * pd.d;
  if (pd.dtype == SGQA_BF16) return launch_e<__nv_bfloat16>(pd, a, n, opart, lpart, st);
  return launch_e<float>(pd, a, n, opart, lpart, st);
}

}  // namespace sgqa
