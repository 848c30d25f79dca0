// Accumulated attention weights of the cached keys, and the entry point.
//
// mass[j] += sum over the rows (token, head of the group) that see key j of
// 2^(q . k_j scale log2 e - lse log2 e).  Unlike the attention itself this sums over rows,
// so a key tile stays while the rows that see it go by, and needs no softmax: the
// attention's lse is given.
//
// fp32 on the CUDA cores, 64 keys to a block.  Many rows: the keys in shared memory, the
// rows 64 at a time, each thread a tile of 4 keys by 4 rows; bound by the products and
// the reads of shared memory beside them.  Few rows (single tokens, drafts) would fill an
// eighth of such a tile: there each warp takes a slice of the dimensions of all 64 keys
// straight into registers, two keys a lane, and the rows 8 at a time, and the warps' partial
// products meet in shared memory; bound by the reading of the keys.
#include "paged_mass.h"

namespace sgqa {
namespace {

constexpr int NT = 256;
constexpr int KB = 64, RB = 64;  // keys and rows of a tile
constexpr int FR = 8;            // rows of a turn of the few
// Rows of an item up to which it goes the way of the few.  16 requests over 3000 keys, 4 groups,
// that way and the other: 8 rows 57 and 145 us, 24 rows 90 and 152, 48 rows 140 and 165, 64 rows
// 173 and 172; at head dim 64, 24 rows 68 and 90, 40 rows 94 and 94, 64 rows 132 and 98.  24 is on
// the few's side of both.
constexpr int kFew = 24;

template <int D>
struct Smem {
  static constexpr int LD = D + 4;  // rows start 16 bytes apart in the banks
  float k[KB * LD], q[RB * LD];
  float lse2[RB];
  int pos[RB];  // of the row's token; kNone: the row adds nothing
  float part[16][KB];
};
template <int D>
struct FewSmem {  // in the same memory
  float q[FR * D];
  float dot[NT / 32][FR][KB + 1];  // each warp's slice of the products
  float part[NT / KB][KB];
};

// The sums of an item of few rows: s[key] in sh.part[0][key] when it returns (the block is
// in step).
template <int D>
__device__ __forceinline__ void few_rows(const MassArgs& a, FewSmem<D>& sh, const MassTile& t,
                                         const int32_t* table, int rows) {
  constexpr int SL = D / (NT / 32), U4 = SL / 4;  // dimensions of a warp's slice
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, G = a.pd.G;
  const float* Q = static_cast<const float*>(a.Q);
  const float* K = static_cast<const float*>(a.K);
  float4 k[2][U4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int key = t.k0 + lane + 32 * i;
    const int64_t at = key < t.kv ? entry_of(a, table, t.g, key) : -1;
#pragma unroll
    for (int u = 0; u < U4; ++u)
      k[i][u] = at >= 0 ? reinterpret_cast<const float4*>(K + at * D + warp * SL)[u]
                        : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  }
  const int key = t.k0 + (tid & (KB - 1)), sub = tid / KB;  // of the second step
  float sum = 0.0f;
  for (int r0 = 0; r0 < rows; r0 += FR) {
    const int nr = min(FR, rows - r0);
    for (int x = tid; x < FR * (D / 4); x += NT) {
      const int r = x / (D / 4), u = x % (D / 4);
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      if (r < nr) {
        const int i = (r0 + r) / G, h = (r0 + r) - i * G;
        v = reinterpret_cast<const float4*>(Q + (int64_t)(t.q0 + t.i0 + i) * a.pd.qs +
                                            (int64_t)(t.g * G + h) * D)[u];
      }
      reinterpret_cast<float4*>(sh.q)[x] = v;
    }
    // the rows' statistics, two for each thread's second step
    float lse[FR * KB / NT];
    int pos[FR * KB / NT];
#pragma unroll
    for (int j = 0; j < FR * KB / NT; ++j) {
      const int r = r0 + sub + j * (NT / KB);
      pos[j] = kNone;
      lse[j] = 0.0f;
      if (r < rows) {
        const int i = r / G, h = r - i * G;
        lse[j] = a.lse[(int64_t)(t.g * G + h) * a.pd.T + t.q0 + t.i0 + i] * 1.4426950408889634f;
        if (lse[j] != -__int_as_float(0x7f800000)) pos[j] = t.kv - t.ql + t.i0 + i;
      }
    }
    __syncthreads();
#pragma unroll
    for (int r = 0; r < FR; ++r) {
      float s0 = 0.0f, s1 = 0.0f;
#pragma unroll
      for (int u = 0; u < U4; ++u) {
        const float4 q = *reinterpret_cast<const float4*>(&sh.q[r * D + warp * SL + 4 * u]);
        s0 = fmaf(k[0][u].x, q.x, s0);
        s1 = fmaf(k[1][u].x, q.x, s1);
        s0 = fmaf(k[0][u].y, q.y, s0);
        s1 = fmaf(k[1][u].y, q.y, s1);
        s0 = fmaf(k[0][u].z, q.z, s0);
        s1 = fmaf(k[1][u].z, q.z, s1);
        s0 = fmaf(k[0][u].w, q.w, s0);
        s1 = fmaf(k[1][u].w, q.w, s1);
      }
      sh.dot[warp][r][lane] = s0;
      sh.dot[warp][r][lane + 32] = s1;
    }
    __syncthreads();
#pragma unroll
    for (int j = 0; j < FR * KB / NT; ++j) {
      const int r = sub + j * (NT / KB);
      float s = 0.0f;
#pragma unroll
      for (int w = 0; w < NT / 32; ++w) s += sh.dot[w][r][tid & (KB - 1)];
      const float w = exp2f(fmaf(s, a.sl2, -lse[j]));
      if (sees(a, pos[j], key)) sum += w;
    }
  }
  sh.part[sub][tid & (KB - 1)] = sum;
  __syncthreads();
  if (tid < KB) {
#pragma unroll
    for (int y = 1; y < NT / KB; ++y) sum += sh.part[y][tid];
    sh.part[0][tid] = sum;
  }
}

template <int D>
__global__ void __launch_bounds__(NT, 2) k_mass_simt(const __grid_constant__ MassArgs a) {
  extern __shared__ __align__(16) uint8_t raw[];
  using S = Smem<D>;
  S& sh = *reinterpret_cast<S*>(raw);
  constexpr int LD = S::LD, UN = D / 4;
  const int tid = threadIdx.x, tx = tid & 15, ty = tid >> 4;
  const int G = a.pd.G;
  const float* Q = static_cast<const float*>(a.Q);
  const float* K = static_cast<const float*>(a.K);
  pdl_next();
  pdl_wait();
  TileWalk walk(a, KB);
  MassTile t;
  while (walk.next(a, t)) {
    const int32_t* table = a.page_table + (int64_t)t.s * a.pd.max_pages;
    const int nk = min(KB, t.kv - t.k0);
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    const int rows = (t.i1 - t.i0) * G;
    if (rows > 0 && rows <= kFew) {
      FewSmem<D>& few = *reinterpret_cast<FewSmem<D>*>(raw);
      few_rows<D>(a, few, t, table, rows);
      if (tid < nk) write_entry(a, table, t, t.k0 + tid, few.part[0][tid]);
      __syncthreads();
      continue;
    }
    if (rows > 0) {
      for (int x = tid; x < KB * UN; x += NT) {
        const int r = x / UN, u = x % UN;
        float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
        if (r < nk) {
          const int64_t at = entry_of(a, table, t.g, t.k0 + r);
          if (at >= 0) v = reinterpret_cast<const float4*>(K + at * D)[u];
        }
        *reinterpret_cast<float4*>(&sh.k[r * LD + 4 * u]) = v;
      }
      for (int r0 = 0; r0 < rows; r0 += RB) {
        const int nr = min(RB, rows - r0);
        for (int x = tid; x < RB * UN; x += NT) {
          const int r = x / UN, u = x % UN;
          float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
          if (r < nr) {
            const int i = (r0 + r) / G, h = (r0 + r) - i * G;
            const int64_t tok = t.q0 + t.i0 + i;
            v = reinterpret_cast<const float4*>(Q + tok * a.pd.qs + (int64_t)(t.g * G + h) * D)[u];
          }
          *reinterpret_cast<float4*>(&sh.q[r * LD + 4 * u]) = v;
        }
        if (tid < RB) {
          int pos = kNone;
          float l = 0.0f;
          if (tid < nr) {
            const int i = (r0 + tid) / G, h = (r0 + tid) - i * G;
            l = a.lse[(int64_t)(t.g * G + h) * a.pd.T + t.q0 + t.i0 + i] * 1.4426950408889634f;
            pos = t.kv - t.ql + t.i0 + i;
            if (l == -__int_as_float(0x7f800000)) pos = kNone;  // it saw nothing
          }
          sh.lse2[tid] = l;
          sh.pos[tid] = pos;
        }
        __syncthreads();
        float s[4][4];
#pragma unroll
        for (int i = 0; i < 4; ++i)
#pragma unroll
          for (int j = 0; j < 4; ++j) s[i][j] = 0.0f;
#pragma unroll 4
        for (int u = 0; u < UN; ++u) {
          float4 kv[4], qv[4];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            kv[i] = *reinterpret_cast<const float4*>(&sh.k[(tx + 16 * i) * LD + 4 * u]);
            qv[i] = *reinterpret_cast<const float4*>(&sh.q[(ty + 16 * i) * LD + 4 * u]);
          }
#pragma unroll
          for (int i = 0; i < 4; ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
              s[i][j] = fmaf(kv[i].x, qv[j].x, s[i][j]);
              s[i][j] = fmaf(kv[i].y, qv[j].y, s[i][j]);
              s[i][j] = fmaf(kv[i].z, qv[j].z, s[i][j]);
              s[i][j] = fmaf(kv[i].w, qv[j].w, s[i][j]);
            }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int pos = sh.pos[ty + 16 * j];
          const float l2 = sh.lse2[ty + 16 * j];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const int key = t.k0 + tx + 16 * i;
            const float w = exp2f(fmaf(s[i][j], a.sl2, -l2));
            if (sees(a, pos, key)) acc[i] += w;
          }
        }
        __syncthreads();
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) sh.part[ty][tx + 16 * i] = acc[i];
    __syncthreads();
    if (tid < nk) {
      float sum = 0.0f;
#pragma unroll
      for (int y = 0; y < 16; ++y) sum += sh.part[y][tid];
      write_entry(a, table, t, t.k0 + tid, sum);
    }
    __syncthreads();
  }
}

template <int D>
int launch(const MassArgs& a, cudaStream_t st) {
  constexpr size_t smem = sizeof(Smem<D>);
  static_assert(sizeof(FewSmem<D>) <= smem, "the few use the same memory");
  if (cudaFuncSetAttribute(k_mass_simt<D>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           (int)smem) != cudaSuccess)
    return SGQA_ERR_CUDA;
  log_begin(SGQA_K_MASS, st);
  const cudaError_t e = launch_pdl(k_mass_simt<D>, 152 * 2, NT, smem, st, a);
  log_end(st);
  return e == cudaSuccess ? SGQA_OK : SGQA_ERR_CUDA;
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

}  // namespace
}  // namespace sgqa

using namespace sgqa;

extern "C" {

SGQA_API size_t sgqa_mass_workspace_bytes(const sgqa_paged_params* p) {
  PagedDims pd;
  if (derive_paged(p, &pd) != SGQA_OK) return 0;
  return (pd.dtype == SGQA_BF16 ? mass_tc_ws_bytes(pd) : 0) + 256;
}

SGQA_API int sgqa_paged_mass(const sgqa_paged_params* p, const void* Q, const void* K_pages,
                             const int32_t* page_table, const int32_t* q_start,
                             const int32_t* kv_len, const float* lse, int32_t observe,
                             const float* mass_in, float* mass_out, const int32_t* positions,
                             int32_t* pos_pages, void* ws, size_t ws_bytes, int32_t* status,
                             sgqa_stream_t stream) {
  MassArgs a;
  const int rc = derive_paged(p, &a.pd);
  if (rc != SGQA_OK) return rc;
  if (observe < 0 || (positions == nullptr) != (pos_pages == nullptr)) return SGQA_ERR_INVALID_ARG;
  if (a.pd.N == 0) return SGQA_OK;
  if (K_pages == nullptr || page_table == nullptr || q_start == nullptr || kv_len == nullptr ||
      mass_in == nullptr || mass_out == nullptr ||
      (a.pd.T > 0 && (Q == nullptr || lse == nullptr)))
    return SGQA_ERR_INVALID_ARG;
  if (!aligned16(Q) || !aligned16(K_pages)) return SGQA_ERR_ALIGNMENT;
  // (lse / scale has to be finite, where the lse goes through the product)
  if (a.pd.dtype == SGQA_BF16 && a.pd.scale < 0x1p-64f) return SGQA_ERR_UNSUPPORTED;
  const size_t need = sgqa_mass_workspace_bytes(p);
  if (ws == nullptr || ws_bytes < need) return SGQA_ERR_WORKSPACE;
  // What is written on what is read: every block goes by the lengths for itself, and finds other
  // work than its neighbours if they change under it.
  const size_t elem = (size_t)a.pd.elem, seqs = (size_t)a.pd.N * 4, toks = (size_t)a.pd.T * 4;
  const size_t entries = (size_t)a.pd.n_pages * a.pd.Hkv * a.pd.ps;
  const size_t rows = a.pd.T ? ((size_t)(a.pd.T - 1) * a.pd.qs + (size_t)a.pd.H * a.pd.d) * elem : 0;
  const struct {
    const void* p;
    size_t n;
  } outs[3] = {{mass_out, entries * 4}, {pos_pages, entries * 4}, {ws, need}};
  for (int i = 0; i < 3; ++i) {
    const auto& o = outs[i];
    if (overlap(o.p, o.n, Q, rows) || overlap(o.p, o.n, K_pages, entries * a.pd.d * elem) ||
        overlap(o.p, o.n, page_table, seqs * a.pd.max_pages) ||
        overlap(o.p, o.n, q_start, seqs + 4) || overlap(o.p, o.n, kv_len, seqs) ||
        overlap(o.p, o.n, lse, toks * a.pd.H) || overlap(o.p, o.n, positions, toks) ||
        ((i != 0 || mass_out != mass_in) && overlap(o.p, o.n, mass_in, entries * 4)) ||
        overlap(o.p, o.n, outs[(i + 1) % 3].p, outs[(i + 1) % 3].n))
      return SGQA_ERR_INVALID_ARG;
  }
  // windows and lengths end at cap: the sums of both stay in 32 bits
  if (a.pd.window > a.pd.cap) a.pd.window = a.pd.cap;
  a.Q = Q;
  a.K = K_pages;
  a.page_table = page_table;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.lse = lse;
  a.observe = observe;
  a.mass_in = mass_in;
  a.mass_out = mass_out;
  a.positions = positions;
  a.pos_pages = pos_pages;
  a.status = status;
  a.sl2 = a.pd.scale * 1.4426950408889634f;
  void* base = reinterpret_cast<void*>((reinterpret_cast<uintptr_t>(ws) + 255) &
                                       ~static_cast<uintptr_t>(255));
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (a.pd.dtype == SGQA_BF16) return launch_mass_tc(a, base, st);
  return a.pd.d == 128 ? launch<128>(a, st) : launch<64>(a, st);
}

}  // extern "C"
