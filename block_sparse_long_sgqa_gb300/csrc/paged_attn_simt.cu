// Ragged attention over the paged pool on the CUDA cores, in fp32 throughout (fp32
// caches).
//
// One pass over an item's keys, 64 at a time, with the running maximum m and sum l of
// an online softmax: for each tile S = Q K^T (scaled to base 2), the new maximum m',
// P = 2^(S - m'), l = l 2^(m - m') + rowsum P, O = O 2^(m - m') + P V; at the end O /
// l and lse = ln 2 (m + log2 l).  An item's rows are (token, head of the group)
// pairs in that order, so every key read serves all of them.  256 threads as 16 x 16:
// thread (ty, tx) holds rows RPT ty .. RPT ty + RPT - 1 and of each 64 keys tx + 16 j,
// and of each row of O the columns 4 tx + 64 c.  Products in the packed f32x2 form: a
// warp's 64 FMAs in 2.0 cycles, against 2 x 1.2 for the scalar one.  What bounds it is
// shared memory: a 4 x 4 tile of S needs 12 wavefronts of reads for 64 cycles of FMAs,
// three quarters of what the SM's four schedulers leave room for (measured: the FMA
// pipe 48 % busy, shared memory 70 %).  An 8 x 4 tile needs half, but leaves 8 warps
// an SM and was slower (2882 us against 2563 on 2656 tokens of 32 heads).
// paged_line.cuh lays the work out over two CTAs per SM; every warp walks it,
// so that a CTA needs no hand-over between its warps.
#include "paged_line.cuh"

namespace sgqa {
namespace {

constexpr int KT = 64;  // keys per tile
constexpr int NT = 256;
constexpr int LPR = NT / KT;  // threads that load a row of a tile

template <int D, int RPT>
struct Cfg {
  static constexpr int R = NT / 16 * RPT;
  static constexpr int PER_SM = 2, GRID = 152 * PER_SM;  // (three of d = 64: registers spill)
  static constexpr int QS = D + 4;   // row strides in shared memory (floats): the
  static constexpr int KS = D + 4;   // 16-byte reads of 8 neighbouring rows fall in
  static constexpr int PS = KT + 4;  // different banks
  static_assert(R * PS <= KT * KS, "P lies over K");
  static constexpr int SMEM = (R * QS + KT * KS + KT * D) * 4;
};

struct SimtArgs : LineArgs {
  const float *Q, *K, *V;
  float *O, *lse;
  float sl2;  // scale * log2(e)
};

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
// 16 bytes global -> shared, zeros unless `on`
__device__ __forceinline__ void copy16(float* dst, const float* src, bool on) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(dst)), "l"(src),
               "r"(on ? 16 : 0)
               : "memory");
}

template <int D, int RPT>
__device__ __noinline__ void simt_piece(const SimtArgs& a, const Piece pc, float* sm) {
  using C = Cfg<D, RPT>;
  constexpr int R = C::R, DC = D / 64;
  float* sQ = sm;
  float* sK = sQ + R * C::QS;
  float* sP = sK;  // over K, once S is done
  float* sV = sK + KT * C::KS;
  const int tid = threadIdx.x, ty = tid >> 4, tx = tid & 15;
  const int h0 = first_head(a, pc.g), nh = heads_of(a, pc.g), rows = pc.ntok * a.heads;
  const int kvh = pc.g / a.head_parts;
  const float ninf = -__int_as_float(0x7f800000);

  __syncthreads();  // the last piece's Q has been read
  for (int i = tid; pc.n > 0 && i < R * (D / 4); i += NT) {
    const int r = i / (D / 4), c = i % (D / 4) * 4;
    const int tok = r / a.heads, h = r - tok * a.heads;
    const bool on = r < rows && h < nh;
    copy16(sQ + r * C::QS + c, a.Q + (on ? (pc.row0 + tok) * a.pd.qs + (int64_t)(h0 + h) * D + c : 0), on);
  }
  float m[RPT], l[RPT];
  uint64_t o[RPT][DC][2];  // columns in pairs
  int end[RPT], beg[RPT];  // keys row i sees
#pragma unroll
  for (int i = 0; i < RPT; ++i) {
    m[i] = ninf;
    l[i] = 0.f;
#pragma unroll
    for (int c = 0; c < DC; ++c) o[i][c][0] = o[i][c][1] = 0ull;
    const int pos = pc.pos0 + (ty * RPT + i) / a.heads;
    end[i] = a.pd.causal ? min(pc.hi, pos + 1) : pc.hi;
    beg[i] = a.pd.window ? max(pc.lo, pos + 1 - a.pd.window) : pc.lo;
  }

  const int kr = tid / LPR;  // the row of the tile that this thread loads a part of
  for (int t = pc.tb; t < pc.tb + pc.n; ++t) {
    const int k0 = t * KT, key = k0 + kr;
    bool on = key >= pc.lo && key < pc.hi;
    int64_t at = 0;
    if (on) {
      const int pi = key / a.pd.ps;
      const int page = a.page_table[(int64_t)pc.s * a.pd.max_pages + pi];
      if (page >= 0 && page < a.pd.n_pages) {
        at = (((int64_t)page * a.pd.Hkv + kvh) * a.pd.ps + (key - pi * a.pd.ps)) * D;
      } else {
        on = false;
        if (tid % LPR == 0) report(a.status, SGQA_ERR_BOUNDS, 302);
      }
    }
    __syncthreads();  // the last tile's P and V have been read
#pragma unroll
    for (int i = 0; i < D / 4 / LPR; ++i) {
      const int c = (tid % LPR + LPR * i) * 4;
      copy16(sK + kr * C::KS + c, a.K + at + c, on);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
#pragma unroll
    for (int i = 0; i < D / 4 / LPR; ++i) {
      const int c = (tid % LPR + LPR * i) * 4;
      copy16(sV + kr * D + c, a.V + at + c, on);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncthreads();
    float p[RPT][4];
    {
      uint64_t q2[RPT][4];  // sums over even and odd columns
#pragma unroll
      for (int i = 0; i < RPT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) q2[i][j] = 0ull;
#pragma unroll 4
      for (int c = 0; c < D; c += 4) {
        ulonglong2 kk[4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
          kk[j] = *reinterpret_cast<const ulonglong2*>(sK + (tx + 16 * j) * C::KS + c);
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
          const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(sQ + (ty * RPT + i) * C::QS + c);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            q2[i][j] = f2_fma(q.x, kk[j].x, q2[i][j]);
            q2[i][j] = f2_fma(q.y, kk[j].y, q2[i][j]);
          }
        }
      }
#pragma unroll
      for (int i = 0; i < RPT; ++i)
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float x, y;
          f2_unpack(q2[i][j], x, y);
          p[i][j] = x + y;
        }
    }
    __syncthreads();  // K has been read: P may be written over it
#pragma unroll
    for (int i = 0; i < RPT; ++i) {
      float mx = ninf;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int k = k0 + tx + 16 * j;
        p[i][j] = k >= beg[i] && k < end[i] ? p[i][j] * a.sl2 : ninf;
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
      const uint64_t ff = f2_pack(f, f);
#pragma unroll
      for (int c = 0; c < DC; ++c) {
        o[i][c][0] = f2_mul(o[i][c][0], ff);
        o[i][c][1] = f2_mul(o[i][c][1], ff);
      }
    }
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();
#pragma unroll 4
    for (int k = 0; k < KT; k += 2) {
      float2 pr[RPT];
#pragma unroll
      for (int i = 0; i < RPT; ++i)
        pr[i] = *reinterpret_cast<const float2*>(sP + (ty * RPT + i) * C::PS + k);
#pragma unroll
      for (int kk = 0; kk < 2; ++kk) {
        ulonglong2 v[DC];
#pragma unroll
        for (int c = 0; c < DC; ++c)
          v[c] = *reinterpret_cast<const ulonglong2*>(sV + (k + kk) * D + c * 64 + tx * 4);
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
          const float x = kk == 0 ? pr[i].x : pr[i].y;
          const uint64_t pv = f2_pack(x, x);
#pragma unroll
          for (int c = 0; c < DC; ++c) {
            o[i][c][0] = f2_fma(pv, v[c].x, o[i][c][0]);
            o[i][c][1] = f2_fma(pv, v[c].y, o[i][c][1]);
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
    const int tok = r / a.heads, h = r - tok * a.heads;
    if (r >= rows || h >= nh) continue;
    const int64_t t = pc.row0 + tok, hq = h0 + h;
    const float inv = lt > 0.f ? 1.f / lt : 0.f;
    const float lse = lt > 0.f ? (m[i] + log2f(lt)) * 0.69314718055994531f : ninf;
    const int64_t part = (int64_t)pc.slot * a.slot_rows + r;
    float* dst = pc.slot >= 0 ? a.opart + part * D : a.O + (t * a.pd.H + hq) * D;
#pragma unroll
    for (int c = 0; c < DC; ++c) {
      float4 v;
      f2_unpack(o[i][c][0], v.x, v.y);
      f2_unpack(o[i][c][1], v.z, v.w);
      *reinterpret_cast<float4*>(dst + c * 64 + tx * 4) =
          make_float4(v.x * inv, v.y * inv, v.z * inv, v.w * inv);
    }
    if (tx == 0) {
      if (pc.slot >= 0)
        a.lpart[part] = lse;
      else
        a.lse[hq * a.pd.T + t] = lse;
    }
  }
}

template <int D, int RPT>
__global__ void __launch_bounds__(NT, (Cfg<D, RPT>::PER_SM))
    k_paged_simt(const __grid_constant__ SimtArgs a) {
  extern __shared__ __align__(16) float sm[];
  __shared__ int64_t warp_sums[NT / 32][4];
  pdl_next();
  pdl_wait();
  {
    const Cut mine = cut_of<KT>(a, threadIdx.x, blockIdx.x == 0);
    line_sums<KT, NT>(a, mine, warp_sums);
  }
  __syncthreads();
  const LineSums sums = add_sums<NT>(a, warp_sums);
  int4 rec;
  walk_line<KT>(a, cut_of<KT>(a, (int)lane_id(), false), sums,
                [&](const Piece& pc) {
                  simt_piece<D, RPT>(a, pc, sm);
                  return true;
                },
                &rec);
  if (threadIdx.x == 0) a.rec[blockIdx.x] = rec;
}

// Rows per item: 16 when the requests have on average at most that many (one token
// each, a group of up to 16 heads), else 64.
int grid_of(const PagedDims& pd) { return pd.d == 128 ? Cfg<128, 4>::GRID : Cfg<64, 4>::GRID; }
int rows_per_item(const PagedDims& pd) {
  return (int64_t)pd.T * pd.G <= (int64_t)16 * pd.N ? 16 : 64;
}

template <int D, int RPT>
int launch(const SimtArgs& a, cudaStream_t st) {
  using C = Cfg<D, RPT>;
  if (cudaFuncSetAttribute(k_paged_simt<D, RPT>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           C::SMEM) != cudaSuccess)
    return SGQA_ERR_CUDA;
  log_begin(SGQA_K_PAGED_ATTN, st);
  const cudaError_t e = launch_pdl(k_paged_simt<D, RPT>, C::GRID, NT, C::SMEM, st, a);
  log_end(st);
  if (e != cudaSuccess) return SGQA_ERR_CUDA;
  return launch_merge<float, D, C::GRID, (C::GRID + 31) / 32 * 32>(a, a.O, a.lse, st);
}

}  // namespace

size_t paged_simt_ws_bytes(const PagedDims& pd) {
  return pd.N == 0 || pd.T == 0 ? 0 : carve_line(grid_of(pd), rows_per_item(pd), pd.d).bytes;
}

int launch_paged_simt(const PagedDims& pd, const PagedAttnArgs& pa, void* ws, cudaStream_t st) {
  const int R = rows_per_item(pd);
  SimtArgs a;
  a.slot_rows = R;
  set_line(a, pd, pa, carve_line(grid_of(pd), R, pd.d), ws);
  a.head_parts = (pd.G + R - 1) / R;
  a.heads = (pd.G + a.head_parts - 1) / a.head_parts;
  a.groups = pd.Hkv * a.head_parts;
  a.tpm = R / a.heads;
  a.tiles_per_item = 1;
  a.tile_rows = 0;
  // 2 to 3 us a tile: four contexts of up to 700 keys 22.7 us (2 and 1: 30.0, 4 and 2: 31.2)
  a.whole = a.part = 1;
  a.uncut = pd.cap <= a.whole * KT;
  a.Q = static_cast<const float*>(pa.Q);
  a.K = static_cast<const float*>(pa.K);
  a.V = static_cast<const float*>(pa.V);
  a.O = static_cast<float*>(pa.O);
  a.lse = pa.lse;
  a.sl2 = pd.scale * 1.4426950408889634f;
  // whole items of a request, over its groups, are counted in 32 bits
  if ((int64_t)a.groups * ((int64_t)pd.T / a.tpm + 1) > 0x7fffffffll) return SGQA_ERR_UNSUPPORTED;
  if (pd.d == 128) return R == 16 ? launch<128, 1>(a, st) : launch<128, 4>(a, st);
  return R == 16 ? launch<64, 1>(a, st) : launch<64, 4>(a, st);
}

}  // namespace sgqa
