// Ragged attention over the paged pool on the CUDA cores, in fp32 throughout (fp32
// caches).
//
// One pass over an item's keys, 64 at a time, with the running maximum m and sum l of
// an online softmax: for each tile S = Q K^T (scaled to base 2), the new maximum m',
// P = 2^(S - m'), l = l 2^(m - m') + rowsum P, O = O 2^(m - m') + P V; at the end O /
// l and lse = ln 2 (m + log2 l).  An item's rows are (token, head of the group)
// pairs in that order, so every key read serves all of them.  256 threads as 16 x 16:
// thread (ty, tx) holds rows 4 ty .. 4 ty + 3 and of each 64 keys tx + 16 j, and of each
// row of O the columns 4 tx + 64 c.  V is copied while S is formed and the next K while
// P V is, so a tile has two barriers and waits for neither; a row of P stays within its
// warp.  Products in the packed f32x2 form: a warp's 64 FMAs in 2.0 cycles, against 2 x
// 1.2 for the scalar one.  What bounds it: the FMA pipe is 60 % busy and shared memory 74
// % (3.1 wavefronts a read) with four warps a scheduler, which registers and shared memory
// both allow and no more: 2656 tokens of 32 heads of 128 on contexts of 500 to 3000 keys
// 2349 us, 38 of the 74 TFLOP/s of the pipe.  8 rows a thread halves the reads but leaves
// two warps a scheduler: 2637 us.  K and V copied at the tile's start: 70 us more.
// paged_line.cuh lays the work out over two CTAs per SM; every warp walks it,
// so that a CTA needs no hand-over between its warps.
#include "paged_line.cuh"

namespace sgqa {
namespace {

constexpr int KT = 64;  // keys per tile
constexpr int NT = 256;
constexpr int LPR = NT / KT;  // threads that load a row of a tile
constexpr int RPT = 4;        // rows of a thread

template <int D>
struct Cfg {
  static constexpr int NTH = NT, KB = KT;
  static constexpr int R = NT / 16 * RPT;
  static constexpr int PER_SM = 2, GRID = 152 * PER_SM;  // (three of d = 64: registers spill)
  static constexpr int QS = D * RPT + 4;  // RPT rows of Q (their reads: 4 banks apart)
  static constexpr int SMEM = (R / RPT * QS + 2 * KT * D + R * KT) * 4;
  static_assert(PER_SM * (SMEM + 1024 + NT) <= 228 * 1024, "two CTAs fit an SM");
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

template <int D>
__device__ __noinline__ void simt_piece(const SimtArgs& a, const Piece pc, float* sm) {
  using C = Cfg<D>;
  constexpr int R = C::R, DC = D / 64;
  float* sQ = sm;
  float* sK = sQ + R / RPT * C::QS;  // rows of 16-byte units, unit u of row r at u ^ (r & 7)
  float* sV = sK + KT * D;
  float* sP = sV + KT * D;           // of an odd ty: keys ^ 16
  // a half warp is 2 ty x 8 tx: its 16-byte reads of an operand are one wavefront
  const int tid = threadIdx.x, ty = tid / 32 * 2 + (tid >> 3 & 1), tx = (tid & 7) + (tid >> 1 & 8);
  const int h0 = first_head(a, pc.g), nh = heads_of(a, pc.g), rows = pc.ntok * a.heads;
  const int kvh = pc.g / a.head_parts;
  const float ninf = -__int_as_float(0x7f800000);

  __syncthreads();  // the last piece's Q has been read
  for (int i = tid; pc.n > 0 && i < R * (D / 4); i += NT) {
    const int r = i / (D / 4), c = i % (D / 4) * 4;
    const int tok = r / a.heads, h = r - tok * a.heads;
    const bool on = r < rows && h < nh;
    copy16(sQ + r / RPT * C::QS + r % RPT * D + c, a.Q + (on ? (pc.row0 + tok) * a.pd.qs + (int64_t)(h0 + h) * D + c : 0), on);
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
  int64_t at = -1;           // and where that row of tile t is
  auto find = [&](int t) {
    const int key = t * KT + kr;
    at = -1;
    if (key < pc.lo || key >= pc.hi) return;
    const int pi = key / a.pd.ps;
    const int page = a.page_table[(int64_t)pc.s * a.pd.max_pages + pi];
    if (page >= 0 && page < a.pd.n_pages)
      at = (((int64_t)page * a.pd.Hkv + kvh) * a.pd.ps + (key - pi * a.pd.ps)) * D;
    else if (tid % LPR == 0)
      report(a.status, SGQA_ERR_BOUNDS, 302);
  };
  auto load = [&](float* dst, const float* src, int swizzle) {
#pragma unroll
    for (int i = 0; i < D / 4 / LPR; ++i) {
      const int u = tid % LPR + LPR * i;
      copy16(dst + kr * D + (u ^ swizzle) * 4, src + (at >= 0 ? at + u * 4 : 0), at >= 0);
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  const float* kRow = sK + tx * D;
  const float* qRow = sQ + ty * C::QS;
  float* pRow = sP + ty * RPT * KT;
  const int psw = (ty & 1) * 16;
  if (pc.n > 0) {
    find(pc.tb);
    load(sK, a.K, kr & 7);
  }
  for (int t = pc.tb; t < pc.tb + pc.n; ++t) {
    const int k0 = t * KT;
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();  // K (and Q) are there, the last tile's V has been read
    load(sV, a.V, 0);
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
          kk[j] = *reinterpret_cast<const ulonglong2*>(kRow + 16 * j * D + (c ^ (tx & 7) * 4));
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
          const ulonglong2 q = *reinterpret_cast<const ulonglong2*>(qRow + i * D + c);
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
    asm volatile("cp.async.wait_group 0;" ::: "memory");
    __syncthreads();  // V is there, K has been read
    if (t + 1 < pc.tb + pc.n) {
      find(t + 1);
      load(sK, a.K, kr & 7);
    }
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
      for (int x : {1, 2, 4, 16}) mx = fmaxf(mx, __shfl_xor_sync(FULL, mx, x));
      const float mn = fmaxf(m[i], mx);
      const float base = mn == ninf ? 0.f : mn;  // nothing seen so far: all P are 0
      const float f = ex2(m[i] - base);
      float sum = 0.f;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        p[i][j] = ex2(p[i][j] - base);
        sum += p[i][j];
        pRow[i * KT + ((tx + 16 * j) ^ psw)] = p[i][j];
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
    __syncwarp();  // a row of P is written and read by one warp
#pragma unroll 8
    for (int k = 0; k < KT; k += 4) {
      float4 pr[RPT];
#pragma unroll
      for (int i = 0; i < RPT; ++i)
        pr[i] = *reinterpret_cast<const float4*>(pRow + i * KT + (k ^ psw));
#pragma unroll
      for (int kk = 0; kk < 4; ++kk) {
        ulonglong2 v[DC];
#pragma unroll
        for (int c = 0; c < DC; ++c)
          v[c] = *reinterpret_cast<const ulonglong2*>(sV + (k + kk) * D + c * 64 + tx * 4);
#pragma unroll
        for (int i = 0; i < RPT; ++i) {
          const float x = kk == 0 ? pr[i].x : kk == 1 ? pr[i].y : kk == 2 ? pr[i].z : pr[i].w;
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
    for (int x : {1, 2, 4, 16}) lt += __shfl_xor_sync(FULL, lt, x);
    const int tok = r / a.heads, h = r - tok * a.heads;
    if (r >= rows || h >= nh) continue;
    const int64_t t = pc.row0 + tok, hq = h0 + h;
    const float inv = lt != 0.f ? 1.f / lt : 0.f;
    const float lse = lt != 0.f ? (m[i] + log2f(lt)) * 0.69314718055994531f : ninf;
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

// Few rows (R = 8 or 16: single tokens of a group of that many heads): the products are
// small and the bytes of K and V count, so the warps share nothing.  Of each tile a warp
// takes 8 keys for itself: it copies their K and V a tile ahead, and keeps a maximum, a
// sum and an output of its own for all R rows; the warps' are joined at the piece's end.
// No barrier inside a piece.  S: a lane sums 4 rows x 4 keys over one of NS parts of the
// columns; the parts are added and dealt out by halves, so that the lane ends with KL
// keys of one row.  O: a lane has 4 columns of every row (d = 64: of every other R / 2).
// What bounds it is reads of shared memory and instructions beside the copies: 16
// requests of 2000 to 4000 keys, 32 on 4 heads of 128, 50 us against 180 with the tiles
// above (188 MB: 28 us); two of 110000 keys 169 us against 729 (0.93 GB: 137 us).  When
// the first took 55: one row and two keys a lane, with no sum over lanes, 70 us; 8 warps
// of d = 128 for 12, 58 us; three stages for two, or P stored in pairs, 2 us more.
template <int D, int R_>
struct Few {
  static constexpr int R = R_, NTH = D == 128 ? 384 : 256, WARPS = NTH / 32, WK = 8, STAGES = 2;
  static constexpr int KB = WARPS * WK;                         // keys of a tile
  static constexpr int KL = WK * R / 32, NS = 128 / R * 4 / WK;
  static constexpr int PER_SM = D == 128 ? 1 : 2, GRID = 152 * PER_SM;
  static constexpr int QS = D + 4, KS = D;  // rows 4 apart: 16 banks apart
  static constexpr int STAGE = WK * (KS + D);                  // floats of a warp's stage
  static constexpr int WARP = STAGES * STAGE + WK * R + 2 * R;  // + P, maxima and sums
  static constexpr int SMEM = (R * QS + WARPS * WARP) * 4;
  static constexpr int RO = D == 128 ? R : R / 2;              // rows of O in a lane
  static_assert(STAGES * STAGE >= R * D, "O lies over the stages at the end");
  static_assert(WARP % 4 == 0 && KL * 32 == WK * R && WK == 8 && (NS == 8 || NS == 4), "");
};

template <int D, int R>
__device__ __noinline__ void few_piece(const SimtArgs& a, const Piece pc, float* sm) {
  using F = Few<D, R>;
  constexpr int KL = F::KL, NS = F::NS;
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
  const int split = lane % NS, rt = lane / NS % (R / 4), kt = lane >> 4;
  const int row = rt * 4 + split / (NS / 4), key0 = kt * 4 + (NS == 8 ? (split & 1) * 2 : 0);
  // over the lanes that have the same row
  auto row_max = [](float x) {
    x = fmaxf(x, __shfl_xor_sync(FULL, x, 16));
    return NS == 8 ? fmaxf(x, __shfl_xor_sync(FULL, x, 1)) : x;
  };
  auto row_sum = [](float x) {
    x += __shfl_xor_sync(FULL, x, 16);
    return NS == 8 ? x + __shfl_xor_sync(FULL, x, 1) : x;
  };
  float* sQ = sm;
  float* mine = sm + R * F::QS + warp * F::WARP;
  float* sP = mine + F::STAGES * F::STAGE;
  float* sM = sP + F::WK * R;
  const int h0 = first_head(a, pc.g), nh = heads_of(a, pc.g), rows = pc.ntok * a.heads;
  const int kvh = pc.g / a.head_parts;
  const float ninf = -__int_as_float(0x7f800000);

  __syncthreads();  // the last piece's outputs have been read
  for (int i = tid; pc.n > 0 && i < R * (D / 4); i += F::NTH) {
    const int r = i / (D / 4), c = i % (D / 4) * 4;
    const int tok = r / a.heads, h = r - tok * a.heads;
    const bool on = r < rows && h < nh;
    copy16(sQ + r * F::QS + c, a.Q + (on ? (pc.row0 + tok) * a.pd.qs + (int64_t)(h0 + h) * D + c : 0), on);
  }
  asm volatile("cp.async.commit_group;" ::: "memory");
  // The warp's keys of a tile are copied row by row, so that an instruction reads whole
  // lines.  Lane i looks up the page of key i (mod WK), a tile before its copy.
  const int first = pc.tb * F::KB + warp * F::WK;
  auto key_of = [&](int t) { return first + t * F::KB + lane % F::WK; };
  auto page_of = [&](int t) {
    const int key = key_of(t);
    return t < pc.n && key >= pc.lo && key < pc.hi
               ? a.page_table[(int64_t)pc.s * a.pd.max_pages + key / a.pd.ps]
               : -1;
  };
  auto load = [&](int t, int page) {
    if (t < pc.n) {
      float* sK = mine + t % F::STAGES * F::STAGE;
      float* sV = sK + F::WK * F::KS;
      const int key = key_of(t);
      int64_t at = -1;
      if (page >= 0 && page < a.pd.n_pages)
        at = ((int64_t)page * a.pd.Hkv + kvh) * a.pd.ps + key % a.pd.ps;
      else if (lane < F::WK && key >= pc.lo && key < pc.hi)
        report(a.status, SGQA_ERR_BOUNDS, 302);
      constexpr int LPK = D / 4;  // lanes of a key
#pragma unroll
      for (int i = 0; i < F::WK; i += 32 / LPK) {
        const int kr = i + lane / LPK, c = lane % LPK * 4;
        const int64_t from = __shfl_sync(FULL, at, kr);
        const bool on = from >= 0;
        copy16(sK + kr * F::KS + c, a.K + (on ? from * D + c : 0), on);
        copy16(sV + kr * D + c, a.V + (on ? from * D + c : 0), on);
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  };
  load(0, page_of(0));
  int page = page_of(1);
  asm volatile("cp.async.wait_group 1;" ::: "memory");
  __syncthreads();  // Q is there

  const int pos = pc.pos0 + row / a.heads;
  const int end = a.pd.causal ? min(pc.hi, pos + 1) : pc.hi;
  const int beg = a.pd.window ? max(pc.lo, pos + 1 - a.pd.window) : pc.lo;
  float m = ninf, l = 0.f;  // of `row`; l: over this lane's keys
  uint64_t o[F::RO][2];
#pragma unroll
  for (int i = 0; i < F::RO; ++i) o[i][0] = o[i][1] = 0ull;
  const int oc = D == 128 ? lane * 4 : lane % 16 * 4;       // columns of O
  const int or0 = D == 128 ? 0 : lane / 16 * F::RO;             // and its first row
  for (int t = 0; t < pc.n; ++t) {
    load(t + 1, page);
    page = page_of(t + 2);
    asm volatile("cp.async.wait_group 1;" ::: "memory");
    __syncwarp();
    const float* sK = mine + t % F::STAGES * F::STAGE;
    const float* sV = sK + F::WK * F::KS;
    float x[16];
    {
      uint64_t s2[16];
#pragma unroll
      for (int e = 0; e < 16; ++e) s2[e] = 0ull;
#pragma unroll
      for (int c = split * 4; c < D; c += NS * 4) {
        ulonglong2 q[4], k[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          q[i] = *reinterpret_cast<const ulonglong2*>(sQ + (rt * 4 + i) * F::QS + c);
          k[i] = *reinterpret_cast<const ulonglong2*>(sK + (kt * 4 + i) * F::KS + c);
        }
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          s2[e] = f2_fma(q[e / 4].x, k[e % 4].x, s2[e]);
          s2[e] = f2_fma(q[e / 4].y, k[e % 4].y, s2[e]);
        }
      }
#pragma unroll
      for (int e = 0; e < 16; ++e) {
        float even, odd;
        f2_unpack(s2[e], even, odd);
        x[e] = even + odd;
      }
    }
#pragma unroll
    for (int n = 8, to = NS / 2; to > 0; n >>= 1, to >>= 1) {
      const bool hi = split & to;
#pragma unroll
      for (int e = 0; e < n; ++e)
        x[e] = (hi ? x[e + n] : x[e]) + __shfl_xor_sync(FULL, hi ? x[e] : x[e + n], to);
    }
    const int k0 = first + t * F::KB + key0;
    float p[KL], mx = ninf;
#pragma unroll
    for (int j = 0; j < KL; ++j) {
      p[j] = k0 + j >= beg && k0 + j < end ? x[j] * a.sl2 : ninf;
      mx = fmaxf(mx, p[j]);
    }
    mx = row_max(mx);
    // the maximum is raised, and O rescaled, only when it is exceeded by 2^8: fp32
    // holds weights up to that with the precision of weights up to 1
    const bool raise = mx > m + 8.f;
    if (__any_sync(FULL, raise)) {
      const float f = raise ? ex2(m - mx) : 1.f;
      l *= f;
      if (raise) m = mx;
#pragma unroll
      for (int i = 0; i < F::RO; ++i) {
        const float fr = __shfl_sync(FULL, f, (or0 + i) * (NS / 4));
        o[i][0] = f2_mul(o[i][0], f2_pack(fr, fr));
        o[i][1] = f2_mul(o[i][1], f2_pack(fr, fr));
      }
    }
    const float base = m == ninf ? 0.f : m;
#pragma unroll
    for (int j = 0; j < KL; ++j) {
      p[j] = ex2(p[j] - base);
      l += p[j];
      sP[(key0 + j) * R + row] = p[j];
    }
    __syncwarp();
#pragma unroll
    for (int k = 0; k < F::WK; ++k) {
      const ulonglong2 v = *reinterpret_cast<const ulonglong2*>(sV + k * D + oc);
#pragma unroll
      for (int i = 0; i < F::RO; i += 4) {
        const float4 w = *reinterpret_cast<const float4*>(sP + k * R + or0 + i);
        const float we[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          o[i + e][0] = f2_fma(f2_pack(we[e], we[e]), v.x, o[i + e][0]);
          o[i + e][1] = f2_fma(f2_pack(we[e], we[e]), v.y, o[i + e][1]);
        }
      }
    }
    __syncwarp();  // P and this stage are written again two steps on
  }

  // ---- the warps' parts joined
  asm volatile("cp.async.wait_group 0;" ::: "memory");
  __syncwarp();
#pragma unroll
  for (int i = 0; i < F::RO; ++i) {
    float4 v;
    f2_unpack(o[i][0], v.x, v.y);
    f2_unpack(o[i][1], v.z, v.w);
    *reinterpret_cast<float4*>(mine + (or0 + i) * D + oc) = v;
  }
  l = row_sum(l);
  if (key0 == 0) {
    sM[row] = m;
    sM[R + row] = l;
  }
  __syncthreads();
  for (int i = tid; i < R * (D / 4); i += F::NTH) {
    const int r = i / (D / 4), c0 = i % (D / 4) * 4;
    const int tok = r / a.heads, h = r - tok * a.heads;
    if (r >= rows || h >= nh) continue;
    const float* warp0 = sm + R * F::QS;
    const float* stats = warp0 + F::STAGES * F::STAGE + F::WK * R + r;
    float mm = ninf, lt = 0.f;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
    for (int w = 0; w < F::WARPS; ++w) mm = fmaxf(mm, stats[w * F::WARP]);
#pragma unroll
    for (int w = 0; w < F::WARPS; ++w) {
      const float mw = stats[w * F::WARP];
      const float f = mw == ninf ? 0.f : ex2(mw - mm);
      const float4 v = *reinterpret_cast<const float4*>(warp0 + w * F::WARP + r * D + c0);
      lt = fmaf(f, stats[w * F::WARP + R], lt);
      acc.x = fmaf(f, v.x, acc.x);
      acc.y = fmaf(f, v.y, acc.y);
      acc.z = fmaf(f, v.z, acc.z);
      acc.w = fmaf(f, v.w, acc.w);
    }
    const int64_t t = pc.row0 + tok, hq = h0 + h;
    const float inv = lt != 0.f ? 1.f / lt : 0.f;
    const int64_t slot_row = (int64_t)pc.slot * a.slot_rows + r;
    float* dst = pc.slot >= 0 ? a.opart + slot_row * D : a.O + (t * a.pd.H + hq) * D;
    *reinterpret_cast<float4*>(dst + c0) = make_float4(acc.x * inv, acc.y * inv, acc.z * inv, acc.w * inv);
    if (c0 == 0) {
      const float lse = lt != 0.f ? (mm + log2f(lt)) * 0.69314718055994531f : ninf;
      (pc.slot >= 0 ? a.lpart[slot_row] : a.lse[hq * a.pd.T + t]) = lse;
    }
  }
}

// The CTA's pieces: every warp walks the line, so that none has to be told.
template <typename C, typename Work>
__device__ __forceinline__ void simt_pieces(const SimtArgs& a, Work work) {
  constexpr int KB = C::KB, N = C::NTH;
  __shared__ int64_t warp_sums[N / 32][4];
  pdl_next();
  pdl_wait();
  {
    const Cut mine = cut_of<KB>(a, threadIdx.x, blockIdx.x == 0);
    line_sums<KB, N>(a, mine, warp_sums);
  }
  __syncthreads();
  const LineSums sums = add_sums<N>(a, warp_sums);
  int4 rec;
  walk_line<KB>(a, cut_of<KB>(a, (int)lane_id(), false), sums,
                [&](const Piece& pc) {
                  work(pc);
                  return true;
                },
                &rec);
  if (threadIdx.x == 0) a.rec[blockIdx.x] = rec;
}

template <int D>
__global__ void __launch_bounds__(NT, (Cfg<D>::PER_SM)) k_paged_simt(const __grid_constant__ SimtArgs a) {
  extern __shared__ __align__(16) float sm[];
  simt_pieces<Cfg<D>>(a, [&](const Piece& pc) { simt_piece<D>(a, pc, sm); });
}
template <int D, int R>
__global__ void __launch_bounds__((Few<D, R>::NTH), (Few<D, R>::PER_SM))
    k_paged_few(const __grid_constant__ SimtArgs a) {
  extern __shared__ __align__(16) float sm[];
  simt_pieces<Few<D, R>>(a, [&](const Piece& pc) { few_piece<D, R>(a, pc, sm); });
}

// Rows per item: 8 or 16 when the requests have on average at most that many and a group
// fits (one token each: 50 and 180 us for 16 requests of 2000 to 4000 keys), else 64.
// The host knows the rows of the buffers, not the lengths, so padding rows count.
int rows_of(const PagedDims& pd) {
  for (int R : {8, 16})
    if (pd.G <= R && (int64_t)pd.T * pd.G <= (int64_t)R * pd.N) return R;
  return 64;
}
int grid_of(const PagedDims& pd) {
  static_assert(Few<128, 8>::GRID == Few<128, 16>::GRID && Few<64, 8>::GRID == Few<64, 16>::GRID, "");
  if (rows_of(pd) <= 16) return pd.d == 128 ? Few<128, 16>::GRID : Few<64, 16>::GRID;
  return pd.d == 128 ? Cfg<128>::GRID : Cfg<64>::GRID;
}

template <typename C, int D>
int launch(void (*kernel)(SimtArgs), SimtArgs& a, cudaStream_t st) {
  a.uncut = a.pd.cap <= a.whole * C::KB;
  if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) !=
      cudaSuccess)
    return SGQA_ERR_CUDA;
  log_begin(SGQA_K_PAGED_ATTN, st);
  const cudaError_t e = launch_pdl(kernel, C::GRID, C::NTH, C::SMEM, st, a);
  log_end(st);
  if (e != cudaSuccess) return SGQA_ERR_CUDA;
  return launch_merge<float, D, C::GRID, (C::GRID + 31) / 32 * 32>(a, a.O, a.lse, st);
}

}  // namespace

size_t paged_simt_ws_bytes(const PagedDims& pd) {
  return pd.N == 0 || pd.T == 0 ? 0 : carve_line(grid_of(pd), rows_of(pd), pd.d).bytes;
}

int launch_paged_simt(const PagedDims& pd, const PagedAttnArgs& pa, void* ws, cudaStream_t st) {
  const int R = rows_of(pd);
  SimtArgs a;
  a.slot_rows = R;
  set_line(a, pd, pa, carve_line(grid_of(pd), R, pd.d), ws);
  a.head_parts = (pd.G + R - 1) / R;
  a.heads = (pd.G + a.head_parts - 1) / a.head_parts;
  a.groups = pd.Hkv * a.head_parts;
  a.tpm = R / a.heads;
  a.tiles_per_item = 1;
  a.tile_rows = 0;
  // (3 chunks of 100 to 401 tokens of 4 heads of 64: 47.1 us, with 2 49.9, with 3 50.5;
  // 16 single tokens over 3000 keys: 51.4 with 2, 52.1 with 1, 53.7 with 3)
  a.over = R == 64 && pd.window == 0 ? 1 : 2;
  // four contexts of up to 700 keys 12.8 us (2: 13.6)
  a.whole = a.part = 1;
  a.Q = static_cast<const float*>(pa.Q);
  a.K = static_cast<const float*>(pa.K);
  a.V = static_cast<const float*>(pa.V);
  a.O = static_cast<float*>(pa.O);
  a.lse = pa.lse;
  a.sl2 = pd.scale * 1.4426950408889634f;
  // whole items of a request, over its groups, are counted in 32 bits
  if ((int64_t)a.groups * ((int64_t)pd.T / a.tpm + 1) > 0x7fffffffll) return SGQA_ERR_UNSUPPORTED;
  if (R == 8)
    return pd.d == 128 ? launch<Few<128, 8>, 128>(k_paged_few<128, 8>, a, st)
                       : launch<Few<64, 8>, 64>(k_paged_few<64, 8>, a, st);
  if (R == 16)
    return pd.d == 128 ? launch<Few<128, 16>, 128>(k_paged_few<128, 16>, a, st)
                       : launch<Few<64, 16>, 64>(k_paged_few<64, 16>, a, st);
  return pd.d == 128 ? launch<Cfg<128>, 128>(k_paged_simt<128>, a, st)
                     : launch<Cfg<64>, 64>(k_paged_simt<64>, a, st);
}

}  // namespace sgqa
