// Verification of drafted tokens against the target's probabilities.
//
// A request's drafts are looked at together, one lane each (32 at a time): accept while
// u D(x) < P(x), a comparison of exact products.  What is left is one draw from w =
// max(P - D, 0) of the row where a draft was turned down, or from P of the last row: the
// first token whose cumulative weight exceeds u times the total.  That takes one pass over
// the row (two rows, with D), shared by a cluster of CTAs: each sums its part of the row,
// the parts' sums go round through distributed shared memory, and the one CTA in whose
// part the place lies looks at the 1/8 of it (one warp's range) once more.
//
// Borders between tokens lie about 1/vocab apart, so the sums have to be much finer than
// fp32: pairs of fp32 numbers (47 bits), w = P - D exactly as rounded value and
// remainder, added without loss to the high word.  The 64-bit pipe has 1/64 of the fp32
// rate: 64-bit additions would take 230 us where the rows of 256 requests of 131072 tokens
// take 32 us to read, and even the scans and the second look in 64 bits took half the
// call (85 us).
#include <cooperative_groups.h>

#include "paged.h"

namespace cg = cooperative_groups;

namespace sgqa {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int NT = 256, NW = NT / 32;
constexpr int kMaxCluster = 8;
constexpr int kBatch = 2;  // 16-byte loads of a row in flight

struct VerifyArgs {
  const void *P, *D;
  const int32_t *tokens, *q_start, *kv_len;
  const float *u, *u_next;
  int32_t *n_accepted, *next_token, *keep_len, *status;
  int64_t ps, ds;  // row strides in elements
  int N, T, V;
};

template <typename T>
struct Unit;  // 16 bytes of a row
template <>
struct Unit<float> {
  static constexpr int N = 4;
  static __device__ __forceinline__ float get(const uint4& r, int i) {
    return __uint_as_float(i == 0 ? r.x : i == 1 ? r.y : i == 2 ? r.z : r.w);
  }
  static __device__ __forceinline__ void set(uint4& r, int i, float x) {
    (i == 0 ? r.x : i == 1 ? r.y : i == 2 ? r.z : r.w) = __float_as_uint(x);
  }
  static __device__ __forceinline__ float wide(float x) { return x; }
};
template <>
struct Unit<__nv_bfloat16> {
  static constexpr int N = 8;
  static __device__ __forceinline__ float get(const uint4& r, int i) {
    const uint32_t w = i < 2 ? r.x : i < 4 ? r.y : i < 6 ? r.z : r.w;
    return __uint_as_float(i & 1 ? w & 0xffff0000u : w << 16);
  }
  static __device__ __forceinline__ void set(uint4& r, int i, float x) {
    uint32_t& w = i < 2 ? r.x : i < 4 ? r.y : i < 6 ? r.z : r.w;
    const uint32_t b = __float_as_uint(x);
    w = i & 1 ? (w & 0xffffu) | b : (w & 0xffff0000u) | (b >> 16);
  }
  static __device__ __forceinline__ float wide(__nv_bfloat16 x) { return __bfloat162float(x); }
};

// Unit k of a row: elements [k N - m, k N - m + N), m the distance of the row of P from
// the 16-byte boundary before it.  Those that reach past the row's ends, and all of a row
// whose units do not lie on such boundaries, go element by element, 0 outside [0, V).
template <typename T>
__device__ __forceinline__ uint4 unit_by_element(const T* row, int m, int V, int k) {
  const int e0 = k * Unit<T>::N - m;
  uint4 r = make_uint4(0, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < Unit<T>::N; ++i)
    if (e0 + i >= 0 && e0 + i < V) Unit<T>::set(r, i, Unit<T>::wide(row[e0 + i]));
  return r;
}

// Two sums, each a high and a low word: w = max(p - d, 0) goes in as its rounded value
// and the remainder (exact, since p >= d >= 0), the value's own rounding in the high word is
// caught in the low one.  (Negative values and NaN count as 0.)
struct Sums {
  uint64_t h, l;
};
__device__ __forceinline__ void weigh(Sums& s, float p0, float d0, float p1, float d1) {
  const uint64_t minus = f2_pack(-1.0f, -1.0f);
  const uint64_t p = f2_pack(fmaxf(p0, 0.0f), fmaxf(p1, 0.0f));
  const uint64_t d = f2_pack(fmaxf(d0, 0.0f), fmaxf(d1, 0.0f));
  uint64_t w = f2_fma(d, minus, p);
  uint64_t rest = f2_fma(d, minus, f2_fma(w, minus, p));
  float w0, w1, r0, r1;
  f2_unpack(w, w0, w1);
  f2_unpack(rest, r0, r1);
  w = f2_pack(fmaxf(w0, 0.0f), fmaxf(w1, 0.0f));
  rest = f2_pack(w0 > 0.0f ? r0 : 0.0f, w1 > 0.0f ? r1 : 0.0f);
  const uint64_t t = f2_add(s.h, w), z = f2_fma(s.h, minus, t);
  const uint64_t lost = f2_add(f2_fma(f2_fma(z, minus, t), minus, s.h), f2_fma(z, minus, w));
  s.l = f2_add(s.l, f2_add(lost, rest));
  s.h = t;
}

// A number as a high and a low word, the high one the nearest to it.
struct Pair {
  float h, l;
};
__device__ __forceinline__ Pair operator+(Pair a, Pair b) {
  const float t = a.h + b.h, z = t - a.h;
  const float e = ((a.h - (t - z)) + (b.h - z)) + (a.l + b.l);
  const float h = t + e;
  return {h, e - (h - t)};
}
__device__ __forceinline__ bool operator>(Pair a, Pair b) {
  return a.h > b.h || (a.h == b.h && a.l > b.l);
}
__device__ __forceinline__ Pair times(Pair a, float u) {
  const float p = a.h * u, e = fmaf(a.h, u, -p) + a.l * u, h = p + e;
  return {h, e - (h - p)};
}
__device__ __forceinline__ Pair joined(const Sums& s) {
  Pair a, b;
  f2_unpack(s.h, a.h, b.h);
  f2_unpack(s.l, a.l, b.l);
  return a + b;
}

// A random number: a NaN stays one, so that nothing is below or passes it.
__device__ __forceinline__ float at_least_0(float u) { return u < 0.0f ? 0.0f : u; }

struct Shared {
  Pair warp[NW];           // sums of the warps' ranges
  Pair part[kMaxCluster];  // sums of the CTAs' parts, written by all CTAs
  Pair scan[NW];
  int accepted;            // drafts
  int bad;                 // the draft that was turned down lies outside the vocabulary
  int thread;              // that holds the place; the last one with a weight
};

__device__ __forceinline__ Pair shfl_xor(Pair x, int o) {
  return {__shfl_xor_sync(FULL, x.h, o), __shfl_xor_sync(FULL, x.l, o)};
}
__device__ __forceinline__ Pair warp_sum(Pair x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x = x + shfl_xor(x, o);
  return x;
}
// Sum of the lanes before this one.
__device__ __forceinline__ Pair warp_before(Pair x) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const Pair y{__shfl_up_sync(FULL, x.h, o), __shfl_up_sync(FULL, x.l, o)};
    if (lane >= o) x = x + y;
  }
  const Pair y{__shfl_up_sync(FULL, x.h, 1), __shfl_up_sync(FULL, x.l, 1)};
  return lane > 0 ? y : Pair{0.0f, 0.0f};
}

template <typename T>
__global__ void __launch_bounds__(NT, 1024 / NT) k_verify(const VerifyArgs a) {
  using U = Unit<T>;
  __shared__ Shared sh;
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int s = (int)(blockIdx.x / (unsigned)C);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // (no pdl_next: the next launch's blocks would take places beside clusters still at work)
  pdl_wait();
  const int q0 = a.q_start[s], q1 = a.q_start[s + 1], kv = a.kv_len[s];
  const bool fits = q0 >= 0 && q1 >= q0 && q1 <= a.T && kv >= q1 - q0;
  if (!fits || q1 == q0) {  // the whole cluster
    if (rank == 0 && tid == 0) {
      if (!fits) report(a.status, SGQA_ERR_BOUNDS, 361);
      a.n_accepted[s] = 0;
      a.next_token[s] = -1;
      a.keep_len[s] = kv;
    }
    return;
  }
  cluster.barrier_arrive();  // (waited for before anything is written to another CTA)
  const int k = q1 - q0 - 1;
  const T* P = static_cast<const T*>(a.P);
  const T* D = static_cast<const T*>(a.D);

  // ---- how many drafts are accepted
  if (warp == 0) {
    int i = 0, bad = 0;
    for (; i < k; i += 32) {
      const int j = i + lane;
      bool good = false, out = false;
      if (j < k) {
        const int x = a.tokens[q0 + j + 1];
        out = x < 0 || x >= a.V;
        if (!out) {
          const float p = fmaxf(U::wide(P[(int64_t)(q0 + j) * a.ps + x]), 0.0f);
          float d = 1.0f;
          if (D != nullptr) d = fmaxf(U::wide(D[(int64_t)(q0 + j) * a.ds + x]), 0.0f);
          good = (double)at_least_0(a.u[q0 + j]) * (double)d < (double)p;
        }
      }
      const unsigned down = __ballot_sync(FULL, !good && j < k);
      if (down) {
        const int l = __ffs(down) - 1;
        bad = __shfl_sync(FULL, (int)out, l);
        i += l;
        break;
      }
    }
    if (lane == 0) {
      sh.accepted = min(i, k);
      sh.bad = bad;
    }
  }
  if (tid == 0) sh.thread = -1;
  __syncthreads();
  const int n = sh.accepted;
  const bool bad = sh.bad != 0;
  const T* row = P + (int64_t)(q0 + n) * a.ps;
  const T* less = n < k && D != nullptr && !bad ? D + (int64_t)(q0 + n) * a.ds : nullptr;
  int out = -1;  // the token without a weight
  if (n < k && D == nullptr && !bad) out = a.tokens[q0 + n + 1];
  if (rank == 0 && tid == 0) {
    if (bad) report(a.status, SGQA_ERR_BOUNDS, 362);
    a.n_accepted[s] = n;
  }

  // ---- this CTA's units, and each warp's range of them
  const int V = a.V, m = (int)((reinterpret_cast<uintptr_t>(row) & 15u) / sizeof(T));
  const int units = (m + V + U::N - 1) / U::N;
  const int per_cta = (units + C - 1) / C, per_warp = (per_cta + NW - 1) / NW;
  const int end = min(units, (rank + 1) * per_cta);
  auto warp_begin = [&](int w) { return min(end, rank * per_cta + w * per_warp); };

  const int inner0 = m > 0 ? 1 : 0, inner1 = (m + V) / U::N;  // units inside the row

  for (int round = 0; round < 2; ++round) {
    // D may lie differently from P: then it is read element by element
    const bool whole = less != nullptr &&
                       ((reinterpret_cast<uintptr_t>(less) ^ reinterpret_cast<uintptr_t>(row)) & 15u) == 0;
    const int out_unit = out >= 0 ? (m + out) / U::N : -1;
    auto load = [&](int unit, uint4& x, uint4& y) {
      const bool inner = unit >= inner0 && unit < inner1;
      x = inner ? *reinterpret_cast<const uint4*>(row + unit * U::N - m)
                : unit_by_element(row, m, V, unit);
      y = make_uint4(0, 0, 0, 0);
      if (less != nullptr)
        y = inner && whole ? *reinterpret_cast<const uint4*>(less + unit * U::N - m)
                           : unit_by_element(less, m, V, unit);
      if (unit == out_unit) U::set(x, m + out - unit * U::N, 0.0f);
    };
    Sums sum{0ull, 0ull};
    const int from = warp_begin(warp), to = warp_begin(warp + 1);
    for (int u0 = from + lane; u0 < to; u0 += 32 * kBatch) {
      uint4 x[kBatch], y[kBatch];
      // all of the warp's units of this turn inside the row: their loads together
      const bool fast = u0 - lane >= inner0 && u0 - lane + 32 * kBatch <= min(to, inner1) &&
                        (less == nullptr || whole) &&
                        (out_unit < u0 - lane || out_unit >= u0 - lane + 32 * kBatch);
      if (fast) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
          x[b] = *reinterpret_cast<const uint4*>(row + (u0 + 32 * b) * U::N - m);
        if (less != nullptr) {
#pragma unroll
          for (int b = 0; b < kBatch; ++b)
            y[b] = *reinterpret_cast<const uint4*>(less + (u0 + 32 * b) * U::N - m);
        } else {
#pragma unroll
          for (int b = 0; b < kBatch; ++b) y[b] = make_uint4(0, 0, 0, 0);
        }
      } else {
#pragma unroll 1
        for (int b = 0; b < kBatch; ++b) {
          uint4 xb = make_uint4(0, 0, 0, 0), yb = xb;
          if (u0 + 32 * b < to) load(u0 + 32 * b, xb, yb);
#pragma unroll
          for (int e = 0; e < kBatch; ++e)
            if (e == b) {
              x[e] = xb;
              y[e] = yb;
            }
        }
      }
#pragma unroll
      for (int b = 0; b < kBatch; ++b)
#pragma unroll
        for (int i = 0; i < U::N; i += 2)
          weigh(sum, U::get(x[b], i), U::get(y[b], i), U::get(x[b], i + 1), U::get(y[b], i + 1));
    }
    const Pair none{0.0f, 0.0f};
    const Pair mine = warp_sum(joined(sum));
    if (lane == 0) sh.warp[warp] = mine;
    __syncthreads();
    if (round == 0) {
      cluster.barrier_wait();  // all CTAs have begun
      // (not before: keep_len may be kv_len, and a CTA that read the new length could take
      // the request for one that does not fit and leave the cluster)
      if (rank == 0 && tid == 0) a.keep_len[s] = kv - k + n;
    }
    if (tid < C) {
      Pair t = none;
#pragma unroll
      for (int w = 0; w < NW; ++w) t = t + sh.warp[w];
      cluster.map_shared_rank(&sh, tid)->part[rank] = t;
    }
    cluster.sync();
    Pair total = none;
    for (int c = 0; c < C; ++c) total = total + sh.part[c];
    if (total > none) {
      // the part, and in it the warp's range, that holds the place; the last one with a
      // weight where rounding (or a u of 1) leaves none
      const Pair place = times(total, at_least_0(a.u_next[s]));
      Pair before = none, at = none;
      int cta = -1;
      for (int c = 0; c < C; ++c) {
        const Pair next = at + sh.part[c];
        if (sh.part[c] > none) {
          cta = c;
          before = at;
          if (next > place) break;
        }
        at = next;
      }
      if (cta != rank) return;
      int r = 0;
      at = before;
      for (int w = 0; w < NW; ++w) {
        const Pair next = at + sh.warp[w];
        if (sh.warp[w] > none) {
          r = w;
          before = at;
          if (next > place) break;
        }
        at = next;
      }
      // its units once more, some in a row to a thread
      const int b0 = warp_begin(r), b1 = warp_begin(r + 1), each = (b1 - b0 + NT - 1) / NT;
      const int f0 = min(b1, b0 + tid * each), f1 = min(b1, f0 + each);
      Sums part{0ull, 0ull};
#pragma unroll 4
      for (int unit = f0; unit < f1; ++unit) {
        uint4 x, y;
        load(unit, x, y);
#pragma unroll
        for (int i = 0; i < U::N; i += 2)
          weigh(part, U::get(x, i), U::get(y, i), U::get(x, i + 1), U::get(y, i + 1));
      }
      const Pair own = joined(part);
      const Pair lanes = warp_before(own);
      if (lane == 31) sh.scan[warp] = lanes + own;
      __syncthreads();
      for (int w = 0; w < warp; ++w) before = before + sh.scan[w];
      Pair run = before + lanes;
      // the first thread whose sum passes the place, else the last one with a weight: the
      // largest of the threads that begin at or before it
      if (own > none && !(run > place)) atomicMax(&sh.thread, tid);
      __syncthreads();
      if (tid == max(sh.thread, 0)) {
        int token = -1;
        for (int unit = f0; unit < f1; ++unit) {
          uint4 x, y;
          load(unit, x, y);
          bool found = false;
#pragma unroll 1
          for (int i = 0; i < U::N; ++i) {
            Sums one{0ull, 0ull};
            weigh(one, U::get(x, i), U::get(y, i), 0.0f, 0.0f);
            const Pair w = joined(one);
            run = run + w;
            if (w > none) {
              token = unit * U::N - m + i;
              found = run > place;
            }
            if (found) break;
          }
          if (found) break;
        }
        a.next_token[s] = token;
      }
      return;
    }
    // no weight at all: P itself
    if (less == nullptr && out < 0) break;
    less = nullptr;
    out = -1;
    cluster.sync();  // all have read the parts' sums
  }
  if (rank == 0 && tid == 0) {
    report(a.status, SGQA_ERR_BOUNDS, 363);
    a.next_token[s] = -1;
  }
}

template <typename T>
int launch(const VerifyArgs& a, cudaStream_t st) {
  // CTAs of a cluster: halved while the call would still have three for each SM, and down
  // to parts of 16 KB (256 requests of 131072 fp32 tokens: 50 us with two, 51 with four, 57
  // with eight, 75 with one; 8 requests of 32768: 8.7 to 9.0 with four and eight, 14.1 with one)
  int c = kMaxCluster;
  while (c > 1 && ((int64_t)a.N * (c / 2) >= 3 * 152 ||
                   (int64_t)a.V * sizeof(T) / (c / 2) < 16384))
    c /= 2;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)c;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.N * c));
  cfg.blockDim = dim3(NT);
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  log_begin(SGQA_K_VERIFY, st);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k_verify<T>, a);
  log_end(st);
  return e == cudaSuccess ? SGQA_OK : SGQA_ERR_CUDA;
}

}  // namespace
}  // namespace sgqa

using namespace sgqa;

extern "C" SGQA_API int sgqa_draft_verify(
    const sgqa_verify_params* p, const void* P, const void* D, const int32_t* tokens,
    const int32_t* q_start, const int32_t* kv_len, const float* u, const float* u_next,
    int32_t* n_accepted, int32_t* next_token, int32_t* keep_len, int32_t* status,
    sgqa_stream_t stream) {
  if (p == nullptr || p->n_seqs < 0 || p->max_tokens < 0 || p->vocab < 1 || p->dtype < 0 ||
      p->dtype > 1 || (p->p_stride && p->p_stride < p->vocab) ||
      (p->d_stride && p->d_stride < p->vocab))
    return SGQA_ERR_INVALID_ARG;
  if (p->n_seqs > (1 << 20) || p->max_tokens > (1 << 24) || p->vocab > (1 << 24))
    return SGQA_ERR_UNSUPPORTED;
  if (p->n_seqs == 0) return SGQA_OK;
  if (q_start == nullptr || kv_len == nullptr || n_accepted == nullptr || next_token == nullptr ||
      keep_len == nullptr || u_next == nullptr ||
      (p->max_tokens > 0 && (P == nullptr || tokens == nullptr || u == nullptr)))
    return SGQA_ERR_INVALID_ARG;
  const unsigned e = p->dtype == SGQA_BF16 ? 2 : 4;
  if (reinterpret_cast<uintptr_t>(P) % e || reinterpret_cast<uintptr_t>(D) % e)
    return SGQA_ERR_ALIGNMENT;
  // Outputs on inputs: the CTAs of a request each read its lengths and drafts for themselves,
  // and have to come to the same verdict whatever other requests have written by then.
  const size_t n = (size_t)p->n_seqs * 4, t = (size_t)p->max_tokens * 4;
  auto rows = [&](int32_t stride) -> size_t {
    if (p->max_tokens == 0) return 0;
    return ((size_t)(p->max_tokens - 1) * (stride ? stride : p->vocab) + p->vocab) * e;
  };
  int32_t* const outs[3] = {n_accepted, next_token, keep_len};
  for (int i = 0; i < 3; ++i) {
    if (overlap(outs[i], n, q_start, n + 4) || overlap(outs[i], n, tokens, t) ||
        overlap(outs[i], n, u, t) || overlap(outs[i], n, u_next, n) ||
        overlap(outs[i], n, P, rows(p->p_stride)) || overlap(outs[i], n, D, rows(p->d_stride)) ||
        (outs[i] != kv_len ? overlap(outs[i], n, kv_len, n) : outs[i] != keep_len) ||
        overlap(outs[i], n, outs[(i + 1) % 3], n))
      return SGQA_ERR_INVALID_ARG;
  }
  VerifyArgs a;
  a.P = P;
  a.D = D;
  a.tokens = tokens;
  a.q_start = q_start;
  a.kv_len = kv_len;
  a.u = u;
  a.u_next = u_next;
  a.n_accepted = n_accepted;
  a.next_token = next_token;
  a.keep_len = keep_len;
  a.status = status;
  a.ps = p->p_stride ? p->p_stride : p->vocab;
  a.ds = p->d_stride ? p->d_stride : p->vocab;
  a.N = p->n_seqs;
  a.T = p->max_tokens;
  a.V = p->vocab;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  return p->dtype == SGQA_BF16 ? launch<__nv_bfloat16>(a, st) : launch<float>(a, st);
}
