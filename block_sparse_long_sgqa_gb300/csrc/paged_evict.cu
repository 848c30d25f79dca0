// Eviction from the paged cache by accumulated attention weight: which entries of each
// (request, KV group) stay and what moves, and the moves.
//
// The plan selects the `budget` largest of up to kv_len keys (an order-preserving map of
// the weights onto 32 bits), ties to the lower index, by radix: histograms of 11, 11 and
// 10 bits from the top, over keys that a block keeps in shared memory, read once through
// the page table.  With the threshold known, walks in index order count the ties where
// some of them are dropped, then holes (dropped below the budget) and movers (kept behind
// it), and write the i-th mover beside the i-th hole.  Long caches, and calls of few
// requests, share a (request, group) among a cluster of CTAs, which adds up its histograms
// through distributed shared memory.
//
// What bounds it: instructions (58 % of the issue slots while a block runs, 43 % over the whole
// call, which ends on the SMs with the longest requests) and the steps' barriers; 64 requests of
// 5K to 32K entries, 8 groups: 49 us where reading weights and positions takes 10.  Single pages
// over the budget are bound by the call.  Both with page tables no wider than the longest
// request: the host picks the form by that width, since it does not see the lengths, and short
// caches in a table of 256K positions take 446 us in place of 49 (single pages 60 in place of 8),
// in one of 1M 679 (76).
//
// Order among the kept entries has no meaning to attention, so entries below the budget
// stay where they are: a step that drops one page of entries moves about a page of rows,
// where a compaction in order would move the whole cache; and since every mover lies
// behind the budget and every hole before it, the moves are independent of each other.
#include <cooperative_groups.h>

#include "paged.h"

namespace cg = cooperative_groups;

namespace sgqa {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int NT = 1024, NW = NT / 32;
constexpr int kMaxCluster = 8;
constexpr int kBins = 2048;
constexpr int kMostKeys = 32768;  // a CTA's keys in shared memory (128 KB)
constexpr int kLoads = 4;         // loads of 4 keys a thread has in flight

struct PlanArgs {
  PagedDims pd;
  const float* mass;
  const int32_t *pos, *page_table, *kv_len, *next_pos;
  int32_t *n_moves, *moves, *kv_len_out, *status;
  int budget, recent, sinks;
};

struct PlanShared {
  uint32_t hist[3][kBins];
  int warp[2][NW];              // sums of the warps
  int part[2][2][kMaxCluster];  // sums of the CTAs, written by all of the cluster
  uint32_t digit;
  int above, equal;
};

// Entries i .. i + 3, i a multiple of 4 (a page holds a multiple of 8): their place in the
// pool, -1 outside it.
__device__ __forceinline__ int64_t place_of(const PlanArgs& a, const int32_t* table, int g, int i) {
  const unsigned pi = (unsigned)i / (unsigned)a.pd.ps;
  const int page = table[pi];
  if (page < 0 || page >= a.pd.n_pages) {
    report(a.status, SGQA_ERR_BOUNDS, 371);
    return -1;
  }
  return ((int64_t)page * a.pd.Hkv + g) * a.pd.ps + (i - (int)pi * a.pd.ps);
}
// The key of an entry of weight m and position p: larger is kept first.
__device__ __forceinline__ uint32_t key_of(const PlanArgs& a, float m, int p, int recent) {
  // the map of order_key; -0 counts as 0, a NaN as -infinity
  const int u = __float_as_int(m + 0.0f);
  uint32_t key = (uint32_t)u ^ ((uint32_t)(u >> 31) | 0x80000000u);
  if (m != m) key = 0x007fffffu;
  return p < a.sinks || p >= recent ? 0xff800000u : key;
}

// Sum of v over the warps before this one, of one value a warp.
__device__ __forceinline__ int before_warp(int* shared, int v) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (lane == 0) shared[warp] = v;
  __syncthreads();
  int inc = shared[lane];
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(FULL, inc, o);
    if (lane >= o) inc += x;
  }
  return __shfl_sync(FULL, inc, warp) - v;
}
static_assert(NW == 32, "a lane for each warp");

// The digit (of kBins) in which the k-th largest lies, how many lie in higher ones and
// how many in it: histograms added up over the cluster, then summed from the top, two
// bins a thread.
template <int C>
__device__ __forceinline__ void find_digit(PlanShared& sh, int pass, int k) {
  static_assert(kBins == 2 * NT, "two bins a thread");
  const int tid = threadIdx.x, lane = tid & 31;
  const int b0 = kBins - 2 - 2 * tid;  // thread 0 has the highest
  uint2 h = make_uint2(0, 0);
  if constexpr (C == 1) {
    h = *reinterpret_cast<const uint2*>(&sh.hist[pass][b0]);
  } else {
    cg::cluster_group cluster = cg::this_cluster();
#pragma unroll
    for (int c = 0; c < C; ++c) {
      const uint2 x = *reinterpret_cast<const uint2*>(&cluster.map_shared_rank(&sh, c)->hist[pass][b0]);
      h.x += x.x;
      h.y += x.y;
    }
  }
  const int mine = (int)(h.x + h.y);
  int inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(FULL, inc, o);
    if (lane >= o) inc += x;
  }
  const int above = before_warp(sh.warp[pass & 1], __shfl_sync(FULL, inc, 31)) + inc - mine;
  if (above < k && above + mine >= k) {
    const bool first = above + (int)h.y >= k;
    sh.digit = (uint32_t)(first ? b0 + 1 : b0);
    sh.above = first ? above : above + (int)h.y;
    sh.equal = (int)(first ? h.y : h.x);
  }
  __syncthreads();
}

template <bool HELD, int C>
__global__ void __launch_bounds__(NT) k_evict_plan(const __grid_constant__ PlanArgs a) {
  __shared__ __align__(16) PlanShared sh;
  extern __shared__ __align__(16) uint32_t keys[];
  const int unit = (int)(blockIdx.x / (unsigned)C), rank = (int)(blockIdx.x % (unsigned)C);
  const int s = unit / a.pd.Hkv, g = unit - s * a.pd.Hkv;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  pdl_next();
  pdl_wait();
  const int kv = a.kv_len[s];
  const bool fits = kv >= 0 && kv <= a.pd.cap;
  if (!fits || kv <= a.budget) {  // the whole cluster
    if (rank == 0 && tid == 0) {
      if (!fits) report(a.status, SGQA_ERR_BOUNDS, 372);
      a.n_moves[unit] = 0;
      if (g == 0) a.kv_len_out[s] = fits ? kv : 0;
    }
    return;
  }
  auto sync = [&]() {
    if constexpr (C > 1)
      cg::this_cluster().sync();
    else
      __syncthreads();
  };
  const int next = a.next_pos != nullptr ? a.next_pos[s] : kv;
  const int32_t* table = a.page_table + (int64_t)s * a.pd.max_pages;
  // the first position that counts as recent (clamped: every position is at least that)
  const int recent = (int)max((int64_t)next - a.recent, (int64_t)-0x80000000ll);
  constexpr uint32_t none = 0x007fffffu;  // -infinity

  // this CTA's entries [i0, i0 + n)
  const int per_cta = (((kv + C - 1) / C) + 3) & ~3;
  const int i0 = min(kv, rank * per_cta), n = min(kv, i0 + per_cta) - i0;
  auto key_at = [&](int x) -> uint32_t {
    if constexpr (HELD) return keys[x];
    const int i = i0 + x;
    const int64_t at = place_of(a, table, g, i & ~3);
    if (at < 0) return none;
    return key_of(a, a.mass[at + (i & 3)], a.pos != nullptr ? a.pos[at + (i & 3)] : i, recent);
  };
  *reinterpret_cast<uint2*>(&sh.hist[0][2 * tid]) = make_uint2(0, 0);
  *reinterpret_cast<uint2*>(&sh.hist[1][2 * tid]) = make_uint2(0, 0);
  *reinterpret_cast<uint2*>(&sh.hist[2][2 * tid]) = make_uint2(0, 0);
  __syncthreads();
  auto count = [&](uint32_t v) { atomicAdd(&sh.hist[0][v >> 21], 1u); };
  if constexpr (HELD) {
    // four entries a load, the loads of several together: what this costs is the trip to
    // the page table and the one behind it
    for (int x0 = 4 * tid; x0 < n; x0 += 4 * NT * kLoads) {
      int64_t at[kLoads];
      float4 m[kLoads];
      int4 p[kLoads];
#pragma unroll
      for (int b = 0; b < kLoads; ++b) {
        const int x = x0 + 4 * NT * b;
        at[b] = x < n ? place_of(a, table, g, i0 + x) : -1;
      }
#pragma unroll
      for (int b = 0; b < kLoads; ++b) {
        const int i = i0 + x0 + 4 * NT * b;
        p[b] = make_int4(i, i + 1, i + 2, i + 3);
        if (at[b] < 0) continue;
        m[b] = *reinterpret_cast<const float4*>(a.mass + at[b]);
        if (a.pos != nullptr) p[b] = *reinterpret_cast<const int4*>(a.pos + at[b]);
      }
#pragma unroll
      for (int b = 0; b < kLoads; ++b) {
        const int x = x0 + 4 * NT * b;
        if (x >= n) continue;
        uint4 v = make_uint4(none, none, none, none);
        if (at[b] >= 0)
          v = make_uint4(key_of(a, m[b].x, p[b].x, recent), key_of(a, m[b].y, p[b].y, recent),
                         key_of(a, m[b].z, p[b].z, recent), key_of(a, m[b].w, p[b].w, recent));
        *reinterpret_cast<uint4*>(keys + x) = v;  // (what lies behind n is not looked at)
        count(v.x);
        if (x + 1 < n) count(v.y);
        if (x + 2 < n) count(v.z);
        if (x + 3 < n) count(v.w);
      }
    }
  } else {
    for (int x = tid; x < n; x += NT) count(key_at(x));
  }

  // ---- the threshold: the budget-th largest key, and how many equal to it stay
  uint32_t prefix = 0;
  int k = a.budget;
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 1 ? 10 : 0, known = pass == 1 ? 11 : 22;
    const uint32_t mask = pass == 2 ? 1023u : 2047u;
    if (pass > 0) {
#pragma unroll 4
      for (int x = tid; x < n; x += NT) {
        const uint32_t v = key_at(x);
        if (v >> (32 - known) == prefix) atomicAdd(&sh.hist[pass][(v >> shift) & mask], 1u);
      }
    }
    sync();
    find_digit<C>(sh, pass, k);
    prefix = prefix << (pass == 2 ? 10 : 11) | sh.digit;
    k -= sh.above;
  }
  const uint32_t limit = prefix;
  const int ties = k;                   // entries equal to it that stay, the first in order
  const bool all = ties == sh.equal;    // all of them, as a rule: nothing to count

  // ---- walks in index order: a warp's range, 32 entries at a time
  const int per_warp = (((n + NW - 1) / NW) + 31) & ~31;
  const int w0 = min(n, warp * per_warp), w1 = min(n, w0 + per_warp);
  // sums over the warps and CTAs before this warp; the CTAs' sums stay in sh.part[which]
  auto before = [&](int which, int v0, int v1, int& b0, int& b1) {
    __syncthreads();
    b0 = before_warp(sh.warp[0], v0);
    b1 = before_warp(sh.warp[1], v1);
    if constexpr (C > 1) {
      cg::cluster_group cluster = cg::this_cluster();
      if (tid >= NT - C) {  // threads of the last warp know the CTA's sums
        PlanShared* to = cluster.map_shared_rank(&sh, tid - (NT - C));
        to->part[which][0][rank] = b0 + v0;
        to->part[which][1][rank] = b1 + v1;
      }
      cluster.sync();
      for (int c = 0; c < rank; ++c) {
        b0 += sh.part[which][0][c];
        b1 += sh.part[which][1][c];
      }
    }
  };
  int tie0 = 0;
  if (!all) {  // (the same in all CTAs of the cluster)
    int equal = 0, unused;
    for (int x = w0 + lane; x < w1; x += 32) equal += key_at(x) == limit;
    before(0, __reduce_add_sync(FULL, equal), 0, tie0, unused);
  }
  const unsigned lower = (1u << lane) - 1u;
  const int edge = min(max(a.budget - i0, w0), w1);  // holes lie before it, movers from it on
  auto walk = [&](auto visit) {
    int tie = tie0;
    auto range = [&](int b, int e, bool holes) {
#pragma unroll 4
      for (int x0 = b; x0 < e; x0 += 32) {
        const int x = x0 + lane;
        const uint32_t v = x < e ? key_at(x) : 0;
        bool kept = v >= limit;
        if (!all) {
          const unsigned eq = __ballot_sync(FULL, x < e && v == limit);
          kept = kept && (v > limit || tie + __popc(eq & lower) < ties);
          tie += __popc(eq);
        }
        visit(i0 + x, __ballot_sync(FULL, x < e && kept != holes), holes);
      }
    };
    range(w0, edge, true);
    range(edge, w1, false);
  };
  int holes = 0, movers = 0;
  if (all) {  // (in any order)
    int below = 0;
#pragma unroll 4
    for (int x = w0 + lane; x < edge; x += 32) below += key_at(x) >= limit;
#pragma unroll 4
    for (int x = edge + lane; x < w1; x += 32) movers += key_at(x) >= limit;
    holes = edge - w0 - __reduce_add_sync(FULL, below);
    movers = __reduce_add_sync(FULL, movers);
  } else {
    walk([&](int, unsigned m, bool hole) { (hole ? holes : movers) += __popc(m); });
  }
  int hole0, mover0;
  before(1, holes, movers, hole0, mover0);
  // the last warp of the last CTA knows how many moves there are
  if (rank == C - 1 && tid == NT - 1) {
    a.n_moves[unit] = mover0 + movers;
    if (g == 0) a.kv_len_out[s] = a.budget;
  }
  int32_t* moves = a.moves + (int64_t)unit * a.budget * 2;
  walk([&](int i, unsigned m, bool hole) {
    int& at = hole ? hole0 : mover0;
    if (m >> lane & 1u) moves[2 * (int64_t)(at + __popc(m & lower)) + (hole ? 1 : 0)] = i;
    at += __popc(m);
  });
}

template <bool HELD, int C>
int launch_plan(const PlanArgs& a, size_t smem, cudaStream_t st) {
  // (less needs no leave; always the most that a call can ask for: the limit belongs to the
  // process, and another thread's smaller call must not lower it before this one's launch)
  if (smem + sizeof(PlanShared) > 48 * 1024 &&
      cudaFuncSetAttribute(k_evict_plan<HELD, C>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                           kMostKeys * 4) != cudaSuccess)
    return SGQA_ERR_CUDA;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = C;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.pd.N * a.pd.Hkv * C));
  cfg.blockDim = dim3(NT);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = C > 1 ? 2 : 1;
  log_begin(SGQA_K_EVICT, st);
  const cudaError_t e = cudaLaunchKernelEx(&cfg, k_evict_plan<HELD, C>, a);
  log_end(st);
  return e == cudaSuccess ? SGQA_OK : SGQA_ERR_CUDA;
}

// ------------------------------------------------------------------------ moves
constexpr int MT = 256;  // threads

struct MoveArgs {
  PagedDims pd;
  const int32_t *page_table, *n_moves, *moves;
  uint4 *K, *V;
  float* mass;
  int32_t* pos;
  int32_t* status;
  int budget;
  int per;  // blocks of a (request, group)
};

// A warp takes 32 moves at a time, a lane looking up the rows of each, and copies the rows
// of K and V a few moves at a time, all loads of a batch before its stores.  No two moves
// touch the same row, so nothing waits for anything else.  Bound by memory in pieces of a
// row: 32 requests of 5K to 32K entries cut to 4096, 8 groups: 136 us, 5.6 TB/s (147 with a
// sixth of the blocks).
template <int LOG_UP>
__global__ void __launch_bounds__(MT, 4) k_evict_move(const __grid_constant__ MoveArgs a) {
  constexpr int UP = 1 << LOG_UP;                  // units of a row
  constexpr int PER = 2 * UP >= 32 ? 1 : 32 / (2 * UP);  // moves in one load of the warp
  constexpr int LOADS = 2 * UP <= 32 ? 1 : 2 * UP / 32;  // loads of a move
  constexpr int BATCH = 8 / LOADS;
  pdl_next();
  pdl_wait();
  const int unit = (int)(blockIdx.x / (unsigned)a.per), part = (int)blockIdx.x - unit * a.per;
  const int s = unit / a.pd.Hkv, g = unit - s * a.pd.Hkv;
  const int lane = lane_id();
  int n = a.n_moves[unit];
  // (targets are distinct, so there are no more moves than places; the index below stays far
  // from 2^31 so)
  if (n < 0 || n > min(a.budget, a.pd.cap)) {
    if (part == 0 && threadIdx.x == 0) report(a.status, SGQA_ERR_BOUNDS, 381);
    n = 0;
  }
  const int32_t* table = a.page_table + (int64_t)s * a.pd.max_pages;
  const int2* moves = reinterpret_cast<const int2*>(a.moves) + (int64_t)unit * a.budget;
  for (int m0 = (part * (MT / 32) + (int)warp_id()) * 32; m0 < n; m0 += a.per * MT) {
    const int here = min(32, n - m0);
    int r[2] = {-1, -1};
    if (lane < here) {
      const int2 mv = moves[m0 + lane];
      r[0] = mv.x;
      r[1] = mv.y;
      bool ok = true;
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        ok = ok && r[e] >= 0 && r[e] < a.pd.cap;
        if (ok) {
          const unsigned pi = (unsigned)r[e] / (unsigned)a.pd.ps;
          const int page = table[pi];
          ok = page >= 0 && page < a.pd.n_pages;
          r[e] = (page * a.pd.Hkv + g) * a.pd.ps + (r[e] - (int)pi * a.pd.ps);
        }
      }
      if (!ok) {
        report(a.status, SGQA_ERR_BOUNDS, 382);
        r[0] = -1;
      }
    }
    float mass = 0.0f;
    int pos = 0;
    if (r[0] >= 0 && a.mass != nullptr) mass = a.mass[r[0]];
    if (r[0] >= 0 && a.pos != nullptr) pos = a.pos[r[0]];
    for (int m = 0; m < here; m += PER * BATCH) {
      uint4 v[BATCH][LOADS];
      int dst[BATCH];  // row
      const int sub = lane / (2 * UP < 32 ? 2 * UP : 32);  // which move of a load
#pragma unroll
      for (int b = 0; b < BATCH; ++b) {
        const int x = m + b * PER + sub;
        const int from = __shfl_sync(0xffffffffu, r[0], x & 31);
        const int to = __shfl_sync(0xffffffffu, r[1], x & 31);
        dst[b] = x < here && from >= 0 ? to : -1;
        if (dst[b] < 0) continue;
#pragma unroll
        for (int l = 0; l < LOADS; ++l) {
          const int u = (lane + 32 * l) & (2 * UP - 1);  // unit of K's row, then of V's
          v[b][l] = (u & UP ? a.V : a.K)[((int64_t)from << LOG_UP) + (u & (UP - 1))];
        }
      }
#pragma unroll
      for (int b = 0; b < BATCH; ++b) {
        if (dst[b] < 0) continue;
#pragma unroll
        for (int l = 0; l < LOADS; ++l) {
          const int u = (lane + 32 * l) & (2 * UP - 1);
          (u & UP ? a.V : a.K)[((int64_t)dst[b] << LOG_UP) + (u & (UP - 1))] = v[b][l];
        }
      }
    }
    if (r[0] >= 0 && a.mass != nullptr) a.mass[r[1]] = mass;
    if (r[0] >= 0 && a.pos != nullptr) a.pos[r[1]] = pos;
  }
}

inline bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

int check_budget(const PagedDims& pd, int budget) {
  if (budget < 1) return SGQA_ERR_INVALID_ARG;
  if ((int64_t)pd.N * pd.Hkv > (1 << 24) || (double)pd.N * pd.Hkv * budget > 2147483647.0)
    return SGQA_ERR_UNSUPPORTED;
  return SGQA_OK;
}

}  // namespace
}  // namespace sgqa

using namespace sgqa;

extern "C" {

SGQA_API int sgqa_evict_plan(const sgqa_paged_params* p, int32_t budget, int32_t recent,
                             int32_t sinks, const float* mass_pages, const int32_t* pos_pages,
                             const int32_t* page_table, const int32_t* kv_len,
                             const int32_t* next_pos, int32_t* n_moves, int32_t* moves,
                             int32_t* kv_len_out, int32_t* status, sgqa_stream_t stream) {
  PagedDims pd;
  int rc = derive_paged(p, &pd);
  if (rc == SGQA_OK) rc = check_budget(pd, budget);
  if (rc != SGQA_OK) return rc;
  if (recent < 0 || sinks < 0 || (int64_t)recent + sinks > budget) return SGQA_ERR_INVALID_ARG;
  if (pd.N == 0) return SGQA_OK;
  if (mass_pages == nullptr || page_table == nullptr || kv_len == nullptr || n_moves == nullptr ||
      moves == nullptr || kv_len_out == nullptr || kv_len_out == kv_len)
    return SGQA_ERR_INVALID_ARG;
  if (!aligned16(mass_pages) || !aligned16(pos_pages)) return SGQA_ERR_ALIGNMENT;
  // Outputs on inputs: the CTAs of a (request, group) read its length and its entries each for
  // itself, and more than once, while other (request, group)s write theirs.
  const size_t seqs = (size_t)pd.N * 4, units = seqs * pd.Hkv;
  const size_t entries = (size_t)pd.n_pages * pd.Hkv * pd.ps * 4;
  const struct {
    const void* p;
    size_t n;
  } outs[3] = {{n_moves, units}, {moves, units * 2 * budget}, {kv_len_out, seqs}};
  for (int i = 0; i < 3; ++i) {
    const auto& o = outs[i];
    if (overlap(o.p, o.n, kv_len, seqs) || overlap(o.p, o.n, next_pos, seqs) ||
        overlap(o.p, o.n, page_table, seqs * pd.max_pages) ||
        overlap(o.p, o.n, mass_pages, entries) || overlap(o.p, o.n, pos_pages, entries) ||
        overlap(o.p, o.n, outs[(i + 1) % 3].p, outs[(i + 1) % 3].n))
      return SGQA_ERR_INVALID_ARG;
  }
  PlanArgs a;
  a.pd = pd;
  a.mass = mass_pages;
  a.pos = pos_pages;
  a.page_table = page_table;
  a.kv_len = kv_len;
  a.next_pos = next_pos;
  a.n_moves = n_moves;
  a.moves = moves;
  a.kv_len_out = kv_len_out;
  a.status = status;
  a.budget = budget;
  a.recent = recent;
  a.sinks = sinks;
  // CTAs of a cluster: as few as hold the keys that a request can have (by the width of the
  // table, the only bound on the lengths that the host knows), since a cluster's barriers and
  // the histograms of the others cost more than they share out (64 requests of 5K to 32K
  // entries, 8 groups: 59 us with one CTA, 81 with two, 153 with four, before both got
  // faster); more where the call would leave SMs idle and a CTA keeps 4096 keys
  int c = 1;
  while (c < kMaxCluster && ((int64_t)c * kMostKeys < pd.cap ||
                             ((int64_t)pd.N * pd.Hkv * c < 152 && (int64_t)c * 8192 < pd.cap)))
    c *= 2;
  const int64_t keys = (((int64_t)pd.cap + c - 1) / c + 3) & ~int64_t(3);
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (keys > kMostKeys) return launch_plan<false, kMaxCluster>(a, 0, st);
  const size_t smem = (size_t)keys * 4;
  return c == 1   ? launch_plan<true, 1>(a, smem, st)
         : c == 2 ? launch_plan<true, 2>(a, smem, st)
         : c == 4 ? launch_plan<true, 4>(a, smem, st)
                  : launch_plan<true, 8>(a, smem, st);
}

SGQA_API int sgqa_evict_move(const sgqa_paged_params* p, int32_t budget,
                             const int32_t* page_table, const int32_t* n_moves,
                             const int32_t* moves, void* K_pages, void* V_pages,
                             float* mass_pages, int32_t* pos_pages, int32_t* status,
                             sgqa_stream_t stream) {
  PagedDims pd;
  int rc = derive_paged(p, &pd);
  if (rc == SGQA_OK) rc = check_budget(pd, budget);
  if (rc != SGQA_OK) return rc;
  if (pd.N == 0) return SGQA_OK;
  if (page_table == nullptr || n_moves == nullptr || moves == nullptr || K_pages == nullptr ||
      V_pages == nullptr)
    return SGQA_ERR_INVALID_ARG;
  if (!aligned16(K_pages) || !aligned16(V_pages) || (reinterpret_cast<uintptr_t>(moves) & 7u))
    return SGQA_ERR_ALIGNMENT;
  MoveArgs a;
  a.pd = pd;
  a.page_table = page_table;
  a.n_moves = n_moves;
  a.moves = moves;
  a.K = static_cast<uint4*>(K_pages);
  a.V = static_cast<uint4*>(V_pages);
  a.mass = mass_pages;
  a.pos = pos_pages;
  a.status = status;
  a.budget = budget;
  // blocks of a (request, group): a move a thread, but not many more blocks in all than
  // the SMs hold at a time
  const int units = pd.N * pd.Hkv, most = (152 * 64 + units - 1) / units;
  a.per = (int)(((int64_t)budget + MT - 1) / MT);
  if (a.per > most) a.per = most;
  cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  const int up = pd.d * pd.elem / 16;  // 8, 16 or 32
  log_begin(SGQA_K_EVICT, st);
  const cudaError_t e =
      up == 8    ? launch_pdl(k_evict_move<3>, (int64_t)units * a.per, MT, 0, st, a)
      : up == 16 ? launch_pdl(k_evict_move<4>, (int64_t)units * a.per, MT, 0, st, a)
                 : launch_pdl(k_evict_move<5>, (int64_t)units * a.per, MT, 0, st, a);
  log_end(st);
  return e == cudaSuccess ? SGQA_OK : SGQA_ERR_CUDA;
}

}  // extern "C"
