// Page tables and slot maps of a ragged serving batch, built on the device
// from its lengths, and the return of pages.
//
// Everything follows from exclusive sums over the requests: of the new tokens
// (q_start) and of the new pages.  Page i of request s, when it is new, is
// free_pages[n_free - 1 - (first_s + i - held_s)] with first_s the sum of the
// new pages of the requests before s, so a token knows its page without
// waiting for the table: one launch writes the table, the slots and the
// positions.  Every CTA computes the sums for itself (a few KB of lengths,
// from L2) and then serves an equal range of tokens, finding a token's request
// by bisection of the sums in shared memory.  The work is a few bytes per
// token (1.6 MB for 129K of them, 0.2 us at the copy rate); what bounds a call is
// the launch and the chain of trips to memory: 3.8 us for 256 requests of one
// token, 5.0 for 512 requests and 129K tokens, in a row of such calls.
#include "paged.h"

namespace sgqa {
namespace {

constexpr int kSMs = 152;       // most CTAs
constexpr int kCheckNT = 160;   // threads that look at one CTA's range each
static_assert(kCheckNT >= kSMs, "");
constexpr int NT = 512;         // threads
constexpr int PER = 4;          // requests per thread and tile
constexpr int TILE = NT * PER;  // requests summed at a time

// Two sums at once: tokens in bits 0-35, pages above.  A tile has at most 2^11
// requests of at most 2^24 tokens each (longer ones are refused), so the lower
// sum cannot carry; the upper one is exact whenever the tokens fit max_tokens
// (pages <= tokens / 8 + requests).
constexpr int kShift = 36;
constexpr uint64_t kLow = (uint64_t(1) << kShift) - 1;

struct Shared {
  uint64_t excl[TILE];   // exclusive sums of the tile, both halves
  uint64_t warp[NT / 32];
  unsigned long long tot[2];
  int bad;
};

__device__ __forceinline__ int pages_of(int len, int ps) { return (len + ps - 1) / ps; }

// Exclusive sums of v[0..PER) over the block (thread t holds requests PER t ..),
// left in sh.excl; returns the tile's total.
__device__ uint64_t block_scan(Shared& sh, const uint64_t (&v)[PER]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  uint64_t mine = 0;
#pragma unroll
  for (int i = 0; i < PER; ++i) mine += v[i];
  uint64_t inc = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const uint64_t x = __shfl_up_sync(0xffffffffu, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) sh.warp[warp] = inc;
  __syncthreads();
  uint64_t before = 0, total = 0;
#pragma unroll
  for (int w = 0; w < NT / 32; ++w) {
    const uint64_t x = sh.warp[w];
    before += w < warp ? x : 0;
    total += x;
  }
  uint64_t e = before + inc - mine;
#pragma unroll
  for (int i = 0; i < PER; ++i) {
    sh.excl[threadIdx.x * PER + i] = e;
    e += v[i];
  }
  __syncthreads();
  return total;
}

// Last request of the tile's first n whose exclusive sum (the half that `part`
// takes) is at most x.
template <typename F>
__device__ __forceinline__ int find(int n, F part, int64_t x) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (part(mid) <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

// What one request asks for; bad = 1 (bounds) or 2 (more tokens than rows).
struct Need {
  int q, kv, held, pages, bad;
};
__device__ __forceinline__ Need need_of(const PagedDims& pd, const int32_t* q_len,
                                        const int32_t* kv_len, int s) {
  Need n{0, 0, 0, 0, 0};
  if (s >= pd.N) return n;
  const int q = q_len[s], kv = kv_len[s];
  if (q < 0 || kv < q || kv > pd.cap) {
    n.bad = 1;
    return n;
  }
  if (q > pd.T) {
    n.bad = 2;
    return n;
  }
  n.q = q;
  n.kv = kv;
  n.held = pages_of(kv - q, pd.ps);
  n.pages = pages_of(kv, pd.ps) - n.held;
  return n;
}

__device__ __forceinline__ uint64_t both(const Need& n) {
  return (uint64_t)n.q | ((uint64_t)n.pages << kShift);
}

// Requests in more than one tile: their totals first.
template <typename F>
__device__ void totals(Shared& sh, int N, F one, uint64_t& tok, uint64_t& pages) {
  if (threadIdx.x == 0) sh.tot[0] = sh.tot[1] = 0;
  __syncthreads();
  unsigned long long a = 0, b = 0;
  int bad = 0;
  for (int s = threadIdx.x; s < N; s += NT) {
    const Need n = one(s);
    a += n.q;
    b += n.pages;
    bad |= n.bad;
  }
  if (a) atomicAdd(&sh.tot[0], a);
  if (b) atomicAdd(&sh.tot[1], b);
  if (bad) atomicOr(&sh.bad, bad);
  __syncthreads();
  tok = sh.tot[0];
  pages = sh.tot[1];
}

__global__ void __launch_bounds__(NT)
    k_page_plan(PagedDims pd, const int32_t* q_len, const int32_t* kv_len,
                const int32_t* free_pages, const int32_t* n_free_p, int32_t* page_table,
                int32_t* q_start, int64_t* slot_map, int32_t* positions, int32_t* n_free_out,
                int32_t* status) {
  __shared__ Shared sh;
  pdl_next();
  pdl_wait();
  const int ntile = (pd.N + TILE - 1) / TILE;
  const int n_free = *n_free_p;
  if (threadIdx.x == 0) sh.bad = 0;
  __syncthreads();
  auto one = [&](int s) { return need_of(pd, q_len, kv_len, s); };
  uint64_t tok = 0, pages = 0;
  if (ntile > 1) totals(sh, pd.N, one, tok, pages);
  uint64_t tok0 = 0, pages0 = 0;  // of the tiles before
  bool ok = false;
  const int64_t per = ((int64_t)pd.T + gridDim.x - 1) / gridDim.x;
  const int t0 = (int)min((int64_t)pd.T, blockIdx.x * per);
  const int t1 = (int)min((int64_t)pd.T, t0 + per);
  for (int tile = 0; tile < max(ntile, 1); ++tile) {
    const int s0 = tile * TILE;
    uint64_t v[PER];
    int bad = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const Need n = one(s0 + threadIdx.x * PER + i);
      v[i] = both(n);
      bad |= n.bad;
    }
    if (bad) atomicOr(&sh.bad, bad);
    const uint64_t sum = block_scan(sh, v);  // (and a barrier behind sh.bad)
    if (ntile <= 1) {
      tok = sum & kLow;
      pages = sum >> kShift;
    }
    if (tile == 0) {
      const int code = (sh.bad & 1) || n_free < 0 || n_free > pd.n_pages ? SGQA_ERR_BOUNDS
                       : sh.bad || tok > (uint64_t)pd.T || pages > (uint64_t)n_free
                           ? SGQA_ERR_CAPACITY
                           : SGQA_OK;
      ok = code == SGQA_OK;
      if (blockIdx.x == 0 && threadIdx.x == 0) {
        if (!ok) report(status, code, 311);
        *n_free_out = ok ? n_free - (int)pages : n_free;
      }
      if (!ok) break;
    }
    if (blockIdx.x == 0) {
      for (int i = threadIdx.x; i < TILE && s0 + i < pd.N; i += NT)
        q_start[s0 + i] = (int)(tok0 + (sh.excl[i] & kLow));
    }
    // this CTA's tokens that belong to requests of the tile
    const int a = (int)max((int64_t)t0, (int64_t)tok0);
    const int b = (int)min((int64_t)t1, (int64_t)(tok0 + (sum & kLow)));
    const int n = min(TILE, pd.N - s0);
    for (int t = a + (int)threadIdx.x; t < b; t += NT) {
      const int64_t x = t - (int64_t)tok0;
      // the last request that starts at or before x holds it: those without
      // tokens start where the next one does
      const int i = find(n, [&](int k) { return (int64_t)(sh.excl[k] & kLow); }, x);
      const int s = s0 + i;
      const int q = q_len[s], kv = kv_len[s];
      const int pos = kv - q + (int)(x - (int64_t)(sh.excl[i] & kLow));
      const int held = pages_of(kv - q, pd.ps), page_i = pos / pd.ps, off = pos % pd.ps;
      int page;
      int32_t* row = page_table + (int64_t)s * pd.max_pages + page_i;
      if (page_i < held) {
        page = *row;
      } else {
        page = free_pages[n_free - 1 - (int)(pages0 + (sh.excl[i] >> kShift)) - (page_i - held)];
        if (off == 0) *row = page;  // every new page starts with a new token
      }
      int64_t slot = (int64_t)page * pd.ps + off;
      if (page < 0 || page >= pd.n_pages) {
        report(status, SGQA_ERR_BOUNDS, 312);
        slot = -1;
      }
      slot_map[t] = slot;
      positions[t] = pos;
    }
    tok0 += sum & kLow;
    pages0 += sum >> kShift;
    __syncthreads();  // the next tile overwrites sh.excl
  }
  if (!ok) {
    if (blockIdx.x == 0)
      for (int i = threadIdx.x; i <= pd.N; i += NT) q_start[i] = 0;
  } else if (blockIdx.x == 0 && threadIdx.x == 0) {
    q_start[pd.N] = (int)tok0;
  }
  for (int t = max(t0, ok ? (int)min((uint64_t)t1, tok) : t0) + (int)threadIdx.x; t < t1; t += NT) {
    slot_map[t] = -1;
    positions[t] = -1;
  }
}

// Pages of the requests' tails pushed on the stack: the same sums, over the
// pages given back; CTAs serve equal ranges of them.  A page number outside the
// pool refuses the whole call, which no CTA can tell for the others' ranges: it
// leaves kBadPage as the first page of its own, behind the stack's present top,
// and the next launch (one CTA) takes the count back if there is one.  1000 requests
// that give back 49 thousand pages: 5.9 us in a row of such calls, 3.7 without the
// second launch; 12 with one cluster of 8 CTAs that looks over all pages, meets and
// then pushes them (2000 requests, 363 thousand pages: 11, 7.5 and 47 us).
constexpr int kBadPage = -1;

// The pages that CTA b of the release's grid gives back.
struct Range {
  int64_t begin, end;
};
__device__ __forceinline__ Range range_of(int64_t pages, unsigned grid, unsigned b) {
  const int64_t per = (pages + grid - 1) / grid;
  return {min(pages, b * per), min(pages, (b + 1) * per)};
}

__global__ void __launch_bounds__(NT)
    k_page_release(PagedDims pd, const int32_t* kv_len, const int32_t* keep_len,
                   const int32_t* page_table, int32_t* free_pages, const int32_t* n_free_p,
                   int32_t* n_free_out, int32_t* status) {
  __shared__ Shared sh;
  pdl_next();
  pdl_wait();
  const int ntile = (pd.N + TILE - 1) / TILE;
  const int n_free = *n_free_p;
  if (threadIdx.x == 0) sh.bad = 0;
  __syncthreads();
  // a request gives back up to 2^22 pages (2^25 positions, 8 a page), 2^11 requests
  // a tile: sums of at most 2^33, one plain 64-bit value
  auto one = [&](int s) {
    Need n{0, 0, 0, 0, 0};
    if (s >= pd.N) return n;
    const int kv = kv_len[s], keep = keep_len[s];
    if (keep < 0 || kv < keep || kv > pd.cap) {
      n.bad = 1;
      return n;
    }
    n.held = pages_of(keep, pd.ps);
    n.pages = pages_of(kv, pd.ps) - n.held;
    return n;
  };
  uint64_t none, pages = 0;
  if (ntile > 1) totals(sh, pd.N, one, none, pages);
  uint64_t pages0 = 0;
  Range mine{0, 0};
  int bad_page = 0;
  for (int tile = 0; tile < max(ntile, 1); ++tile) {
    const int s0 = tile * TILE;
    uint64_t v[PER];
    int bad = 0;
#pragma unroll
    for (int i = 0; i < PER; ++i) {
      const Need n = one(s0 + threadIdx.x * PER + i);
      v[i] = (uint64_t)n.pages;
      bad |= n.bad;
    }
    if (bad) atomicOr(&sh.bad, bad);
    const uint64_t sum = block_scan(sh, v);
    if (ntile <= 1) pages = sum;
    if (tile == 0) {
      const int code = sh.bad || n_free < 0 || n_free > pd.n_pages ? SGQA_ERR_BOUNDS
                       : pages + (uint64_t)n_free > (uint64_t)pd.n_pages ? SGQA_ERR_CAPACITY
                                                                        : SGQA_OK;
      if (blockIdx.x == 0 && threadIdx.x == 0) {
        if (code != SGQA_OK) report(status, code, 313);
        *n_free_out = code == SGQA_OK ? n_free + (int)pages : n_free;
      }
      if (code != SGQA_OK) return;
      mine = range_of((int64_t)pages, gridDim.x, blockIdx.x);
    }
    const int64_t a = max(mine.begin, (int64_t)pages0), b = min(mine.end, (int64_t)(pages0 + sum));
    const int n = min(TILE, pd.N - s0);
    for (int64_t e = a + threadIdx.x; e < b; e += NT) {
      const int64_t x = e - (int64_t)pages0;
      const int i = find(n, [&](int k) { return (int64_t)sh.excl[k]; }, x);
      const int s = s0 + i;
      const int col = pages_of(keep_len[s], pd.ps) + (int)(x - (int64_t)sh.excl[i]);
      const int page = page_table[(int64_t)s * pd.max_pages + col];
      bad_page |= page < 0 || page >= pd.n_pages;
      free_pages[n_free + e] = page;
    }
    pages0 += sum;
    __syncthreads();
  }
  if (__syncthreads_or(bad_page) && threadIdx.x == 0) free_pages[n_free + mine.begin] = kBadPage;
}

// The count of a release taken back where a CTA of its grid met a bad page.
__global__ void __launch_bounds__(kCheckNT)
    k_page_release_check(const int32_t* free_pages, const int32_t* n_free_p, int32_t* n_free_out,
                         unsigned grid, int32_t* status) {
  pdl_next();
  pdl_wait();
  const int n_free = *n_free_p;
  const int64_t pages = (int64_t)*n_free_out - n_free;  // (0: refused already)
  const Range r = range_of(pages, grid, threadIdx.x);
  const bool bad = threadIdx.x < grid && r.begin < r.end && free_pages[n_free + r.begin] == kBadPage;
  if (__syncthreads_or(bad) && threadIdx.x == 0) {
    report(status, SGQA_ERR_BOUNDS, 314);
    *n_free_out = n_free;
  }
}

}  // namespace

int launch_page_plan(const PagedDims& pd, const int32_t* q_len, const int32_t* kv_len,
                     const int32_t* free_pages, const int32_t* n_free, int32_t* page_table,
                     int32_t* q_start, int64_t* slot_map, int32_t* positions,
                     int32_t* n_free_out, int32_t* status, cudaStream_t st) {
  const int64_t want = ((int64_t)pd.T + NT - 1) / NT;
  const unsigned grid = (unsigned)(want < 1 ? 1 : want < kSMs ? want : kSMs);
  log_begin(SGQA_K_PAGES, st);
  const cudaError_t e = launch_pdl(k_page_plan, grid, NT, 0, st, pd, q_len, kv_len, free_pages, n_free,
                                   page_table, q_start, slot_map, positions, n_free_out, status);
  log_end(st);
  return e == cudaSuccess ? SGQA_OK : SGQA_ERR_CUDA;
}

int launch_page_release(const PagedDims& pd, const int32_t* kv_len, const int32_t* keep_len,
                        const int32_t* page_table, int32_t* free_pages, const int32_t* n_free,
                        int32_t* n_free_out, int32_t* status, cudaStream_t st) {
  const int64_t most = (int64_t)pd.N * pd.max_pages;  // pages the requests can hold
  const int64_t want = (most + NT - 1) / NT;
  const unsigned grid = (unsigned)(want < 1 ? 1 : want < kSMs ? want : kSMs);
  log_begin(SGQA_K_PAGES, st);
  cudaError_t e = launch_pdl(k_page_release, grid, NT, 0, st, pd, kv_len, keep_len, page_table,
                             free_pages, n_free, n_free_out, status);
  log_end(st);
  if (e != cudaSuccess) return SGQA_ERR_CUDA;
  log_begin(SGQA_K_PAGES, st);
  e = launch_pdl(k_page_release_check, 1, kCheckNT, 0, st, static_cast<const int32_t*>(free_pages),
                 n_free, n_free_out, grid, status);
  log_end(st);
  return e == cudaSuccess ? SGQA_OK : SGQA_ERR_CUDA;
}

}  // namespace sgqa
