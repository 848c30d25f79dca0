// How a ragged batch's attention work is laid out over persistent CTAs, and the
// merge of what the layout cuts.  Included by the attention kernels (each
// translation unit keeps its own copy).
//
// Who does what follows from the lengths alone.  An item is one or two query tiles
// of a (request, KV group).  All items lie one after another on a line, each as long
// as its work; the line is cut into one equal range per CTA, and a key tile belongs
// to the CTA whose range holds its place.  An item cut by a range's end leaves
// partial outputs, which a second kernel merges in order.  That balances any mix of
// lengths to a tile (64 requests with 500 to 32K keys: 356 us, the rate of a copy,
// against 440 us with whole chunks dealt out in turn), but the CTAs then read
// different keys at any one time.  When the keys that several items share exceed
// what L2 holds, full waves of whole items come first: item w grid + c goes to CTA
// c, so that neighbours read the same keys together, and only the rest of each
// request's items goes on the line.
#pragma once

#include "paged.h"

namespace sgqa {
namespace {

constexpr unsigned FULL = 0xffffffffu;

struct LineArgs {
  PagedDims pd;
  const int32_t *page_table, *q_start, *kv_len;
  int32_t* status;
  int groups;            // KV groups (parts of them, when a tile cannot hold a whole one)
  int head_parts;        // groups that a KV head's query heads are divided into
  int heads;             // query heads of a group (the last of a KV head: at most)
  int tpm;               // tokens of a query tile
  int tiles_per_item;    // query tiles of an item of longer requests: 1 or 2
  int over;              // key tiles that an item's beginning and end count for, >= 1 (a window: 2)
  int whole, part;       // key tiles of an uncut item and of a part, in small calls
  int uncut;             // no item is ever cut (caches are short): nothing to merge
  int tile_rows;         // rows from one query tile of a partial output to the next
  int slot_rows;
  float *opart, *lpart;  // partial outputs [slot][slot_rows][D], their lse [slot][slot_rows];
                         // CTA c's first piece in slot 2 c, its last in 2 c + 1
  int4* rec;             // [grid]: row0, tokens, group and parts of the item that CTA c
                         // begins and another ends
};

struct Piece {
  int s, g, row0, ntok;  // request, KV group, first token row, tokens
  int pos0;              // position of the first token
  int tb, n;             // first key tile, key tiles
  int lo, hi;            // keys that some row of the item sees
  int single;            // one query tile, key tiles alternate between the groups
  int slot;              // partial output (-1: the piece is the whole item)
  int end;               // no further piece
};

// Lengths on the line, in keys times a weight: a key tile takes kWt[..] * KB
// (two query tiles cost about half as much again as one), an item `over` tiles
// more for its beginning and end.  That also keeps every tile's place inside its
// item: the last tile may reach past the item's keys and, with a window, the first.
constexpr int kWtSingle = 2, kWtDouble = 3;
// Shortest range of a CTA, in key tiles of a single query tile.
constexpr int kLeastTiles = 2;
// A range that ends within kSnap tiles of an item's beginning or end leaves the
// item whole, when ranges are long enough for that to leave no part empty.
constexpr int kSnap = 2;
constexpr int kSnapTiles = 8;
// K and V bytes of the requests with several items above which waves are used:
// about half of L2.
constexpr int64_t kWaveBytes = int64_t(64) << 20;

// How a request is cut: items per KV group, item k taking A + B k on the line.
struct Cut {
  int q0, ql, kv;
  int ipt, items;
  int tw;               // a key tile on the line
  int tiles;            // most key tiles of an item
  int64_t A, B, head;   // head: all items of a KV group
};
// Parts of each of the request's items in a small call (see walk_line).
__device__ __forceinline__ int parts_of(const LineArgs& a, const Cut& c) {
  // (a tile of two query tiles takes twice the time)
  const int two = c.ipt > a.tpm ? 1 : 0;
  if (a.uncut || c.tiles <= a.whole >> two) return 1;
  return (int)((unsigned)(c.tiles + (a.part >> two) - 1) / (unsigned)(a.part >> two));
}
template <int KB>
__device__ __forceinline__ Cut cut_of(const LineArgs& a, int s, bool tell) {
  Cut c{0, 0, 0, 1, 0, 0, 0, 0, 0, 0};
  if (s >= a.pd.N) return c;
  const SeqLen q = seq_len_of(a.pd, a.q_start, a.kv_len, s, a.status, tell);
  c.q0 = q.q0;
  c.ql = q.ql;
  c.kv = q.kv;
  const bool one = q.ql <= a.tpm || a.tiles_per_item == 1;
  const int wt = one ? kWtSingle : kWtDouble;
  c.ipt = one ? a.tpm : a.tiles_per_item * a.tpm;
  c.items = q.ql <= a.tpm ? (q.ql > 0) : (int)((unsigned)(q.ql + c.ipt - 1) / (unsigned)c.ipt);
  c.tw = wt * KB;
  // keys an item sees, at most
  int keys = q.kv, slope = 0;
  if (a.pd.window > 0) {
    keys = min(q.kv, a.pd.window + c.ipt - 1);
  } else if (a.pd.causal && q.kv >= q.ql) {
    keys = q.kv - q.ql + c.ipt;
    slope = c.ipt;
  }
  // (a window's first key may lie anywhere in its tile)
  c.tiles = a.pd.window > 0 ? min((keys + KB - 1) / KB + 1, (q.kv + KB - 1) / KB) : (q.kv + KB - 1) / KB;
  c.A = (int64_t)(keys + a.over * KB) * wt;
  c.B = (int64_t)slope * wt;
  c.head = c.A * c.items + c.B * ((int64_t)c.items * (c.items - 1) / 2);
  return c;
}
// Where item k of a KV group begins, from the group's beginning.
__device__ __forceinline__ int64_t item_at(int64_t A, int64_t B, int k) {
  return A * k + B * ((int64_t)k * (k - 1) / 2);
}

// Item k of group g of request s as one piece (warp-uniform arguments).
template <int KB>
__device__ __forceinline__ Piece item_piece(const LineArgs& a, int s, int q0, int ql, int kv, int ipt,
                                            int g, int k) {
  Piece pc;
  pc.s = s;
  pc.g = g;
  pc.row0 = q0 + k * ipt;
  pc.ntok = min(ipt, ql - k * ipt);
  pc.pos0 = kv - ql + k * ipt;
  pc.hi = a.pd.causal ? max(0, min(kv, pc.pos0 + pc.ntok)) : kv;
  pc.lo = a.pd.window ? max(0, pc.pos0 + 1 - a.pd.window) : 0;
  pc.tb = pc.lo / KB;
  pc.n = pc.hi > pc.lo ? (pc.hi + KB - 1) / KB - pc.tb : 0;
  pc.single = pc.ntok <= a.tpm;
  pc.slot = -1;
  pc.end = 0;
  return pc;
}

__device__ __forceinline__ int64_t lane_scan(int64_t v) {
  const int lane = lane_id();
#pragma unroll 1
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t x = __shfl_up_sync(FULL, v, o);
    if (lane >= o) v += x;
  }
  return v;
}

// First query head of group g, and its number of heads.
__device__ __forceinline__ int first_head(const LineArgs& a, int g) {
  return g / a.head_parts * a.pd.G + g % a.head_parts * a.heads;
}
__device__ __forceinline__ int heads_of(const LineArgs& a, int g) {
  return min(a.heads, a.pd.G - g % a.head_parts * a.heads);
}

// 8 values of a row of O, from fp32
__device__ __forceinline__ void store_row8(__nv_bfloat16* p, const float* v) {
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]),
                                            pack_bf16x2(v[4], v[5]), pack_bf16x2(v[6], v[7]));
}
__device__ __forceinline__ void store_row8(float* p, const float* v) {
  reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
  reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

// Sums over the requests that every CTA computes for itself: the line, the part of
// it that waves would take, the keys that several items share, the pieces of a small
// call.  Exact integers, the same in every CTA.
struct LineSums {
  int64_t line, wave, keys, parts;
};
// cut: this thread's request (thread t of the block: request t); out: a row per warp.
template <int KB, int NT>
__device__ __forceinline__ void line_sums(const LineArgs& a, const Cut& cut, int64_t (*out)[4]) {
  const unsigned grid = gridDim.x;
  const int warp = warp_id(), lane = lane_id();
  int64_t line = 0, wave = 0, keys = 0, parts = 0;
  for (int s = threadIdx.x; s < a.pd.N; s += NT) {
    const Cut c = s < NT ? cut : cut_of<KB>(a, s, blockIdx.x == 0);
    line += c.head * a.groups;
    parts += (int64_t)parts_of(a, c) * c.items * a.groups;
    if (c.items > 1 && a.pd.window == 0) {
      const unsigned all = (unsigned)c.items * (unsigned)a.groups, in = all - all % grid;
      const unsigned g = in / (unsigned)c.items;
      wave += c.head * g + item_at(c.A, c.B, (int)(in - g * c.items));
      keys += c.kv;
    }
  }
  if (warp * 32 < a.pd.N) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
      line += __shfl_xor_sync(FULL, line, o);
      wave += __shfl_xor_sync(FULL, wave, o);
      keys += __shfl_xor_sync(FULL, keys, o);
      parts += __shfl_xor_sync(FULL, parts, o);
    }
  }
  if (lane == 0) {
    out[warp][0] = line;
    out[warp][1] = wave;
    out[warp][2] = keys;
    out[warp][3] = parts;
  }
}
template <int NT>
__device__ __forceinline__ LineSums add_sums(const LineArgs& a, const int64_t (*in)[4]) {
  LineSums s{0, 0, 0, 0};
  for (int i = 0; i < NT / 32 && i * 32 < a.pd.N; ++i) {
    s.line += in[i][0];
    s.wave += in[i][1];
    s.keys += in[i][2];
    s.parts += in[i][3];
  }
  return s;
}

// Calls publish(piece) for each of this CTA's pieces, warp-wide, until it returns
// false.  cut: the request of this lane (request lane of the batch).
template <int KB, typename Publish>
__device__ __forceinline__ bool walk_line(const LineArgs& a, Cut cut, const LineSums& sums,
                                          Publish publish, int4* rec) {
  const unsigned grid = gridDim.x;
  const int lane = lane_id();
  const bool waves = sums.keys * a.pd.Hkv * (2 * a.pd.d * a.pd.elem) > kWaveBytes;
  *rec = make_int4(0, 0, 0, 0);

  // Small calls: items of up to `whole` key tiles are not cut, longer ones into parts of
  // about `part` tiles, when that makes no more pieces than there are CTAs: one piece to
  // a CTA, the parts of an item to neighbours.
  if (sums.parts <= (int64_t)grid && !waves) {
    int before = 0;
    for (int s0 = 0; s0 < a.pd.N; s0 += 32) {
      if (s0 > 0) cut = cut_of<KB>(a, s0 + lane, false);
      const int parts = parts_of(a, cut), mine = parts * cut.items * a.groups;
      int inc = mine;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(FULL, inc, o);
        if (lane >= o) inc += x;
      }
      const unsigned m = __ballot_sync(FULL, before + inc > (int)blockIdx.x);
      if (m == 0) {
        before += __shfl_sync(FULL, inc, 31);
        continue;
      }
      const int l = __ffs(m) - 1;
      const unsigned np = __shfl_sync(FULL, (unsigned)parts, l);
      const unsigned items = __shfl_sync(FULL, (unsigned)cut.items, l);
      unsigned r = blockIdx.x - (unsigned)(before + __shfl_sync(FULL, inc - mine, l));
      const int j = (int)(r % np);
      r /= np;
      Piece pc = item_piece<KB>(a, s0 + l, __shfl_sync(FULL, cut.q0, l), __shfl_sync(FULL, cut.ql, l),
                                __shfl_sync(FULL, cut.kv, l), __shfl_sync(FULL, cut.ipt, l),
                                (int)(r / items), (int)(r % items));
      const int n = pc.n, len = (int)((unsigned)(n + np - 1) / np);
      const int t0 = min(n, j * len), t1 = min(n, t0 + len);
      if (n == 0 ? j > 0 : t1 == t0) return true;
      pc.tb += t0;
      pc.n = t1 - t0;
      if (pc.n < n) {
        pc.slot = 2 * blockIdx.x + (j > 0 ? 0 : 1);
        if (j == 0) *rec = make_int4(pc.row0, pc.ntok, pc.g, (n + len - 1) / len);
      }
      return publish(pc);
    }
    return true;
  }

  const int64_t total = sums.line - (waves ? sums.wave : 0);
  const int64_t snap_share = (int64_t)kSnapTiles * KB * kWtDouble;
  int64_t share = (total + grid - 1) / grid;
  if (share < kLeastTiles * KB * kWtSingle) share = kLeastTiles * KB * kWtSingle;
  bool ok = true;
  int held = 0;  // the 32 requests this warp's lanes hold
  auto hold = [&](int s0) {
    if (held != s0) cut = cut_of<KB>(a, s0 + lane, false);
    held = s0;
  };
  // items that go in waves, all KV groups of a request together
  auto wave_items = [&](const Cut& c) -> unsigned {
    if (!waves || c.items <= 1 || a.pd.window != 0) return 0u;
    const unsigned all = (unsigned)c.items * (unsigned)a.groups;
    return all - all % grid;
  };
  if (waves) {
    for (int s0 = 0; ok && s0 < a.pd.N; s0 += 32) {
      hold(s0);
      const unsigned in = wave_items(cut);
      for (unsigned m = __ballot_sync(FULL, in > 0); ok && m; m &= m - 1) {
        const int l = __ffs(m) - 1;
        const int q0 = __shfl_sync(FULL, cut.q0, l), ql = __shfl_sync(FULL, cut.ql, l);
        const int kv = __shfl_sync(FULL, cut.kv, l), ipt = __shfl_sync(FULL, cut.ipt, l);
        const unsigned items = __shfl_sync(FULL, (unsigned)cut.items, l);
        const unsigned lim = __shfl_sync(FULL, in, l);
        for (unsigned f = blockIdx.x; ok && f < lim; f += grid)
          ok = publish(item_piece<KB>(a, s0 + l, q0, ql, kv, ipt, (int)(f / items), (int)(f % items)));
      }
    }
  }
  // this CTA's range of the line
  const int64_t from = share * blockIdx.x;
  const int64_t to = min(total, from + share);
  int64_t base = 0;  // the place of the 32 requests
  for (int s0 = 0; ok && s0 < a.pd.N && base < to; s0 += 32) {
    hold(s0);
    const unsigned in = wave_items(cut);
    int64_t skip = 0;  // of the request's items, those in waves
    if (in > 0) {
      const unsigned g = in / (unsigned)cut.items;
      skip = cut.head * g + item_at(cut.A, cut.B, (int)(in - g * cut.items));
    }
    const int64_t len = cut.head * a.groups - skip;
    const int64_t inc = lane_scan(len);
    for (unsigned m = __ballot_sync(FULL, len > 0 && base + inc > from && base + inc - len < to);
         ok && m; m &= m - 1) {
      const int l = __ffs(m) - 1;
      const int q0 = __shfl_sync(FULL, cut.q0, l), ql = __shfl_sync(FULL, cut.ql, l);
      const int kv = __shfl_sync(FULL, cut.kv, l), ipt = __shfl_sync(FULL, cut.ipt, l);
      const int items = __shfl_sync(FULL, cut.items, l);
      const unsigned tw = __shfl_sync(FULL, (unsigned)cut.tw, l);
      const int64_t A = __shfl_sync(FULL, cut.A, l), B = __shfl_sync(FULL, cut.B, l);
      const int64_t head = __shfl_sync(FULL, cut.head, l);
      // the request's own coordinate of the line's place 0
      const int64_t zero = base + __shfl_sync(FULL, inc - len - skip, l);
      const int64_t begin = max(from, base + __shfl_sync(FULL, inc - len, l)) - zero;
      // the group and item that hold `begin`: an estimate, put right exactly
      int g = 0, k = 0;
      if (head <= begin) g = min((int)__fdividef((float)begin, (float)head), a.groups - 1);
      while (g > 0 && head * g > begin) --g;
      while (g < a.groups - 1 && head * (g + 1) <= begin) ++g;
      const int64_t in_group = begin - head * g;
      if (items > 1 && in_group >= A) {
        const float y = (float)in_group, fa = (float)A - 0.5f * (float)B, fb = (float)B;
        k = (int)(B == 0 ? __fdividef(y, fa)
                         : __fdividef(__fsqrt_rn(fa * fa + 2.0f * fb * y) - fa, fb));
        k = min(max(k, 0), items - 1);
      }
      while (k > 0 && head * g + item_at(A, B, k) > begin) --k;
      while (k < items - 1 && head * g + item_at(A, B, k + 1) <= begin) ++k;
      int64_t at = zero + head * g + item_at(A, B, k);  // the item's place
      while (ok && at < to) {
        Piece pc = item_piece<KB>(a, s0 + l, q0, ql, kv, ipt, g, k);
        const int64_t cost = A + B * k;
        // tiles whose places lie in [from, to): places at, at + tw, ...
        const int n = pc.n;
        auto tiles_before = [&](int64_t x) -> int {  // places before x, ends snapped
          if (x <= at) return 0;
          if (x - at >= cost || a.uncut) return n;  // (uncut: with its first tile)
          const int t = (int)min((unsigned)n, ((unsigned)(x - at) + tw - 1) / tw);
          return share < snap_share ? t : t <= kSnap ? 0 : t >= n - kSnap ? n : t;
        };
        const int t0 = tiles_before(from), t1 = tiles_before(to);
        if (n == 0 ? at >= from : t1 > t0) {
          pc.tb += t0;
          pc.n = t1 - t0;
          if (pc.n < n) {
            pc.slot = 2 * blockIdx.x + (t0 > 0 ? 0 : 1);
            if (t0 == 0) {  // begun here, continued by the CTAs up to the last tile's
              int c = blockIdx.x;
              while (tiles_before(min(total, share * (c + 1))) < n) ++c;
              *rec = make_int4(pc.row0, pc.ntok, pc.g, c - (int)blockIdx.x + 1);
            }
          }
          ok = publish(pc);
        }
        at += cost;
        if (++k == items) {
          k = 0;
          if (++g == a.groups) break;
        }
      }
    }
    base += __shfl_sync(FULL, inc, 31);
  }
  return ok;
}

// Merge of the cut items' partial outputs in order: lse = ln sum e^(lse_j), O =
// sum e^(lse_j - lse) O_j.  The item that CTA c begins has its parts in slots 2 c +
// 1, 2 c + 2, 2 c + 4, ...  All rows of all cut items are dealt out evenly, 8 columns
// to a thread.  What bounds it are the trips to memory in a row: record, then lse and
// values of four parts together (a running maximum in place of a first pass over the
// lse).  9 mixed requests: 11 us of 100, against 16 with the first pass and 16 columns a
// thread; one context of 8K: 6 against 9.  Eight parts together: 2 us more on the mixed
// requests (registers leave half the warps).
template <typename E, int D, int GRID, int NT>
__global__ void __launch_bounds__(NT) k_paged_merge(const __grid_constant__ LineArgs a, E* O,
                                                    float* lse) {
  static_assert(GRID <= NT, "a thread per CTA of the attention");
  __shared__ int4 rec[GRID];
  __shared__ int ends[GRID];  // rows of the items up to and with c
  __shared__ int warp_sum[NT / 32];
  const int tid = threadIdx.x, lane = tid & 31;
  pdl_next();
  pdl_wait();
  int4 r = make_int4(0, 0, 0, 0);
  if (tid < GRID) r = a.rec[tid];
  int inc = r.w > 1 ? r.y * a.heads : 0;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int x = __shfl_up_sync(FULL, inc, o);
    if (lane >= o) inc += x;
  }
  if (lane == 31) warp_sum[tid >> 5] = inc;
  __syncthreads();
  for (int w = 0; w < tid >> 5; ++w) inc += warp_sum[w];
  if (tid < GRID) {
    rec[tid] = r;
    ends[tid] = inc;
  }
  __syncthreads();
  const float ninf = -__int_as_float(0x7f800000);
  constexpr int W = 8, TPR = D / W, B = 4;  // columns of a thread, threads of a row, parts at a time
  const int col = lane % TPR * W;
  for (int row = blockIdx.x * (NT / TPR) + tid / TPR; row < ends[GRID - 1];
       row += gridDim.x * (NT / TPR)) {
    int c = 0, hi = GRID - 1;  // the first c with ends[c] > row
    while (c < hi) {
      const int mid = (c + hi) >> 1;
      if (ends[mid] > row)
        hi = mid;
      else
        c = mid + 1;
    }
    r = rec[c];
    const int in = row - (ends[c] - r.y * a.heads);
    const int tok = in / a.heads, h = in - tok * a.heads;
    if (h >= heads_of(a, r.z)) continue;
    const int tile = tok / a.tpm;
    const int64_t at = tile * a.tile_rows + (tok - tile * a.tpm) * a.heads + h;
    auto place = [&](int j) { return (int64_t)(2 * c + (j == 0 ? 1 : 2 * j)) * a.slot_rows + at; };
    // B parts at a time, all their loads at once
    float m = ninf, sw = 0.0f, acc[W];
#pragma unroll
    for (int e = 0; e < W; ++e) acc[e] = 0.0f;
    for (int j0 = 0; j0 < r.w; j0 += B) {
      float lj[B], mn = m;
      float4 v[B][W / 4];
#pragma unroll
      for (int b = 0; b < B; ++b) {
        lj[b] = ninf;
        if (j0 + b < r.w) {
          const int64_t part = place(j0 + b);
          const float4* src = reinterpret_cast<const float4*>(a.opart + part * D + col);
          lj[b] = a.lpart[part];
#pragma unroll
          for (int e = 0; e < W / 4; ++e) v[b][e] = src[e];
        }
      }
#pragma unroll
      for (int b = 0; b < B; ++b) mn = fmaxf(mn, lj[b]);
      const float base = mn == ninf ? 0.0f : mn;
      const float f = expf(m - base);
      sw *= f;
#pragma unroll
      for (int e = 0; e < W; ++e) acc[e] *= f;
#pragma unroll
      for (int b = 0; b < B; ++b) {
        if (lj[b] == ninf) continue;  // no part, or one in which the row saw nothing
        const float w = expf(lj[b] - base);
        sw += w;
#pragma unroll
        for (int e = 0; e < W / 4; ++e) {
          acc[4 * e] = fmaf(w, v[b][e].x, acc[4 * e]);
          acc[4 * e + 1] = fmaf(w, v[b][e].y, acc[4 * e + 1]);
          acc[4 * e + 2] = fmaf(w, v[b][e].z, acc[4 * e + 2]);
          acc[4 * e + 3] = fmaf(w, v[b][e].w, acc[4 * e + 3]);
        }
      }
      m = mn;
    }
    const float inv = sw == 0.0f ? 0.0f : 1.0f / sw;
    const int64_t t = r.x + tok, hq = first_head(a, r.z) + h;
#pragma unroll
    for (int e = 0; e < W; ++e) acc[e] *= inv;
#pragma unroll
    for (int e = 0; e < W; e += 8) store_row8(O + (t * a.pd.H + hq) * D + col + e, acc + e);
    if (col == 0) lse[hq * a.pd.T + t] = sw == 0.0f ? ninf : m + logf(sw);
  }
}


// The merge (none when no item can be cut).
template <typename E, int D, int GRID, int NT>
int launch_merge(const LineArgs& a, E* O, float* lse, cudaStream_t st) {
  if (a.uncut) return SGQA_OK;
  log_begin(SGQA_K_PAGED_ATTN, st);
  const cudaError_t e = launch_pdl(k_paged_merge<E, D, GRID, NT>, 4 * 152, NT, 0, st, a, O, lse);
  log_end(st);
  return e == cudaSuccess ? SGQA_OK : SGQA_ERR_CUDA;
}

// The workspace: records, lse and outputs of the partial results.
struct LineWs {
  size_t lpart, opart, bytes;
};
inline LineWs carve_line(int grid, int slot_rows, int d) {
  LineWs w;
  const size_t rows = (size_t)2 * grid * slot_rows;
  w.lpart = ((size_t)grid * 16 + 255) & ~size_t(255);
  w.opart = w.lpart + ((rows * 4 + 255) & ~size_t(255));
  w.bytes = w.opart + rows * d * 4;
  return w;
}
inline void set_line(LineArgs& a, const PagedDims& pd, const PagedAttnArgs& pa, const LineWs& w,
                     void* ws) {
  uint8_t* base = static_cast<uint8_t*>(ws);
  a.pd = pd;
  // windows and lengths end at cap: the sums of both stay in 32 bits
  if (a.pd.window > pd.cap) a.pd.window = pd.cap;
  a.page_table = pa.page_table;
  a.q_start = pa.q_start;
  a.kv_len = pa.kv_len;
  a.status = pa.status;
  a.rec = reinterpret_cast<int4*>(base);
  a.lpart = reinterpret_cast<float*>(base + w.lpart);
  a.opart = reinterpret_cast<float*>(base + w.opart);
}

}  // namespace
}  // namespace sgqa
