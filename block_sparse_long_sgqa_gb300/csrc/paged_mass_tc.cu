// Accumulated attention weights on tcgen05 tensor cores (bf16).
//
// S^T = K Q^T with the keys as the M = 128 rows of a product and up to 128 rows (token,
// head of the group) as its columns, so that a thread of the epilogue holds one key: the
// sum over the rows stays inside the thread, in fp32.  The rows' -lse comes in through the
// product too: a last step of K = 16 multiplies ones by -lse / scale in three bf16 terms (24
// bits, as many as its fp32 value has), so that what a thread reads is the exponent but for
// a factor.  (From shared memory every thread would have to read every row's: as many
// wavefronts as the operands, and the two together were 78 % of what it can give.)  An
// item is 256 keys of a (request, KV group), two products for each tile of rows: the keys
// stay in shared memory while the rows that see them go by.
//
// Layout over one CTA per SM: the items of all requests lie one after another on a line,
// each as long as the tokens that add to it (counted from the lengths alone) plus a fixed
// part for its keys; the line is cut into one equal range per CTA.  Items of more than
// kWhole tiles of rows may be cut; their parts' sums are added in order by a second
// kernel.  So results depend on the lengths only.
//
// Roles (12 warps): 0 walks this CTA's pieces and looks up their pages, 1 loads keys, 2
// loads rows of Q and their lse, 3 issues the products, 4-7 and 8-11 add up the weights of
// the two halves of the keys.  An adding thread takes all 128 columns of its key into
// registers before it begins, so that the next product but one can be written meanwhile
// (with four groups and 32 columns at a time a product waited for the exponentials of the
// one before: 1011 us on the chunks below).
//
// What bounds it.  64 single tokens over 500 to 32K keys, 8 groups: the keys' bytes, 178 us,
// 6.2 TB/s.  Chunks of 1024 and 2048 tokens over 4K to 16K keys, 64 heads: 975 us, 1145
// TFLOP/s; a tile of 256 keys by 128 rows takes 2200 cycles, 1200 of them products (the
// tensor pipe is 54 % active) and 1024 exponentials.  Neither is the limit by itself: with
// one product in nine the time is the same, with one exponential in eight it is 1650
// cycles, with both 1300, the way from the sums' last read of a tile through the barriers
// and the products to the next one.
#include "paged_mass.h"
#include "paged_tc.cuh"

namespace sgqa {
namespace {

constexpr unsigned FULL = 0xffffffffu;
constexpr int KB = 256, KH = 128;  // keys of an item, of a product
constexpr int BM = 128;            // rows of a tile, at most
constexpr int NTHREADS = 384;
constexpr int kGrid = 152;         // one CTA per SM
constexpr int NPC = 4;             // pieces in the ring
// Tiles of rows up to which an item is not cut.  Three requests of 100 tokens (7 tiles) over 8K to
// 16K keys: 65 us uncut, 68 cut (a limit of 2); of 300 tokens (19 tiles): 160 us cut (limits of 2, 8
// and 16), 173 uncut (32).
constexpr int kWhole = 8;
constexpr int kOver = 2;           // an item's keys, in tiles of rows

template <int D>
struct Cfg {
  static constexpr int KC = D / 64;                // 64-column halves
  static constexpr int TILE = KC * 128 * 128;      // bytes of 128 rows
  static constexpr int SK = D == 128 ? 3 : 7, SQ = 3;
  static constexpr int OFF_K = 0;
  static constexpr int OFF_Q = OFF_K + SK * TILE;
  // The last step's operands, 32 bytes a row: those of the SQ tiles of rows, then the ones.
  static constexpr int OFF_E = OFF_Q + SQ * TILE;
  static constexpr int OFF_PC = OFF_E + 128 * 128;
  static constexpr int PC = 192;                   // bytes of a piece: 128 for its pages
  static constexpr int OFF_BAR = OFF_PC + NPC * PC;
  static constexpr int NBAR = 2 * NPC + 2 * SK + 2 * SQ + 4 + 4 + 2;
  static constexpr int SMEM = OFF_BAR + NBAR * 8 + 16;
  static_assert(SMEM <= 232448, "shared memory of one CTA");
};

struct TcArgs : MassArgs {
  int tpm, tps;   // tokens of a tile of rows; of a small one (16 rows, or one token)
  int box;        // rows of a K box: gcd(page size, 128)
  float inv;      // 1 / scale
  int cuts;       // an item may be cut: the merge runs
  float* part;    // [2 kGrid][KB]: CTA c's first piece at 2 c, its last at 2 c + 1
  int4* rec;      // [kGrid]: request, group, first key and parts of the item that CTA c
                  // begins and another ends
};

struct Piece {     // 64 bytes at most
  int s, g, k0, kv;
  int first;       // position of the request's token 0
  int row0;        // first token row
  int i0, ntok;    // first token (of the request), tokens
  int q0;          // row of the request's token 0
  int slot;        // partial sums (-1: the piece is the whole item)
  int end;
};

static_assert(sizeof(Piece) <= 64, "ring slot");

// ------------------------------------------------------------------ the line
struct Cut {
  int q0, ql, kv, tiles;
  int rows;      // tokens that add to an item, at most
  int flat;      // items with that many, the others lose KB tokens each (causal)
  int64_t len;   // all items of a group
};
// Place of item kt in its group: over and tokens of those before it.
__device__ __forceinline__ int64_t item_at(const TcArgs& a, const Cut& c, int kt) {
  const int64_t k = kt, over = (int64_t)kOver * a.tpm;
  if (kt <= c.flat) return k * (over + c.rows);
  const int64_t f = c.flat;
  return k * over + f * c.rows + (k - f) * c.kv - KB * ((k * (k - 1) - f * (f - 1)) / 2);
}
__device__ __forceinline__ Cut cut_of(const TcArgs& a, int s, bool tell) {
  Cut c{0, 0, 0, 0, 0, 0, 0};
  if (s >= a.pd.N) return c;
  const SeqLen q = seq_len_of(a.pd, a.q_start, a.kv_len, s, a.status, tell);
  c.q0 = q.q0;
  c.ql = q.ql;
  c.kv = q.kv;
  c.tiles = (q.kv + KB - 1) / KB;
  c.rows = a.observe > 0 ? min(q.ql, a.observe) : q.ql;
  c.flat = c.tiles;
  if (a.pd.window > 0)
    c.rows = min(c.rows, a.pd.window + KB - 1);
  else if (a.pd.causal && q.kv >= q.ql)
    c.flat = min(c.tiles, (q.kv - c.rows) / KB + 1);
  c.len = item_at(a, c, c.tiles);
  return c;
}
// Item kt of a group: its first token and tiles of rows (0: nothing adds to it).
__device__ __forceinline__ void item_rows(const TcArgs& a, int ql, int kv, int kt, int& i0, int& i1,
                                          int& nt) {
  const int k0 = kt * KB;
  rows_of(a, ql, kv, k0, min(kv, k0 + KB), i0, i1);
  nt = (int)((unsigned)(i1 - i0 + a.tpm - 1) / (unsigned)a.tpm);
}

// Calls publish(piece) for each of this CTA's pieces, warp-wide, until it returns false.
template <typename Publish>
__device__ __forceinline__ bool walk(const TcArgs& a, int64_t total, Publish publish, int4* rec) {
  const int lane = lane_id();
  *rec = make_int4(0, 0, 0, 0);
  int64_t share = (total + gridDim.x - 1) / gridDim.x;
  share = max(share, (int64_t)(kOver + 1) * a.tpm);
  const int64_t from = share * blockIdx.x, to = min(total, from + share);
  const bool in_place = a.mass_in == a.mass_out;
  int64_t base = 0;
  for (int s0 = 0; s0 < a.pd.N && base < to; s0 += 32) {
    const Cut cut = cut_of(a, s0 + lane, false);
    const int64_t len = cut.len * a.pd.Hkv;
    int64_t inc = len;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t x = __shfl_up_sync(FULL, inc, o);
      if (lane >= o) inc += x;
    }
    for (unsigned m = __ballot_sync(FULL, len > 0 && base + inc > from && base + inc - len < to); m;
         m &= m - 1) {
      const int l = __ffs(m) - 1;
      Cut c;
      c.q0 = __shfl_sync(FULL, cut.q0, l);
      c.ql = __shfl_sync(FULL, cut.ql, l);
      c.kv = __shfl_sync(FULL, cut.kv, l);
      c.tiles = __shfl_sync(FULL, cut.tiles, l);
      c.rows = __shfl_sync(FULL, cut.rows, l);
      c.flat = __shfl_sync(FULL, cut.flat, l);
      c.len = __shfl_sync(FULL, cut.len, l);
      const int64_t zero = base + __shfl_sync(FULL, inc - len, l);
      const int64_t begin = max(from - zero, (int64_t)0);
      int g = (int)(begin / c.len);
      const int64_t in = begin - g * c.len;
      int kt = 0;  // the last item whose place is at most `in`
      for (int hi = c.tiles; hi - kt > 1;) {
        const int mid = (kt + hi) >> 1;
        if (item_at(a, c, mid) <= in)
          kt = mid;
        else
          hi = mid;
      }
      int64_t at = zero + g * c.len + item_at(a, c, kt);
      while (at < to) {
        int i0, i1, nt;
        item_rows(a, c.ql, c.kv, kt, i0, i1, nt);
        const int64_t cost = item_at(a, c, kt + 1) - item_at(a, c, kt);
        // tiles whose places lie before x: at, at + tpm, ..  (an item that is not cut goes
        // with its first)
        const int units = max(nt, 1);
        auto before = [&](int64_t x) -> int {
          if (x <= at) return 0;
          if (x - at >= cost || !a.cuts || nt <= kWhole) return units;
          return (int)min((int64_t)units, (x - at + a.tpm - 1) / a.tpm);
        };
        const int t0 = before(from), t1 = before(to);
        // (in place, entries that nothing adds to are there already)
        if (t1 > t0 && !(in_place && nt == 0 && (kt + 1) * KB <= c.kv - c.ql)) {
          Piece pc;
          pc.s = s0 + l;
          pc.g = g;
          pc.k0 = kt * KB;
          pc.kv = c.kv;
          pc.first = c.kv - c.ql;
          pc.q0 = c.q0;
          pc.i0 = i0 + t0 * a.tpm;
          pc.ntok = min(i1, i0 + t1 * a.tpm) - pc.i0;
          pc.row0 = c.q0 + pc.i0;
          pc.slot = -1;
          pc.end = 0;
          if (t1 - t0 < units) {
            pc.slot = 2 * blockIdx.x + (t0 > 0 ? 0 : 1);
            if (t0 == 0) {
              // begun here, continued by the CTAs up to that of the item's last tile (of those
              // there are, should the lengths have changed since the line was laid)
              const int e = (int)min((at + (int64_t)(units - 1) * a.tpm) / share, (int64_t)kGrid - 1);
              *rec = make_int4(pc.s, pc.g, pc.k0, e - (int)blockIdx.x + 1);
            }
          }
          if (!publish(pc)) return false;
        }
        at += cost;
        if (++kt == c.tiles) {
          kt = 0;
          if (++g == a.pd.Hkv) break;
        }
      }
    }
    base += __shfl_sync(FULL, inc, 31);
  }
  return true;
}

// The sum of a tile of rows for one key, row by row, where the sum from the products is NaN:
// a row whose lse is -infinity adds nothing, whatever it or the key holds, and once -infinity
// has been added to a product that is not finite nothing tells whose the NaN was.  (One of a row
// that counts is found here too, and ends the loop.)  At most 128 rows, some 0.1 ms, far from
// the waits' limit: the chunks above take 104 ms with a NaN in one left-out row of every tile, 975 us
// with finite rows left out.  Out of line and for NaN only: leaving such rows out where the products are
// read cost single tokens 16 % (176 to 204 us), a flag that led to a second copy of that
// code 11 %; this costs 0.3 to 0.5 % of both.
template <int D>
__device__ __noinline__ float again(const TcArgs& a, int at, int row0, int rows, int pos0, int key) {
  const int g = (int)((unsigned)at / (unsigned)a.pd.ps % (unsigned)a.pd.Hkv), G = a.pd.G;
  uint4 k[D / 8];
#pragma unroll
  for (int i = 0; i < D / 8; ++i)
    k[i] = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.K) + (int64_t)at * D)[i];
  float sum = 0.0f;
  for (int t = 0; t < rows; ++t) {
    if (!sees(a, pos0 + t, key)) continue;
    for (int h = g * G; h < g * G + G; ++h) {
      const float l = a.lse[(int64_t)h * a.pd.T + row0 + t];
      if (l == -__int_as_float(0x7f800000)) continue;
      const uint4* q = reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.Q) +
                                                      (int64_t)(row0 + t) * a.pd.qs + (int64_t)h * D);
      float s = 0.0f;
#pragma unroll
      for (int i = 0; i < D / 8; ++i) {
        const uint4 x = q[i], y = k[i];
        const uint32_t xs[4] = {x.x, x.y, x.z, x.w}, ys[4] = {y.x, y.y, y.z, y.w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s = fmaf(__uint_as_float(xs[j] << 16), __uint_as_float(ys[j] << 16), s);
          s = fmaf(__uint_as_float(xs[j] & 0xffff0000u), __uint_as_float(ys[j] & 0xffff0000u), s);
        }
      }
      sum += exp2f(fmaf(s, a.sl2, -l * 1.4426950408889634f));
      if (sum != sum) return sum;
    }
  }
  return sum;
}

template <int D>
__global__ void __launch_bounds__(NTHREADS, 1)
    k_mass(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap ms,
           const __grid_constant__ CUtensorMap mk, const __grid_constant__ TcArgs a) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  pdl_next();
  if (smem_u32(smem) & 1023u) {  // the operand tiles' swizzle needs it
    pdl_wait();
    if (threadIdx.x == 0) a.rec[blockIdx.x] = make_int4(0, 0, 0, 0);  // nothing to merge
    if (blockIdx.x == 0 && threadIdx.x == 0) report(a.status, SGQA_ERR_BOUNDS, 400);
    return;
  }
  auto piece_at = [&](int i) -> Piece& {
    return *reinterpret_cast<Piece*>(smem + C::OFF_PC + (i % NPC) * C::PC);
  };
  auto rows_at = [&](int i) -> int* {  // rows of the pool of the piece's boxes (-1: none)
    return reinterpret_cast<int*>(smem + C::OFF_PC + (i % NPC) * C::PC + 64);
  };
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* pc_full = bars;             // [NPC]
  uint64_t* pc_empty = pc_full + NPC;   // [NPC]
  uint64_t* k_full = pc_empty + NPC;    // [SK]
  uint64_t* k_empty = k_full + C::SK;   // [SK]
  uint64_t* q_full = k_empty + C::SK;   // [SQ]
  uint64_t* q_empty = q_full + C::SQ;   // [SQ]
  uint64_t* s_full = q_empty + C::SQ;   // [2 halves][2]
  uint64_t* s_empty = s_full + 4;       // [2][2]
  uint64_t* mma_done = s_empty + 4;
  uint64_t* stall_bar = mma_done + 1;   // nothing arrives on it
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::NBAR);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  const int warp = warp_id(), lane = lane_id();

  if (threadIdx.x == 0) {
    for (int i = 0; i < NPC; ++i) {
      mbar_init(&pc_full[i], 1);
      mbar_init(&pc_empty[i], 11);  // K, Q, products, 8 adding warps
    }
    for (int i = 0; i < C::SK; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < C::SQ; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
    }
    for (int i = 0; i < 4; ++i) {
      mbar_init(&s_full[i], 1);
      mbar_init(&s_empty[i], 4);
    }
    mbar_init(mma_done, 1);
    mbar_init(stall_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 3) tmem_alloc(tmem_slot, 512);
  // rows of zeros but for the ones (1, 1, 1, 0, ..): 16 bytes a place, swizzled
  for (int x = threadIdx.x; x < 128 * 8; x += NTHREADS) {
    const int row = x >> 3, chunk = (x & 7) ^ (row & 7);
    *reinterpret_cast<uint4*>(smem + C::OFF_E + x * 16) =
        chunk == 2 * C::SQ ? make_uint4(0x3f803f80u, 0x3f80u, 0, 0) : make_uint4(0, 0, 0, 0);
  }
  fence_proxy_async_smem();
  pdl_wait();
  if (lane == 0 && (warp == 1 || warp == 2)) {
    tma_prefetch_desc(warp == 1 ? &mk : &mq);
    if (warp == 2) tma_prefetch_desc(&ms);
  }
  // the line's length: an exact integer sum, the same in every CTA
  int64_t* sums = reinterpret_cast<int64_t*>(smem + C::OFF_K);
  {
    int64_t line = 0;
    for (int s = threadIdx.x; s < a.pd.N; s += NTHREADS)
      line += cut_of(a, s, blockIdx.x == 0).len * a.pd.Hkv;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) line += __shfl_xor_sync(FULL, line, o);
    if (lane == 0) sums[warp] = line;
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const GiveUp up{abort_flag};
  int64_t total = 0;
  for (int w = 0; w < NTHREADS / 32; ++w) total += sums[w];
  __syncthreads();  // (the sums' place is used again)

  constexpr int kRegsLess = 88, kRegsMore = 208;
  static_assert(256 * kRegsMore + 128 * kRegsLess <= NTHREADS * 168, "the launch's registers");
  if (warp < 4) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLess));
  if (warp == 0) {
    // ================================================================== pieces
    // A piece goes out when the next one has been found, so that the trip to the page
    // table passes meanwhile.
    int pub = 0;
    const int nbox = KB / a.box;
    Piece held{};
    int page = 0, off = -1;  // of this lane's box (off -1: none)
    bool holds = false;
    auto put = [&]() -> bool {  // the piece held
      int at = -1;
      if (off >= 0) {
        if (page >= 0 && page < a.pd.n_pages)
          at = (page * a.pd.Hkv + held.g) * a.pd.ps + off;
        else
          report(a.status, SGQA_ERR_BOUNDS, 391);
      }
      if (!warp_wait(&pc_empty[pub % NPC], (uint32_t)(((pub / NPC) & 1) ^ 1), up, 401)) return false;
      rows_at(pub)[lane] = at;
      if (lane == 0) piece_at(pub) = held;
      __syncwarp();
      if (lane == 0) mbar_arrive(&pc_full[pub % NPC]);
      ++pub;
      return true;
    };
    auto publish = [&](const Piece& pc) -> bool {
      // the pages of its boxes, one a lane (a box of 8 keys at least: 32 boxes at most)
      int next = 0, noff = -1;
      const int key = pc.k0 + lane * a.box;
      if (!pc.end && lane < nbox && key < pc.kv) {
        const int pi = (int)((unsigned)key / (unsigned)a.pd.ps);
        next = a.page_table[(int64_t)pc.s * a.pd.max_pages + pi];
        noff = key - pi * a.pd.ps;
      }
      if (holds && !put()) return false;
      held = pc;
      page = next;
      off = noff;
      holds = true;
      return true;
    };
    int4 rec;
    const bool ok = walk(a, total, publish, &rec);
    if (lane == 0) a.rec[blockIdx.x] = rec;  // for the merge
    if (ok) {
      Piece pc{};
      pc.end = 1;
      if (publish(pc)) put();
    }
  } else if (warp == 1) {
    // ==================================================================== keys
    const int per_half = KH / a.box;
    const int rows_total = a.pd.n_pages * a.pd.Hkv * a.pd.ps;
    int cnt = 0;
    bool ok = true;
    for (int i = 0; ok; ++i) {
      ok = warp_wait(&pc_full[i % NPC], (uint32_t)((i / NPC) & 1), up, 402);
      if (!ok) break;
      const Piece pc = piece_at(i);
      int at[2];
      bool on[2];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        on[h] = lane < per_half && pc.k0 + h * KH + lane * a.box < pc.kv;
        at[h] = on[h] ? rows_at(i)[h * per_half + lane] : -1;
        if (at[h] < 0) at[h] = rows_total;  // outside the pool: zeros
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&pc_empty[i % NPC]);
      if (pc.end) break;
      if (pc.ntok == 0) continue;
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const int boxes = __popc(__ballot_sync(FULL, on[h]));
        if (boxes == 0) continue;
        const int sl = cnt % C::SK;
        ok = warp_wait(&k_empty[sl], (uint32_t)(((cnt / C::SK) & 1) ^ 1), up, 403);
        if (!ok) break;
        if (lane == 0) mbar_expect_tx(&k_full[sl], (uint32_t)(boxes * a.box * 128 * C::KC));
        __syncwarp();
        if (on[h])
          for (int c = 0; c < C::KC; ++c)
            tma_load_2d(smem + C::OFF_K + sl * C::TILE + c * (KH * 128) + lane * a.box * 128, &mk,
                        &k_full[sl], c * 64, at[h]);
        __syncwarp();
        ++cnt;
      }
    }
    // copies land before the CTA ends, whoever gives up and whenever
    if (lane == 0)
      for (int k = 0; k < C::SK; ++k) {
        const int uses = cnt / C::SK + (k < cnt % C::SK ? 1 : 0);
        if (uses > 0) mbar_wait_drain(&k_full[k], (uint32_t)((uses - 1) & 1), a.status, 411);
      }
  } else if (warp == 2) {
    // ====================================================== rows of Q, their lse
    const float ninf = -__int_as_float(0x7f800000);
    const int G = a.pd.G;
    int cnt = 0;
    bool ok = true;
    for (int i = 0; ok; ++i) {
      ok = warp_wait(&pc_full[i % NPC], (uint32_t)((i / NPC) & 1), up, 404);
      if (!ok) break;
      const Piece pc = piece_at(i);
      __syncwarp();
      if (lane == 0) mbar_arrive(&pc_empty[i % NPC]);
      if (pc.end) break;
      const bool small = pc.ntok <= a.tps;
      const int step = small ? a.tps : a.tpm;
      // rows lane, lane + 32, .. of a tile: their lse, asked for a tile ahead
      float l[4];
      auto fetch = [&](int t) {
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          const int r = lane + 32 * x, rt = r / G;
          l[x] = 0.0f;
          if (rt < step && t + rt < pc.ntok)
            l[x] = a.lse[(int64_t)(pc.g * G + r - rt * G) * a.pd.T + pc.row0 + t + rt];
        }
      };
      if (pc.ntok > 0) fetch(0);
      for (int t = 0; t < pc.ntok; t += step, ++cnt) {
        const int sl = cnt % C::SQ;
        ok = warp_wait(&q_empty[sl], (uint32_t)(((cnt / C::SQ) & 1) ^ 1), up, 405);
        if (!ok) break;
#pragma unroll
        for (int x = 0; x < 4; ++x) {
          // three terms, each the bf16 nearest to what is left; a row that saw nothing adds
          // nothing (2 to the -inf, or by again() where its product is not finite)
          const float v = l[x] == ninf ? ninf : -(l[x] * a.inv);
          const float hi = __bfloat162float(__float2bfloat16_rn(v));
          const bool more = fabsf(hi) < -ninf;
          const float mid = more ? __bfloat162float(__float2bfloat16_rn(v - hi)) : 0.0f;
          const float low = more ? v - hi - mid : 0.0f;
          const int row = lane + 32 * x;
          *reinterpret_cast<uint4*>(smem + C::OFF_E + row * 128 + (((2 * sl) ^ (row & 7)) << 4)) =
              make_uint4(pack_bf16x2(hi, mid), pack_bf16x2(low, 0.0f), 0, 0);
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_expect_tx(&q_full[sl], (uint32_t)(C::KC * 128 * G * step));
          for (int c = 0; c < C::KC; ++c)
            tma_load_3d(smem + C::OFF_Q + sl * C::TILE + c * (BM * 128), small ? &ms : &mq,
                        &q_full[sl], c * 64, pc.g * G, pc.row0 + t);
        }
        __syncwarp();
        if (t + step < pc.ntok) fetch(t + step);
      }
    }
    if (lane == 0)
      for (int k = 0; k < C::SQ; ++k) {
        const int uses = cnt / C::SQ + (k < cnt % C::SQ ? 1 : 0);
        if (uses > 0) mbar_wait_drain(&q_full[k], (uint32_t)((uses - 1) & 1), a.status, 412);
      }
  } else {
    // ================================================================ products
    // (the whole warp walks the loop and one elected lane issues: uniform registers)
    const bool leader = elect_one();
    const uint32_t lk = (smem_u32(smem + C::OFF_K) >> 4) | (1u << 16);
    const uint32_t lq = (smem_u32(smem + C::OFF_Q) >> 4) | (1u << 16);
    const uint32_t le = (smem_u32(smem + C::OFF_E) >> 4) | (1u << 16);
    int ks = 0, qs = 0;             // slots of the next keys and rows
    uint32_t kph = 0, qph = 0;      // and their phases
    uint32_t buf = 0;               // tensor memory of the next tile of rows
    uint32_t eph = 15;              // phases of s_empty to wait for, a bit each
    bool first = true, ok = true;
    for (int i = 0; ok; ++i) {
      ok = warp_poll(&pc_full[i % NPC], (uint32_t)((i / NPC) & 1), up, 406);
      if (!ok) break;
      const Piece& pc = piece_at(i);
      // (reductions of equal values: uniform registers)
      const int ntok = __reduce_max_sync(FULL, pc.ntok), end = __reduce_max_sync(FULL, pc.end);
      const int halves = __reduce_max_sync(FULL, pc.kv - pc.k0 > KH ? 2 : 1);
      __syncwarp();
      if (leader) mbar_arrive(&pc_empty[i % NPC]);
      if (end) break;
      // Debug request (host-set status[3]): the first piece waits on a barrier that
      // nothing arrives on, so the pipeline gives up (detail 420) with copies in flight.
      if (first && blockIdx.x == 0 && debug_request(a.status) == SGQA_DEBUG_STALL)
        ok = warp_wait(stall_bar, 0, up, 420, kDebugStallNs);
      first = false;
      for (int t = 0; ok && t < ntok; t += a.tpm) {
        const int n = min(a.tpm, ntok - t) * a.pd.G;
        const uint32_t idesc = idesc_bf16_f32(KH, (uint32_t)((n + 15) & ~15), 0, 0);
        ok = warp_poll(&q_full[qs], qph, up, 407);
        if (!ok) break;
        const uint32_t lb = lq + (uint32_t)qs * (C::TILE / 16);
        for (int h = 0; h < halves; ++h) {
          const int sb = h * 2 + (int)buf;
          int sl = ks + h;
          uint32_t ph = kph;
          if (sl >= C::SK) {
            sl -= C::SK;
            ph ^= 1;
          }
          ok = (t > 0 || warp_poll(&k_full[sl], ph, up, 408)) &&
               warp_poll(&s_empty[sb], (eph >> sb) & 1, up, 409);
          if (!ok) break;
          eph ^= 1u << sb;
          tc_fence_after();
          const uint32_t la = lk + (uint32_t)sl * (C::TILE / 16), d = tmem + (uint32_t)sb * 128;
          if (leader) {
#pragma unroll
            for (int kk = 0; kk < D / 16; ++kk) {
              const uint32_t off = (kk >> 2) * (128 * 128 / 16) + (kk & 3) * 2;
              umma_ss(d, la + off, lb + off, idesc, kk > 0);
            }
            // (last, so that its size counts in one rounding of the sum only)
            umma_ss(d, le + 2 * C::SQ, le + 2 * (uint32_t)qs, idesc, 1);
            umma_commit(&s_full[sb]);
            if (t + a.tpm >= ntok) umma_commit(&k_empty[sl]);
            if (h == halves - 1) umma_commit(&q_empty[qs]);
          }
          __syncwarp();
        }
        buf ^= 1;
        if (++qs == C::SQ) {
          qs = 0;
          qph ^= 1;
        }
      }
      if (ntok > 0) {
        ks += halves;
        if (ks >= C::SK) {
          ks -= C::SK;
          kph ^= 1;
        }
      }
    }
    if (leader) {
      umma_commit(mma_done);
      mbar_wait_drain(mma_done, 0, a.status, 413);
    }
    __syncwarp();
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsMore));
    // ================================================================= weights
    const int half = (warp - 4) >> 2, quad = warp & 3;
    const int r = quad * 32 + lane;  // key of the half
    const uint32_t tS = tmem + (static_cast<uint32_t>(quad * 32) << 16) + (uint32_t)half * 256;
    const uint64_t sl2x2 = f2_pack(a.sl2, a.sl2);
    const int G = a.pd.G;
    uint32_t buf = 0;  // tensor memory of the next tile of rows
    uint32_t ph = 0;   // phases of s_full, a bit each
    // A piece as this thread needs it, with what its key's entry holds: asked for when the
    // piece before it is begun, if it is known by then.
    struct Mine {
      int key, kv, first, i0, row0, ntok, slot, end, here, at, pos;
      float old;
    };
    auto take = [&](int i) -> Mine {
      const Piece& pc = piece_at(i);
      Mine m;
      m.key = pc.k0 + half * KH + r;
      m.kv = pc.kv;
      m.first = pc.first;
      m.i0 = pc.i0;
      m.row0 = pc.row0;
      m.ntok = pc.ntok;
      m.slot = pc.slot;
      m.end = pc.end;
      m.here = pc.k0 + half * KH < pc.kv;
      m.at = -1;
      m.old = 0.0f;
      m.pos = 0;
      const int row0 = pc.q0;
      if (!m.end && m.key < m.kv) {
        const int b = (half * KH + r) / a.box;
        m.at = rows_at(i)[b];
        if (m.at >= 0) m.at += half * KH + r - b * a.box;
      }
      __syncwarp();
      if (lane == 0) mbar_arrive(&pc_empty[i % NPC]);
      if (m.at >= 0 && m.slot < 0) {
        const int fresh = m.key - m.first;
        if (fresh < 0)
          m.old = a.mass_in[m.at];
        else if (a.pos_pages != nullptr)
          m.pos = a.positions[row0 + fresh];
      }
      return m;
    };
    bool ok = warp_wait(&pc_full[0], 0, up, 421);
    Mine m;
    if (ok) m = take(0);
    for (int i = 0; ok && !m.end; ++i) {
      uint64_t* next_full = &pc_full[(i + 1) % NPC];
      const uint32_t next_phase = (uint32_t)(((i + 1) / NPC) & 1);
      const bool known = __all_sync(FULL, mbar_test(next_full, next_phase));
      Mine n;
      if (known) n = take(i + 1);
      float sum = 0.0f;
      for (int t = 0; t < m.ntok; t += a.tpm, buf ^= 1) {
        if (!m.here) continue;
        ok = warp_wait(&s_full[half * 2 + buf], (ph >> buf) & 1, up, 423);
        if (!ok) break;
        ph ^= 1u << buf;
        tc_fence_after();
        const int rows = min(a.tpm, m.ntok - t), nr = rows * G;
        // rows [c0, c1) of the tile see the key
        int c0 = 0, c1 = nr;
        if (m.key < m.kv) {
          const int d = m.key - m.first - (m.i0 + t);
          if (a.pd.causal) c0 = min(max(d, 0), rows) * G;
          if (a.pd.window > 0) c1 = min(max(d + a.pd.window, 0), rows) * G;
        }
        auto release = [&]() {  // the tile has been read: its place may be written
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_empty[half * 2 + buf]);
        };
        uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
        // (of groups that divide 128: other tiles have fewer rows, and go the second way; chunks
        // of 28 heads on 4 486 us, of 32 on 4 494)
        const bool whole = __all_sync(FULL, c0 == 0 && c1 == BM);
        if (whole) {
          uint32_t v[128];
#pragma unroll
          for (int w = 0; w < 4; ++w)
            tmem_ld32(tS + buf * 128 + w * 32, *reinterpret_cast<uint32_t(*)[32]>(&v[w * 32]));
          tmem_wait_ld();
          release();
          // in stages, so that an exponential's latency lies under the others: products of a
          // group, its exponentials, the sums of the group before
          constexpr int GR = 16;
          float p[BM];
#pragma unroll
          for (int g = 0; g <= BM; g += GR) {
            if (g < BM) {
#pragma unroll
              for (int e = g; e < g + GR; e += 2)
                f2_unpack(f2_mul(f2_pack(__uint_as_float(v[e]), __uint_as_float(v[e + 1])), sl2x2), p[e],
                          p[e + 1]);
#pragma unroll
              for (int e = g; e < g + GR; ++e) p[e] = ex2(p[e]);
            }
            if (g > 0) {
#pragma unroll
              for (int e = g - GR; e < g; e += 2)
                acc[(e >> 1) & 3] = f2_add(acc[(e >> 1) & 3], f2_pack(p[e], p[e + 1]));
            }
          }
        } else if (nr > 32) {
          // Some rows do not see the key, or the tile is not full: 32 columns at a time, by
          // selection (what a row does not see may be NaN), away from the code above, which
          // the selections slowed down where no row needed them.
#pragma unroll 1
          for (int c = 0; c < nr; c += 32) {
            uint32_t v[32];
            tmem_ld32(tS + buf * 128 + c, v);
            tmem_wait_ld();
            const uint32_t see = seen_bits(c, c0, c1);
#pragma unroll
            for (int e = 0; e < 32; e += 2) {
              float x0, x1;
              f2_unpack(f2_mul(f2_pack(__uint_as_float(see >> e & 1u ? v[e] : 0xff800000u),
                                       __uint_as_float(see >> (e + 1) & 1u ? v[e + 1] : 0xff800000u)),
                               sl2x2), x0, x1);
              acc[(e >> 1) & 3] = f2_add(acc[(e >> 1) & 3], f2_pack(ex2(x0), ex2(x1)));
            }
          }
          release();
        } else {
          // Few rows, 8 at a time in a short loop: code that runs once a piece costs its way
          // into the instruction cache (unrolled over 32 columns it took 1000 cycles for 8
          // rows, and 64 single tokens 190 us in place of 176).
#pragma unroll 1
          for (int c = 0; c < nr; c += 8) {
            uint32_t v[8];
            tmem_ld8(tS + buf * 128 + c, v);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 8; e += 2) {
              const float p0 = ex2(__uint_as_float(v[e]) * a.sl2);
              const float p1 = ex2(__uint_as_float(v[e + 1]) * a.sl2);
              acc[(e >> 1) & 3] = f2_add(acc[(e >> 1) & 3],
                                         f2_pack(c + e >= c0 && c + e < c1 ? p0 : 0.0f,
                                                 c + e + 1 >= c0 && c + e + 1 < c1 ? p1 : 0.0f));
            }
          }
          release();
        }
        float s0, s1;
        f2_unpack(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), s0, s1);
        float add = s0 + s1;
        if (__any_sync(FULL, add != add)) {
          if (add != add && m.at >= 0)
            add = again<D>(a, m.at, m.row0 + t, rows, m.first + m.i0 + t, m.key);
          __syncwarp();
        }
        sum += add;
      }
      if (!ok) break;
      if (m.here) {
        if (m.slot >= 0) {
          a.part[(int64_t)m.slot * KB + half * KH + r] = sum;
        } else if (m.at >= 0) {
          const bool fresh = m.key >= m.first;
          a.mass_out[m.at] = fresh ? sum : m.old + sum;
          if (fresh && a.pos_pages != nullptr) a.pos_pages[m.at] = m.pos;
        }
      }
      if (!known) {
        ok = warp_wait(next_full, next_phase, up, 421);
        if (!ok) break;
        n = take(i + 1);
      }
      m = n;
    }
    tc_fence_before();
  }
  __syncthreads();
  if (threadIdx.x == 0 && *abort_flag != 0) report(a.status, SGQA_ERR_TIMEOUT, *abort_flag);
  if (warp == 3) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// The sums of cut items: the item that CTA c begins has its parts in slots 2 c + 1,
// 2 c + 2, 2 c + 4, ..., added in that order; a block an item, a thread a key.
__global__ void __launch_bounds__(KB) k_mass_merge(const __grid_constant__ TcArgs a) {
  pdl_next();
  pdl_wait();
  const int c = blockIdx.x;
  const int4 rec = a.rec[c];
  if (rec.w <= 1) return;
  const SeqLen q = seq_len_of(a.pd, a.q_start, a.kv_len, rec.x, a.status, false);
  const int key = rec.z + threadIdx.x;
  if (key >= q.kv) return;
  float sum = a.part[(int64_t)(2 * c + 1) * KB + threadIdx.x];
  constexpr int B = 8;  // parts loaded together
  for (int j0 = 1; j0 < rec.w; j0 += B) {
    float v[B];
#pragma unroll
    for (int b = 0; b < B; ++b)
      v[b] = j0 + b < rec.w ? a.part[(int64_t)(2 * (c + j0 + b)) * KB + threadIdx.x] : 0.0f;
#pragma unroll
    for (int b = 0; b < B; ++b) sum += v[b];
  }
  MassTile t;
  t.s = rec.x;
  t.g = rec.y;
  t.q0 = q.q0;
  t.ql = q.ql;
  t.kv = q.kv;
  write_entry(a, a.page_table + (int64_t)rec.x * a.pd.max_pages, t, key, sum);
}

// Q [T][H][d] with row stride qs, boxes of `tokens` tokens of a group's heads.
bool q_map(const PagedDims& pd, int tokens, const void* Q, CUtensorMap* m) {
  auto fn = tmap_encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[3] = {(cuuint64_t)pd.d, (cuuint64_t)pd.H, (cuuint64_t)(pd.T > 0 ? pd.T : 1)};
  cuuint64_t str[2] = {(cuuint64_t)pd.d * 2, (cuuint64_t)pd.qs * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)pd.G, (cuuint32_t)tokens}, es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(Q), dims, str, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

constexpr size_t kRecBytes = (kGrid * sizeof(int4) + 255) & ~size_t(255);

template <int D>
int launch(const TcArgs& a, cudaStream_t st) {
  using C = Cfg<D>;
  const PagedDims& pd = a.pd;
  CUtensorMap mq, ms, mk;
  if (!q_map(pd, a.tpm, a.Q, &mq) || !q_map(pd, a.tps, a.Q, &ms) ||
      !make_tmap_2d_bf16(&mk, a.K, D, (uint64_t)pd.n_pages * pd.Hkv * pd.ps, D * 2, 64,
                         (uint32_t)a.box))
    return SGQA_ERR_CUDA;
  if (cudaFuncSetAttribute(k_mass<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) !=
      cudaSuccess)
    return SGQA_ERR_CUDA;
  log_begin(SGQA_K_MASS, st);
  cudaError_t e = launch_pdl(k_mass<D>, kGrid, NTHREADS, C::SMEM, st, mq, ms, mk, a);
  log_end(st);
  if (e != cudaSuccess) return SGQA_ERR_CUDA;
  if (!a.cuts) return SGQA_OK;
  log_begin(SGQA_K_MASS, st);
  e = launch_pdl(k_mass_merge, kGrid, KB, 0, st, a);
  log_end(st);
  return e == cudaSuccess ? SGQA_OK : SGQA_ERR_CUDA;
}

}  // namespace

size_t mass_tc_ws_bytes(const PagedDims&) { return kRecBytes + (size_t)2 * kGrid * KB * 4; }

int launch_mass_tc(const MassArgs& m, void* ws, cudaStream_t st) {
  TcArgs a;
  static_cast<MassArgs&>(a) = m;
  const PagedDims& pd = a.pd;
  a.tpm = BM / pd.G;
  a.tps = pd.G >= 16 ? 1 : 16 / pd.G;
  // an item has at most all tokens' tiles
  a.cuts = ((int64_t)pd.T + a.tpm - 1) / a.tpm > kWhole;
  a.rec = reinterpret_cast<int4*>(ws);
  a.part = reinterpret_cast<float*>(static_cast<uint8_t*>(ws) + kRecBytes);
  int x = pd.ps, y = KH;
  while (y) {
    const int t = x % y;
    x = y;
    y = t;
  }
  a.box = x;
  a.inv = 1.0f / pd.scale;
  if (pd.T == 0) a.Q = a.K;  // (no row is loaded, but a map wants an address)
  return pd.d == 128 ? launch<128>(a, st) : launch<64>(a, st);
}

}  // namespace sgqa
