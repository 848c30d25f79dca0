// Ragged attention over the paged pool on tcgen05 tensor cores (bf16).
//
// Online softmax in one pass over a request's keys, 128 at a time: S = Q K^T
// into tensor memory, P = 2^(S scale log2 e - m) rounded to bf16 (m: a running
// reference maximum, raised only when a tile exceeds it by much), O += P V, and
// at the end O / l with l the sum of P in fp32.  P is rounded because both operands
// of a product have one type: each weight is off by at most 2^-8 of itself, which for
// random values adds 1.5e-3 of O (root mean square) to the 1.65e-3 that O's own rounding
// costs; two bf16 terms of P would double P V.
//
// A query tile is 128 / G tokens with their G query heads as the M = 128 rows of
// every product, so each K and V tile that is read serves the whole KV group.
// paged_line.cuh lays the work out over one CTA per SM, in items of up to two query
// tiles.  Requests with one query tile (single tokens, drafts) let the two softmax
// groups take alternate key tiles; longer ones give each group its own query tile,
// and each key tile serves both.
//
// Roles (12 warps): 0 walks this CTA's pieces, publishes them in a ring and
// loads Q; 1 and 2 load K and V tiles through the page table (TMA boxes of
// gcd(page size, 128) rows, one lane each); 3 issues the products; 4-7 and 8-11
// are the softmax groups, one thread per row, and write the outputs.  All rings
// run on across pieces, so the next piece's keys load during the current one.
//
// What bounds it.  Single tokens over long caches: the bytes of K and V (1M keys of 8
// heads in 590 us, 7.3 TB/s; 64 ragged contexts in 356 us, 6.9 TB/s).  Chunks: the
// chain of a group from S to P to the products that give the next S, 2970 cycles for
// the 2 x 1050 that the products of both groups take (4096 tokens over 36K keys, 64
// heads: 3.05 to 3.1 ms, 1510 TFLOP/s; the tensor pipe is 66 % active).  Short pieces (a
// window of 512 keys, 167 us): 5 of a piece's 21 thousand cycles pass between the last
// P and the next first S, and three of its five key tiles are masked.
#include "paged_line.cuh"

namespace sgqa {
namespace {

constexpr int BM = 128;   // rows of a query tile
constexpr int KB = 128;   // keys of a tile
constexpr int NPC = 4;    // pieces in the ring
constexpr int NTHREADS = 384;
constexpr int kGrid = 152;  // one CTA per SM

// A tile's maximum may exceed the reference by a factor of 2^kLazy before the
// reference is raised and O rescaled: bf16 and fp32 hold weights up to 2^kLazy with
// the same relative precision as weights up to 1.
constexpr float kLazy = 8.0f;

template <int D>
struct Cfg {
  static constexpr int KC = D / 64;                    // 64-column halves
  static constexpr int TILE = KC * BM * 128;           // bytes of a 128-row operand tile
  static constexpr int SK = D == 128 ? 3 : 6, SV = D == 128 ? 2 : 5;
  static constexpr int OFF_Q = 0;                      // two query tiles
  static constexpr int OFF_K = OFF_Q + 2 * TILE;
  static constexpr int OFF_V = OFF_K + SK * TILE;
  static constexpr int OFF_X = OFF_V + SV * TILE;      // maxima and sums [2][2][BM] floats
  static constexpr int OFF_PC = OFF_X + 4 * BM * 4;    // piece ring
  static constexpr int OFF_BAR = OFF_PC + NPC * 64;
  static constexpr int NBAR = 2 * NPC + 4 + 2 * SK + 2 * SV + 10 + 4;
  static constexpr int SMEM = OFF_BAR + NBAR * 8 + 64;
  // Tensor memory columns: S of the groups at 0 and 128; with d = 64 there is room
  // for P beside S, so the next S can be computed as soon as the last one has been
  // read; with d = 128 P lies over S.
  static constexpr bool OWN_P = D == 64;
  static constexpr int TP = OWN_P ? 256 : 0, TP_STEP = OWN_P ? 64 : 128;
  static constexpr int TO = OWN_P ? 384 : 256, TO_STEP = D;
  static_assert(SMEM <= 232448, "shared memory of one CTA");
};

struct TcArgs : LineArgs {
  __nv_bfloat16* O;
  float* lse;
  int box;               // rows of a K/V box: gcd(page size, 128)
  int wide;              // O is 32-byte aligned
  float sl2;             // scale * log2(e)
};

static_assert(sizeof(Piece) <= 64, "ring slot");

__device__ __forceinline__ float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// Once a role gives up waiting, the others stop at their next wait; the kernel's end
// reports the detail.  (The waits are kept short: a tile's loop of all roles has to
// stay in the instruction cache.)
struct GiveUp {
  volatile int* flag;
  __device__ __forceinline__ bool now(uint64_t t0, int where, uint64_t limit_ns = kWaitLimitNs) const {
    if (*flag != 0) return true;
    if (globaltimer() - t0 <= limit_ns) return false;
    *flag = where;
    return true;
  }
};
// Bounded wait of a warp, with a warp-uniform outcome.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, const GiveUp& up, int where,
                                          uint64_t limit_ns = kWaitLimitNs) {
  bool there = mbar_try_wait(bar, parity);
  if (!there) {
    const uint64_t t0 = globaltimer();
    for (uint32_t i = 1; !there; ++i) {
      there = mbar_try_wait(bar, parity);
      if ((i & 63) == 0 && !there && up.now(t0, where, limit_ns)) break;
    }
  }
  return __all_sync(FULL, there);
}
// Same, polling: for the hand-offs of the product pipeline, where a suspended wait's
// wake-up costs more than the polling.
__device__ __forceinline__ bool warp_poll(uint64_t* bar, uint32_t parity, const GiveUp& up, int where) {
  uint64_t t0 = 0;
  for (uint32_t i = 0; !__all_sync(FULL, mbar_test(bar, parity)); ++i) {
    if (i == 0) t0 = globaltimer();
    if ((i & 255) == 255 && __any_sync(FULL, up.now(t0, where))) return false;
  }
  return true;
}

// tcgen05.mma, bf16 operands and fp32 accumulation, from the low words of the
// shared-memory descriptors: D (+)= A B^T with A in shared or tensor memory.
constexpr uint32_t kDescHigh = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ void umma_ss(uint32_t d, uint32_t alo, uint32_t blo, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 a, b;\n setp.ne.b32 p, %4, 0;\n mov.b64 a, {%1, %5};\n"
      " mov.b64 b, {%2, %5};\n tcgen05.mma.cta_group::1.kind::f16 [%0], a, b, %3, p;\n}" ::"r"(d),
      "r"(alo), "r"(blo), "r"(idesc), "r"(accumulate), "r"(kDescHigh)
      : "memory");
}
__device__ __forceinline__ void umma_ts(uint32_t d, uint32_t a_tmem, uint32_t blo, uint32_t idesc,
                                        uint32_t accumulate) {
  asm volatile(
      "{\n .reg .pred p;\n .reg .b64 b;\n setp.ne.b32 p, %4, 0;\n mov.b64 b, {%2, %5};\n"
      " tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], b, %3, p;\n}" ::"r"(d),
      "r"(a_tmem), "r"(blo), "r"(idesc), "r"(accumulate), "r"(kDescHigh)
      : "memory");
}

// Bits of keys [k, k + 32) that lie in [lo, hi).
__device__ __forceinline__ uint32_t seen_bits(int k, int lo, int hi) {
  const int a = max(lo - k, 0), b = min(hi - k, 32);
  if (b <= a) return 0u;
  return (b >= 32 ? FULL : (1u << b) - 1u) & ~((1u << a) - 1u);
}

// 8 consecutive 32-bit words of one row
__device__ __forceinline__ void store8(void* p, const uint32_t* w, bool wide) {
  if (wide) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]),
                 "r"(w[1]), "r"(w[2]), "r"(w[3]), "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
                 : "memory");
  } else {
    uint4* q = static_cast<uint4*>(p);
    q[0] = make_uint4(w[0], w[1], w[2], w[3]);
    q[1] = make_uint4(w[4], w[5], w[6], w[7]);
  }
}

template <int D>
__global__ void __launch_bounds__(NTHREADS, 1)
    k_paged_attn(const __grid_constant__ CUtensorMap mq, const __grid_constant__ CUtensorMap mk,
                 const __grid_constant__ CUtensorMap mv, const __grid_constant__ TcArgs a) {
  using C = Cfg<D>;
  extern __shared__ __align__(1024) uint8_t smem[];
  pdl_next();
  if (smem_u32(smem) & 1023u) {  // the operand tiles' swizzle needs it
    pdl_wait();
    if (threadIdx.x == 0) a.rec[blockIdx.x] = make_int4(0, 0, 0, 0);  // nothing to merge
    if (blockIdx.x == 0 && threadIdx.x == 0) report(a.status, SGQA_ERR_BOUNDS, 330);
    return;
  }
  auto piece_at = [&](int i) -> Piece& {
    return *reinterpret_cast<Piece*>(smem + C::OFF_PC + (i % NPC) * 64);
  };
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::OFF_BAR);
  uint64_t* pc_full = bars;                 // [NPC]
  uint64_t* pc_empty = pc_full + NPC;       // [NPC]
  uint64_t* q_full = pc_empty + NPC;        // [2] query tiles
  uint64_t* q_empty = q_full + 2;           // [2]
  uint64_t* k_full = q_empty + 2;           // [SK]
  uint64_t* k_empty = k_full + C::SK;       // [SK]
  uint64_t* v_full = k_empty + C::SK;       // [SV]
  uint64_t* v_empty = v_full + C::SV;       // [SV]
  uint64_t* s_full = v_empty + C::SV;       // [2] S of a group's key tile
  uint64_t* p_full = s_full + 2;            // [2] its P
  uint64_t* s_empty = p_full + 2;           // [2] S has been read (OWN_P)
  uint64_t* p_empty = s_empty + 2;          // [2] the product with P is done (OWN_P)
  uint64_t* o_full = p_empty + 2;           // [2] a group's last product of a piece done
  uint64_t* x_bar = o_full + 2;             // [2] groups joined: statistics, outputs read
  uint64_t* mma_done = x_bar + 2;
  uint64_t* stall_bar = mma_done + 1;       // nothing arrives on it
  uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(bars + C::NBAR);
  int* abort_flag = reinterpret_cast<int*>(tmem_slot + 1);
  float* xmax = reinterpret_cast<float*>(smem + C::OFF_X);  // [2][BM]
  float* xsum = xmax + 2 * BM;                              // [2][BM]
  const int warp = warp_id(), lane = lane_id();

  if (threadIdx.x == 0) {
    for (int i = 0; i < NPC; ++i) {
      mbar_init(&pc_full[i], 1);
      mbar_init(&pc_empty[i], 11);  // K, V, products, 8 softmax warps
    }
    for (int i = 0; i < C::SK; ++i) {
      mbar_init(&k_full[i], 1);
      mbar_init(&k_empty[i], 1);
    }
    for (int i = 0; i < C::SV; ++i) {
      mbar_init(&v_full[i], 1);
      mbar_init(&v_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(&q_full[i], 1);
      mbar_init(&q_empty[i], 1);
      mbar_init(&s_full[i], 1);
      mbar_init(&p_full[i], 4);
      mbar_init(&s_empty[i], 4);
      mbar_init(&p_empty[i], 1);
      mbar_init(&o_full[i], 1);
      mbar_init(&x_bar[i], 8);
    }
    mbar_init(mma_done, 1);
    mbar_init(stall_bar, 1);
    *abort_flag = 0;
    fence_mbar_init();
  }
  if (warp == 3) tmem_alloc(tmem_slot, 512);
  pdl_wait();
  if (lane == 0 && warp >= 1 && warp <= 3) tma_prefetch_desc(warp == 1 ? &mk : warp == 2 ? &mv : &mq);

  // ---- the line: its length, the part of it that waves would take, and the keys
  // that several items share.  Exact integer sums, the same in every CTA.
  int64_t(*warp_sums)[4] = reinterpret_cast<int64_t(*)[4]>(xmax);
  Cut cut = cut_of<KB>(a, threadIdx.x, blockIdx.x == 0);  // (warp 0 keeps its 32)
  line_sums<KB, NTHREADS>(a, cut, warp_sums);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  const GiveUp up{abort_flag};
  // The others sleep until the first piece is there: waiting on its barrier they
  // slowed the walk of warp 0 from 2 to 12 thousand cycles.
  if (warp != 0) asm volatile("bar.sync 1, 384;" ::: "memory");
  // Registers: a softmax thread holds a row's 128 scores.  2 x 128 x kRegsMore +
  // 128 x kRegsLess stays within the 384 x 168 of the launch.
  constexpr int kRegsLess = 88, kRegsMore = 208;
  static_assert(256 * kRegsMore + 128 * kRegsLess <= NTHREADS * 168, "the launch's registers");
  if (warp < 4) {
  asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsLess));
  if (warp == 0) {
    // ============================================================ pieces, Q
    const LineSums sums = add_sums<NTHREADS>(a, warp_sums);
    int pub = 0, nq = 0;     // pieces published, their Q looked after
    int qs = 0;              // query slot of the next single tile
    uint32_t qph = 3u;       // phases of q_empty to wait for, bit = slot
    uint32_t loaded = 0, lph = 0;  // slots with a load issued, its phase
    // Q of the next piece, once its slots are free
    auto pump = [&]() -> bool {
      if (nq >= pub) return false;
      const Piece& pc = piece_at(nq);
      if (pc.n == 0) {
        ++nq;
        return true;
      }
      const uint32_t slots = pc.single ? 1u << qs : 3u;
      for (int i = 0; i < 2; ++i)
        if ((slots >> i & 1u) &&
            !__shfl_sync(FULL, (int)mbar_test(&q_empty[i], (qph >> i) & 1u), 0))
          return false;
      if (lane == 0) {
        int row = pc.row0;
        for (int i = 0; i < 2; ++i) {
          if (!(slots >> i & 1u)) continue;
          mbar_expect_tx(&q_full[i], (uint32_t)(C::KC * 128 * a.pd.G * a.tpm));
          for (int c = 0; c < C::KC; ++c)  // rows (token, head) of the box
            tma_load_3d(smem + C::OFF_Q + i * C::TILE + c * (BM * 128), &mq, &q_full[i], c * 64,
                        pc.g * a.pd.G, row);
          row += a.tpm;
        }
      }
      __syncwarp();
      lph = (lph & ~slots) | (~qph & slots);  // a slot's n-th load completes phase n
      qph ^= slots;
      loaded |= slots;
      if (pc.single) qs ^= 1;
      ++nq;
      return true;
    };
    // progress or, after a while without, the limit
    uint64_t t_prog = 0;
    uint32_t idle = 0;
    auto waited = [&](bool progress) -> bool {
      if (progress) {
        idle = 0;
        return true;
      }
      if (idle == 0) t_prog = globaltimer();
      __nanosleep(1000);  // (500: windowed chunks 1 % slower)
      if ((++idle & 63) != 0) return true;
      return !__any_sync(FULL, up.now(t_prog, 331));
    };
    auto publish = [&](const Piece& pc) -> bool {
      for (bool there = false;;) {
        if (!there && pub - nq < NPC &&
            __shfl_sync(FULL, (int)mbar_test(&pc_empty[pub % NPC], (uint32_t)(((pub / NPC) & 1) ^ 1)),
                        0)) {
          if (lane == 0) {
            piece_at(pub) = pc;
            mbar_arrive(&pc_full[pub % NPC]);
          }
          __syncwarp();
          if (pub == 0) asm volatile("bar.arrive 1, 384;" ::: "memory");
          ++pub;
          there = true;
        }
        const bool moved = pump();
        if (there) {
          idle = 0;
          return true;
        }
        if (!waited(moved)) return false;
      }
    };

    int4 rec;
    bool ok = walk_line<KB>(a, cut, sums, publish, &rec);
    if (lane == 0) a.rec[blockIdx.x] = rec;  // for the merge
    if (ok) {
      Piece pc{};
      pc.end = 1;
      ok = publish(pc);
    }
    while (ok && nq < pub) ok = waited(pump());
    // Copies land before the CTA ends, whoever gives up and whenever: a role that has
    // issued its last one may be done long before another one's wait runs out.
    if (lane == 0)
      for (int i = 0; i < 2; ++i)
        if (loaded >> i & 1u) mbar_wait_drain(&q_full[i], (lph >> i) & 1u, a.status, 391);
  } else if (warp <= 2) {
    // ========================================================== K or V loads
    const bool isK = warp == 1;
    const CUtensorMap* map = isK ? &mk : &mv;
    uint64_t* full = isK ? k_full : v_full;
    uint64_t* empty = isK ? k_empty : v_empty;
    const int NS = isK ? C::SK : C::SV;
    uint8_t* slots = smem + (isK ? C::OFF_K : C::OFF_V);
    const int rows_total = a.pd.n_pages * a.pd.Hkv * a.pd.ps;
    const int nbox = KB / a.box;
    int cnt = 0;  // tiles loaded
    bool ok = true;
    for (int i = 0; ok; ++i) {
      ok = warp_wait(&pc_full[i % NPC], (uint32_t)((i / NPC) & 1), up, 332);
      if (!ok) break;
      const Piece pc = piece_at(i);
      __syncwarp();
      if (lane == 0) mbar_arrive(&pc_empty[i % NPC]);
      if (pc.end) break;
      const int32_t* row = a.page_table + (int64_t)pc.s * a.pd.max_pages;
      for (int t = 0; t < pc.n; ++t, ++cnt) {
        // this lane's box: keys key .. key + box - 1, skipped when none is seen
        const int key = (pc.tb + t) * KB + lane * a.box;
        const bool on = lane < nbox && key < pc.hi && key + a.box > pc.lo;
        int at = rows_total;  // outside the pool: zeros
        if (on) {
          const int pi = key / a.pd.ps, page = row[pi];
          if (page >= 0 && page < a.pd.n_pages)
            at = (page * a.pd.Hkv + pc.g) * a.pd.ps + (key - pi * a.pd.ps);
          else
            report(a.status, SGQA_ERR_BOUNDS, 302);
        }
        const int boxes = __popc(__ballot_sync(FULL, on));
        const int sl = cnt % NS;
        ok = warp_wait(&empty[sl], (uint32_t)(((cnt / NS) & 1) ^ 1), up, isK ? 333 : 334);
        if (!ok) break;
        if (lane == 0) mbar_expect_tx(&full[sl], (uint32_t)(boxes * a.box * 128 * C::KC));
        __syncwarp();
        if (on)
          for (int c = 0; c < C::KC; ++c)
            tma_load_2d(slots + sl * C::TILE + c * (KB * 128) + lane * a.box * 128, map, &full[sl],
                        c * 64, at);
        __syncwarp();
      }
    }
    if (lane == 0)  // (as for Q above)
      for (int k = 0; k < NS; ++k) {
        const int uses = cnt / NS + (k < cnt % NS ? 1 : 0);
        if (uses > 0) mbar_wait_drain(&full[k], (uint32_t)((uses - 1) & 1), a.status, isK ? 392 : 393);
      }
  } else {
    // ============================================================== products
    // The whole warp walks the loop and one elected lane issues, so that the
    // loop's state and the operand descriptors stay in uniform registers: with
    // the loop inside a one-lane branch every product's descriptors were built
    // in vector registers and moved over, 108 cycles an instruction, and the
    // issue took twice as long as the products (chunk of 4096 tokens over 36K
    // keys: 4.33 ms).
    const bool leader = elect_one();
    constexpr uint32_t idesc_qk = idesc_bf16_f32(BM, KB, 0, 0);
    constexpr uint32_t idesc_pv = idesc_bf16_f32(BM, D, 0, 1);
    // low words of the operand descriptors (address and leading-dimension
    // offset); the high word is the same for all: 1024 bytes between 8-row
    // groups, 128-byte swizzle
    const uint32_t lq = (smem_u32(smem + C::OFF_Q) >> 4) | (1u << 16);
    const uint32_t lk = (smem_u32(smem + C::OFF_K) >> 4) | (1u << 16);
    const uint32_t lv = (smem_u32(smem + C::OFF_V) >> 4) | ((uint32_t)(KB * 128 / 16) << 16);
    int ks = 0, vs = 0;             // slots of the next key tile
    uint32_t kph = 0, vph = 0;      // and their phases
    uint32_t pph = 0, sph = 0;      // phases of p_full and s_empty, bit = group
    uint32_t used = 0;              // groups that have had an S
    int qs = 0;                     // query slot of the next single tile
    uint32_t qph = 0;               // phases of q_full, bit = slot
    bool first = true, ok = true;
    for (int i = 0; ok; ++i) {
      ok = warp_poll(&pc_full[i % NPC], (uint32_t)((i / NPC) & 1), up, 335);
      if (!ok) break;
      const Piece& pc = piece_at(i);
      // (reductions of equal values: uniform registers)
      const int n = __reduce_max_sync(FULL, pc.n), single = __reduce_max_sync(FULL, pc.single);
      const int end = __reduce_max_sync(FULL, pc.end);
      if (n > 0) {
        ok = warp_poll(&q_full[single ? qs : 0], (qph >> (single ? qs : 0)) & 1u, up, 336) &&
             (single || warp_poll(&q_full[1], qph >> 1, up, 336));
        // Debug request (host-set status[3]): the first piece waits on a barrier
        // nothing arrives on, so the pipeline gives up (detail 220) while its K
        // and V copies are in flight.
        if (ok && first && blockIdx.x == 0 && debug_request(a.status) == SGQA_DEBUG_STALL)
          ok = warp_wait(stall_bar, 0, up, 220, kDebugStallNs);
        if (!ok) break;
        qph ^= single ? 1u << qs : 3u;
        first = false;
      }
      if (leader) mbar_arrive(&pc_empty[i % NPC]);
      if (end) break;
      const int sh = single ? 0 : 1;  // a key tile serves 1 << sh products of each kind
      const int J = n << sh;
      const int slot = single ? qs : 0;  // of the first query tile
      // S of step j: group j & 1, query tile j & sh, the next key tile when j & sh is 0
      auto qk = [&](int j) {
        tc_fence_after();
        const uint32_t d = tmem + (uint32_t)(j & 1) * 128;
        const uint32_t la = lq + (uint32_t)(slot + (j & sh)) * (C::TILE / 16), lb = lk + (uint32_t)ks * (C::TILE / 16);
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < D / 16; ++kk) {
            const uint32_t off = (kk >> 2) * (BM * 128 / 16) + (kk & 3) * 2;
            umma_ss(d, la + off, lb + off, idesc_qk, kk > 0);
          }
          umma_commit(&s_full[j & 1]);
          if ((j & sh) == sh) umma_commit(&k_empty[ks]);
          if (j >= J - 1 - sh) umma_commit(&q_empty[slot + (j & sh)]);  // its last product
        }
        __syncwarp();
        if ((j & sh) == sh && ++ks == C::SK) {
          ks = 0;
          kph ^= 1;
        }
      };
      // O of group j & 1 += P V
      auto pv = [&](int j) {
        const int grp = j & 1;
        tc_fence_after();
        const uint32_t d = tmem + C::TO + (uint32_t)grp * C::TO_STEP;
        const uint32_t pa = tmem + C::TP + (uint32_t)grp * C::TP_STEP;
        const uint32_t lb = lv + (uint32_t)vs * (C::TILE / 16);
        const uint32_t more = j > 1;
        if (leader) {
#pragma unroll
          for (int kk = 0; kk < KB / 16; ++kk)
            umma_ts(d, pa + kk * 8, lb + kk * 128, idesc_pv, kk > 0 ? 1u : more);
          if constexpr (C::OWN_P) umma_commit(&p_empty[grp]);
          if ((j & sh) == sh) umma_commit(&v_empty[vs]);
          if (j + 2 >= J) umma_commit(&o_full[grp]);  // the group's last product
        }
        __syncwarp();
        if ((j & sh) == sh && ++vs == C::SV) {
          vs = 0;
          vph ^= 1;
        }
      };
      if constexpr (C::OWN_P) {
        // Both products as soon as what they need is there, each kind in step order; P
        // first (4096 tokens over 32768 keys, 32 heads: 1280 us, S first 1309).  A warp
        // for each kind, with one for both loads, was slower (window 201 us).
        int nqk = 0, npv = 0;
        uint64_t t_prog = 0;
        uint32_t idle = 0;
        while (npv < J) {
          bool progress = false;
          if (npv < nqk) {
            const int g = npv & 1;
            if (__all_sync(FULL, mbar_test(&p_full[g], (pph >> g) & 1u) &&
                                     ((npv & sh) != 0 || mbar_test(&v_full[vs], vph)))) {
              pph ^= 1u << g;
              pv(npv++);
              progress = true;
            }
          }
          if (nqk < J) {
            const int g = nqk & 1;
            if (__all_sync(FULL, ((used >> g & 1u) == 0u || mbar_test(&s_empty[g], (sph >> g) & 1u)) &&
                                     ((nqk & sh) != 0 || mbar_test(&k_full[ks], kph)))) {
              if (used >> g & 1u) sph ^= 1u << g;
              used |= 1u << g;
              qk(nqk++);
              progress = true;
            }
          }
          if (progress) {
            idle = 0;
          } else {
            if (idle == 0) t_prog = globaltimer();
            if ((++idle & 255) == 0 && __any_sync(FULL, up.now(t_prog, 337))) {
              ok = false;
              break;
            }
          }
        }
      } else {
        // The product with P, and behind it the next S, which overwrites P: products
        // of one thread run in issue order.  The next key tile is looked for while P
        // is waited for, so that the two are issued without a pause.
        auto k_there = [&](int j) -> bool {
          return (j & sh) != 0 || warp_poll(&k_full[ks], kph, up, 337);
        };
        for (int j = 0; ok && j < 2 && j < J; ++j) {
          ok = k_there(j);
          if (ok) qk(j);
        }
        for (int j = 0; ok && j < J; ++j) {
          const int g = j & 1;
          const bool next = j + 2 < J;
          bool key = !next || (j & sh) != 0;
          uint64_t t_prog = 0;
          for (uint32_t i2 = 0;; ++i2) {
            const bool there = mbar_test(&p_full[g], (pph >> g) & 1u) &
                               ((j & sh) != 0 || mbar_test(&v_full[vs], vph));
            if (!key) key = __all_sync(FULL, mbar_test(&k_full[ks], kph));
            if (__all_sync(FULL, there)) break;
            if ((i2 & 255) == 255) {
              if (t_prog == 0) t_prog = globaltimer();
              if (__any_sync(FULL, up.now(t_prog, 339))) {
                ok = false;
                break;
              }
            }
          }
          if (!ok) break;
          pph ^= 1u << g;
          pv(j);
          if (next) {
            if (!key) ok = k_there(j + 2);
            if (ok) qk(j + 2);
          }
        }
      }
      if (single && n > 0) qs ^= 1;
    }
    if (leader) {
      umma_commit(mma_done);
      mbar_wait_drain(mma_done, 0, a.status, 399);
    }
    __syncwarp();
  }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsMore));
    // =============================================================== softmax
    const int grp = (warp - 4) >> 2, quad = warp & 3;
    const int r = quad * 32 + lane;
    const uint32_t tl = tmem + (static_cast<uint32_t>(quad * 32) << 16);
    const uint32_t tS = tl + grp * 128, tP = tl + C::TP + grp * C::TP_STEP;
    const uint32_t tO = tl + C::TO + grp * C::TO_STEP;
    const float ninf = -__int_as_float(0x7f800000);
    const float sl2 = a.sl2;
    const uint64_t sl2x2 = f2_pack(sl2, sl2);
    const int G = a.pd.G, rt = r / G, rh = r - rt * G;  // token and head of the row in its tile
    int sc = 0, oc = 0, xc = 0, vbase = 0;
    bool ok = true;
    for (int i = 0; ok; ++i) {
      ok = warp_wait(&pc_full[i % NPC], (uint32_t)((i / NPC) & 1), up, 340);
      if (!ok) break;
      const Piece pc = piece_at(i);
      __syncwarp();
      if (lane == 0) mbar_arrive(&pc_empty[i % NPC]);
      if (pc.end) break;
      const int tok = rt + (pc.single ? 0 : grp * a.tpm);
      const bool row_ok = rt < a.tpm && tok < pc.ntok;
      const bool active = __any_sync(FULL, row_ok);
      const int pos = pc.pos0 + tok;
      const int hi = !row_ok ? 0x7fffffff : a.pd.causal ? min(pc.hi, pos + 1) : pc.hi;
      const int lo = !row_ok ? 0 : a.pd.window ? max(pc.lo, pos + 1 - a.pd.window) : pc.lo;
      float m_used = ninf, l = 0.0f;
      const int step = pc.single ? 2 : 1;
      const int t0 = pc.single ? grp : 0;
      for (int t = t0; t < pc.n; t += step) {
        const int k0 = (pc.tb + t) * KB;
        ok = warp_wait(&s_full[grp], (uint32_t)(sc & 1), up, 341);
        if (!ok) break;
        ++sc;
        tc_fence_after();
        // P may be written, and O rescaled, once the last product with them is done
        // (without its own P, S was computed behind that product)
        auto p_free = [&]() -> bool {
          if constexpr (C::OWN_P) {
            if (sc > 1)
              return warp_wait(&p_empty[grp], (uint32_t)(sc & 1), up, 348);
          }
          return true;
        };
        uint32_t v[128];
        if (active) {
#pragma unroll
          for (int w = 0; w < 4; ++w)
            tmem_ld32(tS + w * 32, *reinterpret_cast<uint32_t(*)[32]>(&v[w * 32]));
          tmem_wait_ld();
        }
        if constexpr (C::OWN_P) {  // S is in registers: the next one may be computed
          tc_fence_before();
          __syncwarp();
          if (lane == 0) mbar_arrive(&s_empty[grp]);
        }
        if (active) {
          if (!__all_sync(FULL, lo <= k0 && k0 + KB <= hi)) {
            // by selection: S of keys outside the cache may be NaN
#pragma unroll
            for (int w = 0; w < 4; ++w) {
              const uint32_t m = seen_bits(k0 + 32 * w, lo, hi);
#pragma unroll
              for (int e = 0; e < 32; ++e)
                v[w * 32 + e] = ((m >> e) & 1u) ? v[w * 32 + e] : __float_as_uint(ninf);
            }
          }
          float mx[4] = {ninf, ninf, ninf, ninf};
#pragma unroll
          for (int e = 0; e < 128; e += 8) {
#pragma unroll
            for (int c = 0; c < 4; ++c)
              mx[c] = fmaxf(fmaxf(mx[c], __uint_as_float(v[e + 2 * c])), __uint_as_float(v[e + 2 * c + 1]));
          }
          const float smax = fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2;
          const bool raise = smax > m_used + kLazy;
          if (__any_sync(FULL, raise)) {
            const float f = raise ? ex2(m_used - smax) : 1.0f;  // 0 for the first keys a row sees
            if (t > t0) {
              ok = p_free();
              if (!ok) break;
#pragma unroll 1
              for (int c = 0; c < D / 8; ++c) {
                uint32_t o[8];
                tmem_ld8(tO + c * 8, o);
                tmem_wait_ld();
#pragma unroll
                for (int e = 0; e < 8; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * f);
                tmem_st8(tO + c * 8, o);
              }
            }
            l *= f;
            if (raise) m_used = smax;
          }
          const float nm = m_used == ninf ? 0.0f : -m_used;
          const uint64_t nm2 = f2_pack(nm, nm);
          uint64_t acc[4] = {0ull, 0ull, 0ull, 0ull};
#pragma unroll
          for (int h = 0; h < 2; ++h) {
            uint32_t pk[32];
#pragma unroll
            for (int e = 0; e < 64; e += 2) {
              float x0, x1;
              f2_unpack(f2_fma(f2_pack(__uint_as_float(v[h * 64 + e]), __uint_as_float(v[h * 64 + e + 1])),
                               sl2x2, nm2), x0, x1);
              const float p0 = ex2(x0), p1 = ex2(x1);
              acc[(e >> 1) & 3] = f2_add(acc[(e >> 1) & 3], f2_pack(p0, p1));
              pk[e >> 1] = pack_bf16x2(p0, p1);
            }
            if (h == 0) {
              ok = p_free();
              if (!ok) break;
            }
            tmem_st32(tP + h * 32, pk);
          }
          if (!ok) break;
          float s0, s1;
          f2_unpack(f2_add(f2_add(acc[0], acc[1]), f2_add(acc[2], acc[3])), s0, s1);
          l += s0 + s1;
        } else {
          // (a warp without rows must not run ahead: its next arrival on p_full
          // would count for this tile)
          ok = p_free();
          if (!ok) break;
        }
        // Rows of V that no row of the item sees are zeroed before the product: they
        // may hold anything, and 0 times an infinity or NaN would count.  (Not before
        // S is there: only then has the slot's last tile been used.)
        if ((pc.single || grp == 0) && (pc.lo > k0 || pc.hi < k0 + KB)) {
          const int vt = vbase + t, vs = vt % C::SV;
          ok = warp_wait(&v_full[vs], (uint32_t)((vt / C::SV) & 1), up, 342);
          if (!ok) break;
          if (k0 + r < pc.lo || k0 + r >= pc.hi) {
            uint8_t* vr = smem + C::OFF_V + vs * C::TILE + r * 128;
            for (int c = 0; c < C::KC; ++c)
#pragma unroll
              for (int b = 0; b < 8; ++b)  // (lanes start at different banks)
                *reinterpret_cast<uint4*>(vr + c * (KB * 128) + ((b + lane) & 7) * 16) =
                    make_uint4(0, 0, 0, 0);
          }
          fence_proxy_async_smem();
        }
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&p_full[grp]);
      }
      if (!ok) break;
      vbase += pc.n;
      // ---- outputs
      const int n0 = pc.single ? (pc.n + 1) / 2 : pc.n, n1 = pc.single ? pc.n / 2 : pc.n;
      auto o_done = [&]() -> bool {
        if ((grp == 0 ? n0 : n1) == 0) return true;
        const bool done =
            warp_wait(&o_full[grp], (uint32_t)(oc & 1), up, 343);
        ++oc;
        return done;
      };
      // a single tile with a part in each accumulator: the groups exchange their
      // maxima and sums and share out the columns; else the group that has the
      // part writes all of it
      const bool share = pc.single && n1 > 0;
      float g0, g1, lt = l, mm = m_used;
      bool part0 = true, part1 = true;  // the row saw keys in the group's tiles
      if (share) {
        ok = o_done();
        if (!ok) break;
        xmax[grp * BM + r] = m_used;
        xsum[grp * BM + r] = l;
        __syncwarp();
        if (lane == 0) mbar_arrive(&x_bar[0]);
        ok = warp_wait(&x_bar[0], (uint32_t)(xc & 1), up, 345);
        if (!ok) break;
        const float m0 = xmax[r], m1 = xmax[BM + r];
        mm = fmaxf(m0, m1);
        g0 = m0 == ninf ? 0.0f : ex2(m0 - mm);
        g1 = m1 == ninf ? 0.0f : ex2(m1 - mm);
        lt = xsum[r] * g0 + xsum[BM + r] * g1;
        part0 = m0 != ninf || lt != lt;
        part1 = m1 != ninf || lt != lt;
      } else {
        g0 = grp == 0 ? 1.0f : 0.0f;
        g1 = 1.0f - g0;
      }
      // all that needs no output comes before the wait for the last product
      const float inv = lt != 0.0f ? 1.0f / lt : 0.0f;  // (a NaN stays one)
      const float lse = lt != 0.0f ? (mm + __log2f(lt)) * 0.69314718055994531f : ninf;
      const bool mine = share || !pc.single || grp == 0;
      const int64_t orow = (int64_t)(pc.row0 + tok) * a.pd.H + (int64_t)pc.g * G + rh;
      const int64_t prow = (int64_t)pc.slot * a.slot_rows + (pc.single ? 0 : grp * BM) + r;
      uint8_t* dst = pc.slot >= 0 ? reinterpret_cast<uint8_t*>(a.opart + prow * D)
                                  : reinterpret_cast<uint8_t*>(a.O + orow * D);
      if (row_ok && (grp == 0 || !pc.single)) {
        if (pc.slot >= 0)
          a.lpart[prow] = lse;
        else
          a.lse[(int64_t)(pc.g * G + rh) * a.pd.T + pc.row0 + tok] = lse;
      }
      if (!share) {
        ok = o_done();
        if (!ok) break;
      }
      tc_fence_after();
      if (active && mine) {
        g0 *= inv;
        g1 *= inv;
        const int c0 = share ? grp * (D / 2) : 0, c1 = share ? c0 + D / 2 : D;
#pragma unroll 1
        for (int c = c0; c < c1; c += 32) {
          uint32_t o[32];
          if (share) {
            uint32_t o1[32];
            tmem_ld32(tl + C::TO + c, o);
            tmem_ld32(tl + C::TO + C::TO_STEP + c, o1);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e)
              o[e] = __float_as_uint((part0 ? __uint_as_float(o[e]) * g0 : 0.0f) +
                                     (part1 ? __uint_as_float(o1[e]) * g1 : 0.0f));
          } else if (pc.n > 0) {
            tmem_ld32(tO + c, o);
            tmem_wait_ld();
#pragma unroll
            for (int e = 0; e < 32; ++e)
              o[e] = lt != 0.0f ? __float_as_uint(__uint_as_float(o[e]) * inv) : 0u;
          } else {
#pragma unroll
            for (int e = 0; e < 32; ++e) o[e] = 0u;
          }
          if (row_ok && pc.slot >= 0) {
#pragma unroll
            for (int e = 0; e < 32; e += 8) store8(dst + c * 4 + e * 4, o + e, true);
          } else if (row_ok) {
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e)
              w[e] = pack_bf16x2(__uint_as_float(o[2 * e]), __uint_as_float(o[2 * e + 1]));
            store8(dst + c * 2, w, a.wide);
            store8(dst + c * 2 + 32, w + 8, a.wide);
          }
          __syncwarp();  // the loads from tensor memory are warp-wide
        }
      }
      if (share) {  // both groups have read both accumulators and the statistics
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&x_bar[1]);
        ok = warp_wait(&x_bar[1], (uint32_t)(xc & 1), up, 346);
        ++xc;
      }
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

int slot_rows(const PagedDims& pd) {
  const int64_t rows = (int64_t)pd.T * pd.G;
  return (int)(rows < BM ? rows : 2 * BM);
}

// Q [T][H][d] with row stride qs, boxes of one query tile's heads and tokens.
bool q_map(const PagedDims& pd, int tpm, const void* Q, CUtensorMap* m) {
  auto fn = tmap_encode_fn();
  if (fn == nullptr) return false;
  cuuint64_t dims[3] = {(cuuint64_t)pd.d, (cuuint64_t)pd.H, (cuuint64_t)pd.T};
  cuuint64_t str[2] = {(cuuint64_t)pd.d * 2, (cuuint64_t)pd.qs * 2};
  cuuint32_t box[3] = {64, (cuuint32_t)pd.G, (cuuint32_t)tpm}, es[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(Q), dims, str, box, es,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <int D>
int launch(const TcArgs& a, const PagedAttnArgs& pa, cudaStream_t st) {
  using C = Cfg<D>;
  const PagedDims& pd = a.pd;
  CUtensorMap mq, mk, mv;
  const uint64_t rows = (uint64_t)pd.n_pages * pd.Hkv * pd.ps;
  if (!q_map(pd, a.tpm, pa.Q, &mq) ||
      !make_tmap_2d_bf16(&mk, pa.K, D, rows, D * 2, 64, (uint32_t)a.box) ||
      !make_tmap_2d_bf16(&mv, pa.V, D, rows, D * 2, 64, (uint32_t)a.box))
    return SGQA_ERR_CUDA;
  if (cudaFuncSetAttribute(k_paged_attn<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, C::SMEM) !=
      cudaSuccess)
    return SGQA_ERR_CUDA;
  log_begin(SGQA_K_PAGED_ATTN, st);
  const cudaError_t e = launch_pdl(k_paged_attn<D>, kGrid, NTHREADS, C::SMEM, st, mq, mk, mv, a);
  log_end(st);
  if (e != cudaSuccess) return SGQA_ERR_CUDA;
  return launch_merge<__nv_bfloat16, D, kGrid, 256>(a, a.O, a.lse, st);
}

}  // namespace

size_t paged_tc_ws_bytes(const PagedDims& pd) {
  return pd.N == 0 || pd.T == 0 ? 0 : carve_line(kGrid, slot_rows(pd), pd.d).bytes;
}

int launch_paged_tc(const PagedDims& pd, const PagedAttnArgs& pa, void* ws, cudaStream_t st) {
  TcArgs a;
  a.slot_rows = slot_rows(pd);
  set_line(a, pd, pa, carve_line(kGrid, a.slot_rows, pd.d), ws);
  a.groups = pd.Hkv;
  a.head_parts = 1;
  a.heads = pd.G;
  a.tpm = BM / pd.G;
  a.tiles_per_item = 2;
  a.tile_rows = BM;
  a.over = 3;  // (2 to 4 are alike: mixed chunks 100, 99, 99 us, 64 ragged contexts 358, 361, 360)
  // 0.8 us a tile, 4 us for a merge: four contexts of 300 to 2047 keys 14.8 us, of 1000
  // to 5000 16.7 (8 and 6: 15.5 and 16.5; 4 and 3: 15.4 and 17.3).  Without a merge where
  // the page table holds at most 8 tiles, so that no cache can be longer: four contexts
  // of 1000 keys 13.2 us, against 14.2.
  a.whole = a.part = 4;
  a.uncut = pd.cap <= 8 * KB;
  a.O = static_cast<__nv_bfloat16*>(pa.O);
  a.lse = pa.lse;
  int x = pd.ps, y = KB;
  while (y) {
    const int t = x % y;
    x = y;
    y = t;
  }
  a.box = x;
  a.wide = (reinterpret_cast<uintptr_t>(pa.O) & 31u) == 0;
  a.sl2 = pd.scale * 1.4426950408889634f;
  // whole items of a request, over its KV groups, are counted in 32 bits
  if ((int64_t)pd.Hkv * ((int64_t)pd.T / a.tpm + 1) > 0x7fffffffll) return SGQA_ERR_UNSUPPORTED;
  return pd.d == 128 ? launch<128>(a, pa, st) : launch<64>(a, pa, st);
}

}  // namespace sgqa
