// window_long.cu -- the window attention of many tokens over windows that take many blocks: tiles of
// 256 rows on clusters of 4 SMs.
//
// The same mathematics as window.cu.  There, a tile of 64 rows and its outputs fit one SM, and its chain
// (scores, softmax, outputs) has nothing beside it: with as few rows a product reads 6 KB of shared memory
// for 48 cycles' worth of it, and the tensor cores wait while the softmax is formed.  Here scores and
// outputs live on different SMs, as 128 rows x 512 fp32 outputs fill an SM's tensor memory:
//   two scores CTAs (128 rows each)  queries in tensor memory (288 columns); blocks of 64 positions come by
//       TMA, 32 of them to each CTA; S[256 x 64] = Q . K^T as one product of the pair (M 256, N 64, K 576);
//       softmax, one thread a row; P as bf16 goes to the values CTA of the same rows by an asynchronous
//       copy between their shared memories;
//   two values CTAs                  the same block's rows, 256 of the 512 channels to each;
//       O[256 x 512] += P . V (M 256, N 2 x 256, K 64).
// Data flow one way only, so each side runs ahead through its rings (4 blocks of keys or values, 3 score
// buffers, 3 blocks of P).  Tensor work of a block: 1,152 and 1,024 cycles, at the tensor cores' own rate:
// the pair's operands are read once for 256 rows.
//
// The softmax reference is a score of the row (window.cu says why not a logit), raised to a block's maximum only
// when that passes it by more than 16 (base 2), so that outputs are rarely rescaled (8: 430 in place of 410 us for
// the call below).  Sums are fp32, of the unrounded P.
//
// Masks are formed only in blocks that some row of the tile does not see whole.  There, positions whose
// scores are no numbers are passed on with P, and the values CTAs make zeros of those whose values are
// not either (0 * P would be NaN in rows that do not see them); rows that do see them become NaN by their sums.
//
// P is rounded to bf16, as the rows are (window.cu): in two parts it would take 2,048 cycles of values a block.
//
// Measured (GB300, 64 heads): 2,048 tokens at 32,768, window 2,048, 4 sinks 384-415 us (the clock gives way to power
// within a second), 1.4-1.5 PFLOP/s on what the rows see (window.cu's tiles: 705), bound by the tensor cores: a block takes
// 1,280-1,340 cycles for the 1,152 of its scores (one more block a tile costs 0.66-0.69 us in 15 rounds of tiles,
// windows of 2,048 to 8,192 positions, at 1.85-1.94 GHz); of a tile's 35 blocks four or five are half masked; a tile's
// queries (147 KB a CTA) leave a gap of 3,000 to 4,000 cycles between its products and those of the tile before; and 512
// tiles are 15 rounds of the 36 clusters that fit.  Two slots of P in place of three: 524 us, two score buffers: 407.
#include <cuda.h>

#include <atomic>

#include "common.cuh"
#include "kernels.cuh"
#include "profile.cuh"
#include "tc.cuh"
#include "window.cuh"
#include "window_tiles.cuh"

namespace csa2 {

namespace {

constexpr int kHalfRows = kLongRows / 2;             // of a CTA
constexpr int kBlk = kPage;                          // positions of a block: one page
constexpr int kRowWarps = 8;                         // softmax: lane quarter w % 4, the blocks of one parity w / 4; outputs: half of the columns
constexpr int kQueryWarp0 = 8;                       // four: queries to tensor memory (scores CTAs)
constexpr int kMmaWarp = 12, kLoadWarp = 13, kAuxWarp = 14, kPlanWarp = 15;
constexpr int kLongThreads = 16 * 32;

constexpr int kStages = 4;                           // ring: 32 positions x 576 channels, or 64 x 256; 32 query rows x 576
constexpr int kKStage = 9 * 4096, kVStage = 4 * 8192;
constexpr int kPSlots = 3, kPBytes = kHalfRows * 128;
constexpr int kRingOff = kPSlots * kPBytes;
constexpr int kOutOff = kRingOff + kStages * kVStage;     // values CTA: output staging, 4 KB a warp
constexpr int kLongSmem = kOutOff + kRowWarps * 4096;
static_assert(kStages == 4, "a tile's queries take each stage once");
static_assert(kRingOff + kStages * kKStage <= kLongSmem && kKStage % 1024 == 0, "the ring of keys fits, too");

constexpr uint32_t kSCol = 320;                      // score buffers behind the 288 query columns
constexpr int kSBufs = 3;
constexpr int kMetaWarp = 4 * 32 * 4;                // alpha, sum, reference of a warp's rows; hidden positions
constexpr int kPlanSlots = 3;

struct __align__(16) LongPiece {
  int n;                        // blocks, -1 behind the last piece
  Tile t;
  int sp;                       // sinks' pages
  // first position of block j
  __device__ int start(int j) const { return (j < sp ? j : t.lo / kPage + j - sp) * kPage; }
};

struct LongSmall {
  uint64_t full[kStages], empty[kStages];            // ring (full: of keys or values)
  // 32 query rows have come to their place in the ring: barriers apart from `full`, as a wait by parity needs all
  // of a barrier's phases, and those who copy the queries see none of the blocks between
  uint64_t q_place[4];
  uint64_t k_ready[kStages];                         // leading scores CTA: the other's half of a block is there
  uint64_t s_full[kSBufs], s_empty[kSBufs];
  uint64_t q_full, q_free;                           // queries in tensor memory (both CTAs); read by the tile's last product
  uint64_t ref_full[2][4];                           // reference of a row, from the warp of one block to that of the next
  uint64_t p_free[kPSlots];                          // scores CTA: slot read by the values CTA (remote arrival)
  uint64_t p_full[kPSlots];                          // values CTA: bytes of P and meta have arrived
  uint64_t corr[kPSlots];                            // leading values CTA: outputs brought to the slot's reference, values whole
  uint64_t pv_done[kPSlots];
  uint64_t o_free;
  uint64_t drain;
  uint64_t plan_full[kPlanSlots], plan_empty[kPlanSlots];
  uint32_t tmem_slot;
  int abort;
  int bad, tiles;
  LongPiece plan[kPlanSlots];
  __align__(16) float meta[kPSlots][4][4][32];
  float ref[2][kHalfRows];
};
static_assert(kLongSmem + (sizeof(LongSmall) + 1023) / 1024 * 1024 <= 232448, "shared memory; the dynamic part starts on a multiple of its alignment");

__device__ inline uint32_t peer_addr(const void* p, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(tc::smem_u32(p)), "r"(rank));
  return r;
}
__device__ inline void copy_to_peer(uint32_t raddr, const void* src, uint32_t bytes, uint32_t rbar) {
  asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
               ::"r"(raddr), "r"(tc::smem_u32(src)), "r"(bytes), "r"(rbar)
               : "memory");
}
// Arrival on another CTA's barrier.  What it hands over is never read by that CTA's ordinary loads.
__device__ inline void arrive_remote(uint32_t rbar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(rbar) : "memory");
}
__device__ inline void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(tc::smem_u32(bar)) : "memory");
}
__device__ inline bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// One try; kCluster: acquires what another CTA wrote.
template <bool kCluster>
__device__ inline bool try_wait(uint64_t* bar, uint32_t parity) {
  if constexpr (!kCluster) return tc::mbar_try_wait(bar, parity);
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done) : "r"(tc::smem_u32(bar)), "r"(parity) : "memory");
  return done != 0;
}
// Every wait is bounded (200 ms against microseconds) and cut short once another role of the CTA has given up.
template <bool kCluster>
__device__ __forceinline__ bool wait_slow(LongSmall& sm, uint64_t* bar, uint32_t parity, uint8_t* ws) {
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    if (try_wait<kCluster>(bar, parity)) return true;
    if (*reinterpret_cast<volatile int*>(&sm.abort)) return false;
    if ((i & 31u) == 0) {
      const uint64_t t = tc::globaltimer_ns();
      if (t0 == 0) t0 = t;
      if (t - t0 > 200ull * 1000 * 1000) {
        *reinterpret_cast<volatile int*>(&sm.abort) = 1;
        raise_err(ws, CSA2_DEV_TIMEOUT);
        return false;
      }
    }
  }
}
// For a converged warp: one answer for all lanes.
template <bool kCluster = false>
__device__ inline bool wait_warp(LongSmall& sm, uint64_t* bar, uint32_t parity, uint8_t* ws) {
  return __all_sync(0xFFFFFFFFu, try_wait<kCluster>(bar, parity) || wait_slow<kCluster>(sm, bar, parity, ws));
}

// One product of the pair: rows of both CTAs, B shared, each CTA holding half of its columns.
__device__ inline void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(uint32_t(acc)) : "memory");
}
__device__ inline void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
      ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(acc)) : "memory");
}
// Arrive on `bar` of the CTAs in `mask` once the MMAs so far are done.
__device__ inline void commit_to(uint64_t* bar, uint16_t mask) {
  asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
               ::"r"(tc::smem_u32(bar)), "h"(mask) : "memory");
}
__device__ inline uint4 ld_shared16(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr) : "memory");
  return v;
}
__device__ inline void tmem_st16_nowait(uint32_t taddr, const uint32_t (&v)[16]) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], "
      "{%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16};"
      ::"r"(taddr), "r"(v[0]), "r"(v[1]), "r"(v[2]), "r"(v[3]), "r"(v[4]), "r"(v[5]), "r"(v[6]), "r"(v[7]), "r"(v[8]),
        "r"(v[9]), "r"(v[10]), "r"(v[11]), "r"(v[12]), "r"(v[13]), "r"(v[14]), "r"(v[15])
      : "memory");
}
__device__ inline void tmem_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }

// Two fp32 operations an instruction.
__device__ inline uint64_t pack2(float lo, float hi) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
  return r;
}
__device__ inline void unpack2(uint64_t v, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(v)); }
__device__ inline uint64_t mul2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ inline uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}
__device__ inline float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ inline uint32_t bf16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// The next piece, for a converged warp; false behind the last.
__device__ inline bool next_piece(LongSmall& sm, uint32_t& k, int lane, uint8_t* ws, LongPiece& p) {
  const uint32_t slot = k % kPlanSlots;
  if (!wait_warp(sm, &sm.plan_full[slot], (k / kPlanSlots) & 1, ws)) return false;
  p = sm.plan[slot];
  __syncwarp();
  if (lane == 0) arrive(&sm.plan_empty[slot]);
  ++k;
  return p.n >= 0;
}

// One warp of each CTA walks the cluster's tiles and tells the others, a few tiles ahead.
__device__ inline void plan_role(const WindowArgs& a, LongSmall& sm, int first, int tiles, int step, int values, Sequences<kLongRows>& q, int lane) {
  q.count(lane);
  uint32_t k = 0;
  for (int t = first;; t += step, ++k) {
    LongPiece p = {};
    p.n = -1;
    if (t < tiles) {
      p.t = find_tile(a, q, t, lane);
      const TilePages pages = pages_of(a, p.t.lo, p.t.last);
      p.n = pages.all;
      p.sp = pages.sinks;
    }
    const uint32_t slot = k % kPlanSlots;
    if (!wait_warp(sm, &sm.plan_empty[slot], ((k / kPlanSlots) & 1) ^ 1, a.ws)) return;
    if (lane == 0) {
      sm.plan[slot] = p;
      arrive(&sm.plan_full[slot]);
      // values CTAs: the other attention's outputs of their rows (one piece of memory) to L2
      const int rows = p.n < 0 || values < 0 ? 0 : min(kHalfRows, p.t.have - kHalfRows * values);
      if (a.prev_out && rows > 0)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;"
                     ::"l"(a.prev_out + (int64_t(p.t.row) + kHalfRows * values) * kLatent), "r"(rows * kLatent * 2) : "memory");
    }
    __syncwarp();
    if (p.n < 0) return;
  }
}

// Copies a cluster's tiles and their blocks into the ring: queries as four places of 32 rows, then a block a
// place; a tile's queries take every stage of the ring once, so that block n of the cluster's has stage
// n % kStages, and fills it for the (n / kStages)-th time.  A page id out of range is reported and page 0 copied in its place (the
// softmax gives it no weight).
template <bool kScores>
__device__ inline void load_role(const WindowArgs& a, LongSmall& sm, uint8_t* base, int part, int lane, const CUtensorMap* qmap,
                                 const CUtensorMap* kvmap) {
  constexpr uint32_t kBytes = kScores ? kKStage : kVStage;
  constexpr int kGroups = kScores ? 9 : 4;           // of 64 channels, a lane each
  LongPiece p;
  uint32_t nu = 0, u = 0;
  bool more = next_piece(sm, nu, lane, a.ws, p);
  while (more) {
    const LongPiece now = p;
    if (kScores && now.n > 0) {
#pragma unroll 1
      for (int k = 0; k < 4; ++k, ++u) {
        const uint32_t st = u % kStages;
        if (!wait_warp(sm, &sm.empty[st], ((u / kStages) & 1) ^ 1, a.ws)) return;
        if (lane == 0) tc::mbar_expect_tx(&sm.q_place[k], kBytes);
        __syncwarp();
        if (lane < kGroups)
          tc::tma_load_2d(qmap, base + kRingOff + st * kBytes + lane * 4096, 64 * lane, now.t.row + kHalfRows * part + 32 * k, &sm.q_place[k]);
        __syncwarp();
      }
    }
    more = next_piece(sm, nu, lane, a.ws, p);
    if (kScores && more && lane == 0) {
      // the next tile's queries (one piece of memory) to L2
      const int64_t row = int64_t(p.t.row) + kHalfRows * part;
      const int rows = min(kHalfRows, p.t.have - kHalfRows * part);
      if (rows > 0)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(a.q + row * kDqk), "r"(rows * kDqk * 2) : "memory");
    }
    __syncwarp();
    int row = 0;
#pragma unroll 1
    for (int j = 0; j < now.n; ++j, ++u) {
      if ((j & 31) == 0 && j + lane < now.n) row = row_of(a, now.t.seq, now.start(j + lane));
      const int at = __shfl_sync(0xFFFFFFFFu, row, j & 31);
      const uint32_t st = u % kStages;
      if (!wait_warp(sm, &sm.empty[st], ((u / kStages) & 1) ^ 1, a.ws)) return;
      if (lane == 0) {
        if (kScores && part == 0 && at < 0) raise_err(a.ws, CSA2_DEV_PAGE_ID);
        tc::mbar_expect_tx(&sm.full[st], kBytes);
      }
      __syncwarp();
      if (lane < kGroups)
        tc::tma_load_2d(kvmap, base + kRingOff + st * kBytes + lane * (kBytes / kGroups), 64 * (kScores ? lane : 4 * part + lane),
                        max(at, 0) + (kScores ? 32 * part : 0), &sm.full[st]);
      __syncwarp();
    }
  }
}

// ---------------------------------------------------------------------------
// Scores CTAs
// ---------------------------------------------------------------------------
// Queries from the ring into tensor memory: warp k has rows 32 k .. + 31, one place.
__device__ inline void query_role(const WindowArgs& a, LongSmall& sm, uint8_t* base, int k, int lane, uint32_t tmem) {
  LongPiece p;
  uint32_t nu = 0, nt = 0, n = 0;
  while (next_piece(sm, nu, lane, a.ws, p)) {
    if (p.n == 0) continue;
    if (!wait_warp(sm, &sm.q_place[k], nt & 1, a.ws)) return;
    if (!wait_warp(sm, &sm.q_free, (nt++ & 1) ^ 1, a.ws)) return;
    tc::tc_fence_after_sync();
    const uint32_t st = (n + k) % kStages, src = tc::smem_u32(base) + kRingOff + st * kKStage;
    const uint32_t to = tmem + (uint32_t(32 * k) << 16);
#pragma unroll 1
    for (int g = 0; g < 9; ++g)
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        uint32_t v[16];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint4 x = ld_shared16(src + g * 4096 + tc::sw128_offset(lane, 4 * h + i));
          v[4 * i] = x.x; v[4 * i + 1] = x.y; v[4 * i + 2] = x.z; v[4 * i + 3] = x.w;
        }
        tmem_st16_nowait(to + 32 * g + 16 * h, v);
      }
    tmem_wait_st();
    tc::tc_fence_before_sync();
    __syncwarp();
    if (lane == 0) {
      arrive(&sm.empty[st]);
      arrive_remote(peer_addr(&sm.q_full, 0));
    }
    __syncwarp();
    n += uint32_t(p.n);
  }
}

// Second scores CTA: tells the first that its half of a block has come.
__device__ inline void relay_role(const WindowArgs& a, LongSmall& sm, int lane) {
  LongPiece p;
  uint32_t nu = 0, n = 0;
  while (next_piece(sm, nu, lane, a.ws, p)) {
#pragma unroll 1
    for (int j = 0; j < p.n; ++j, ++n) {
      if (!wait_warp(sm, &sm.full[n % kStages], (n / kStages) & 1, a.ws)) return;
      if (lane == 0) arrive_remote(peer_addr(&sm.k_ready[n % kStages], 0));
      __syncwarp();
    }
  }
}

__device__ inline void scores_mma_role(const WindowArgs& a, LongSmall& sm, uint8_t* base, int lane, uint32_t tmem) {
  constexpr uint32_t id = tc::idesc_bf16(kLongRows, kBlk, 0, 0);
  LongPiece p;
  uint32_t nu = 0, nt = 0, n = 0;
  const bool leader = elect_one();
  while (next_piece(sm, nu, lane, a.ws, p)) {
    if (p.n == 0) continue;
    if (!wait_warp(sm, &sm.q_full, nt++ & 1, a.ws)) return;
#pragma unroll 1
    for (int j = 0; j < p.n; ++j, ++n) {
      const uint32_t st = n % kStages, buf = n % kSBufs;
      if (!wait_warp(sm, &sm.full[st], (n / kStages) & 1, a.ws)) return;
      if (!wait_warp(sm, &sm.k_ready[st], (n / kStages) & 1, a.ws)) return;
      if (!wait_warp(sm, &sm.s_empty[buf], ((n / kSBufs) & 1) ^ 1, a.ws)) return;
      tc::tc_fence_after_sync();
      if (leader) {
        const uint64_t bd = tc::smem_desc(tc::smem_u32(base + kRingOff + st * kKStage), 16, 1024, 2);
        const uint32_t d = tmem + kSCol + buf * kBlk;
#pragma unroll 1
        for (int g = 0; g < 9; ++g)
#pragma unroll
          for (int k4 = 0; k4 < 4; ++k4) mma_ts(d, tmem + g * 32 + k4 * 8, bd + ((g * 4096 + k4 * 32) >> 4), id, g + k4 > 0);
        commit_to(&sm.empty[st], 0x3);
        commit_to(&sm.s_full[buf], 0x3);
        if (j == p.n - 1) commit_to(&sm.q_free, 0x3);
      }
      __syncwarp();
    }
  }
}

// The lowest n bits.
__device__ inline uint64_t below(int n) { return n <= 0 ? 0 : n >= 64 ? ~0ull : (1ull << n) - 1; }
// Of the block's positions in `among` (the same for the warp), up to the last, those whose cache rows (the first's:
// `row`) hold values that are no numbers.
__device__ __noinline__ uint64_t not_finite(const WindowArgs& a, int row, int last, uint64_t among, int lane) {
  uint64_t found = 0;
#pragma unroll 1
  for (int e = 0; e < kBlk && e <= last; ++e) {
    if (!(among >> e & 1)) continue;
    const uint4* at = reinterpret_cast<const uint4*>(a.kv + (int64_t(row) + e) * kDqk);
    const bool finite = bf16x8_finite(__ldg(at + lane)) && bf16x8_finite(__ldg(at + 32 + lane));
    if (!__all_sync(0xFFFFFFFFu, finite)) found |= 1ull << e;
  }
  return found;
}

// Warp rw: rows 32 (rw % 4) .. + 31 of the CTA's (one a lane), of every block n with n % 2 = rw / 4: the two
// warps of a row take turns, each with two block periods for the latencies of a block.  What must go in
// order is the reference: block n's warp takes it from block n - 1's as soon as that one has its maximum,
// and hands it on (across tiles, too, where it says nothing but that its place is free).
__device__ inline void softmax_role(const WindowArgs& a, LongSmall& sm, uint8_t* base, int part, int rw, int lane, uint32_t tmem) {
  const int wq = rw & 3, half = rw >> 2, r = 32 * wq + lane;
  const uint32_t lanes = tmem + (uint32_t(32 * wq) << 16);
  const float c = score_to_log2(a);
  LongPiece p;
  uint32_t nu = 0, n = 0;
  while (next_piece(sm, nu, lane, a.ws, p)) {
    // positions this row sees: t <= last, t >= first or t < sinks
    const int tr = kHalfRows * part + r, last = tr < p.t.have ? p.t.pos + over_heads(a, p.t.rem + tr) : -1;
    const int first = last - a.window + 1;
    const bool whole = p.t.have == kLongRows;
    float own = -INFINITY, sum = 0.0f;               // reference of this warp's last block, its sum under it
    int j = int((half ^ n) & 1), row = j < p.n ? row_of(a, p.t.seq, p.start(j)) : 0;
    const uint32_t n0 = n;
    for (n += uint32_t(j); j < p.n; j += 2, n += 2) {
      const uint32_t buf = n % kSBufs, slot = n % kPSlots;
      const int t0 = p.start(j);
      const bool lost = row < 0;
      if (j + 2 < p.n) row = row_of(a, p.t.seq, p.start(j + 2));
      // whether every row of the tile sees the whole block: the same for all warps of both CTAs
      const bool edge = !whole || t0 + kBlk - 1 > p.t.pos || (t0 <= p.t.last - a.window && t0 + kBlk > a.sinks);
      uint8_t* ps = base + slot * kPBytes;
      if (!wait_warp(sm, &sm.s_full[buf], (n / kSBufs) & 1, a.ws)) return;
      tc::tc_fence_after_sync();
      float x[64];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float y[32];
        tc::tmem_ld32(lanes + kSCol + buf * kBlk + 32 * h, y);
#pragma unroll
        for (int i = 0; i < 32; ++i) x[32 * h + i] = y[i];
      }
      tc::tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) arrive_remote(peer_addr(&sm.s_empty[buf], 0));
      if (a.scale < 0.0f) {
#pragma unroll
        for (int i = 0; i < 64; ++i) x[i] = -x[i];
      }
      uint32_t hidden[2] = {0, 0};                   // positions whose scores are no numbers
      if (edge || lost) {
        const int hi = lost ? -1 : last - t0, lo = first - t0, sk = a.sinks - t0;
        float any = 0.0f;                            // 0, or NaN where a score is no number
#pragma unroll
        for (int i = 0; i < 64; ++i) any = fmaf(x[i], 0.0f, any);
        if (__any_sync(0xFFFFFFFFu, any != 0.0f)) {
#pragma unroll
          for (int i = 0; i < 64; ++i)
            if (__any_sync(0xFFFFFFFFu, !(fabsf(x[i]) < INFINITY))) hidden[i >> 5] |= 1u << (i & 31);
          // Of those whose values are not numbers either, which the values CTAs hide from all rows, the rows that
          // see them become NaN by their sums.  (Else a score of -inf, by the rotary channels alone, is weight 0, and
          // one of +inf makes NaN by itself.)
          const uint64_t see = below(hi + 1) & (~below(lo) | below(sk));
          if (!lost && (not_finite(a, row_of(a, p.t.seq, t0), p.t.last - t0, uint64_t(hidden[1]) << 32 | hidden[0], lane) & see)) sum = NAN;
        }
#pragma unroll
        for (int i = 0; i < 64; ++i) x[i] = i <= hi && (i >= lo || i < sk) ? x[i] : -INFINITY;
      }
      float t4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
      for (int i = 4; i < 64; i += 4)
#pragma unroll
        for (int k = 0; k < 4; ++k) t4[k] = fmaxf(t4[k], x[i + k]);
      const float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3]));
      float before = -INFINITY;
      if (n > 0) {
        if (!wait_warp(sm, &sm.ref_full[half ^ 1][wq], ((n - 1) >> 1) & 1, a.ws)) return;
        if (n != n0) before = sm.ref[half ^ 1][r];
      }
      float ref = before, alpha = 1.0f;
      if ((top - ref) * c > kWinSlack) {             // (no score yet: NaN, or inf)
        ref = top;                                   // the largest weight so far is 1, which bf16 holds exactly
        if (before != -INFINITY) alpha = ex2((before - ref) * c);
      }
      sm.ref[half][r] = ref;
      __syncwarp();
      if (lane == 0) arrive(&sm.ref_full[half][wq]);
      if (own != ref && own != -INFINITY) sum *= ex2((own - ref) * c);     // (no reference yet: 0, or NaN)
      own = ref;
      const float sub = ref == -INFINITY ? 0.0f : ref;
      if (!wait_warp(sm, &sm.p_free[slot], ((n / kPSlots) & 1) ^ 1, a.ws)) return;
      const uint64_t cc = pack2(c, c), ss = pack2(-sub, -sub);
      uint64_t acc[2] = {0, 0};                      // +0, +0
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint32_t pk[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float p0, p1;
          unpack2(mul2(add2(pack2(x[8 * i + 2 * k], x[8 * i + 2 * k + 1]), ss), cc), p0, p1);
          p0 = ex2(p0);
          p1 = ex2(p1);
          acc[k & 1] = add2(acc[k & 1], pack2(p0, p1));
          pk[k] = bf16x2_rn(p0, p1);
        }
        *reinterpret_cast<uint4*>(ps + tc::sw128_offset(r, i)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
      }
      {
        float s0, s1;
        unpack2(add2(acc[0], acc[1]), s0, s1);
        sum += s0 + s1;
      }
      sm.meta[slot][wq][0][lane] = alpha;
      sm.meta[slot][wq][1][lane] = sum;
      sm.meta[slot][wq][2][lane] = sub;
      if (lane < 2) sm.meta[slot][wq][3][lane] = __uint_as_float(lane == 0 ? hidden[0] : hidden[1]);
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        const uint32_t to = uint32_t(2 + part), bar = peer_addr(&sm.p_full[slot], to);
        copy_to_peer(peer_addr(ps + wq * 4096, to), ps + wq * 4096, 4096, bar);
        copy_to_peer(peer_addr(&sm.meta[slot][wq][0][0], to), &sm.meta[slot][wq][0][0], kMetaWarp, bar);
      }
      __syncwarp();
    }
    n = n0 + uint32_t(p.n);
  }
}

// ---------------------------------------------------------------------------
// Values CTAs
// ---------------------------------------------------------------------------
// Hands each slot of P back once its products are done.
__device__ inline void slot_role(const WindowArgs& a, LongSmall& sm, int part, int lane) {
  LongPiece p;
  uint32_t nu = 0, n = 0;
  while (next_piece(sm, nu, lane, a.ws, p)) {
#pragma unroll 1
    for (int j = 0; j < p.n; ++j, ++n) {
      const uint32_t slot = n % kPSlots;
      if (!wait_warp(sm, &sm.pv_done[slot], (n / kPSlots) & 1, a.ws)) return;
      if (lane == 0) {
        tc::mbar_expect_tx(&sm.p_full[slot], kPBytes + 4 * kMetaWarp);
        arrive_remote(peer_addr(&sm.p_free[slot], uint32_t(part)));
      }
      __syncwarp();
    }
  }
}

__device__ inline void values_mma_role(const WindowArgs& a, LongSmall& sm, uint8_t* base, int lane, uint32_t tmem) {
  constexpr uint32_t id = tc::idesc_bf16(kLongRows, 256, 0, 1);
  LongPiece p;
  uint32_t nu = 0, nt = 0, n = 0;
  const bool leader = elect_one();
  while (next_piece(sm, nu, lane, a.ws, p)) {
    if (p.n == 0) continue;
    if (!wait_warp(sm, &sm.o_free, (nt++ & 1) ^ 1, a.ws)) return;
#pragma unroll 1
    for (int j = 0; j < p.n; ++j, ++n) {
      const uint32_t st = n % kStages, slot = n % kPSlots;
      // both CTAs have seen P and the values arrive
      if (!wait_warp(sm, &sm.corr[slot], (n / kPSlots) & 1, a.ws)) return;
      tc::tc_fence_after_sync();
      if (leader) {
        const uint64_t ad = tc::smem_desc(tc::smem_u32(base + slot * kPBytes), 16, 1024, 2);
        const uint64_t bd = tc::smem_desc(tc::smem_u32(base + kRingOff + st * kVStage), 8192, 1024, 2);
#pragma unroll
        for (int ks = 0; ks < kBlk / 16; ++ks)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            mma_ss(tmem + h * 256, ad + ((ks * 32) >> 4), bd + ((h * 2 * 8192 + ks * 2048) >> 4), id, j > 0 || ks > 0);
        commit_to(&sm.empty[st], 0xC);
        commit_to(&sm.pv_done[slot], 0xC);
      }
      __syncwarp();
    }
  }
}

// Values that are no numbers become 0: of the positions in `hidden`, every eighth.
__device__ __noinline__ void hide_values(uint8_t* stage, uint64_t hidden, int rw, int lane) {
#pragma unroll 1
  for (int e = rw; e < kBlk; e += kRowWarps) {
    if (!(hidden >> e & 1)) continue;
    uint4* at = reinterpret_cast<uint4*>(stage + (lane >> 3) * 8192 + tc::sw128_offset(e, lane & 7));
    if (!bf16x8_finite(*at)) *at = make_uint4(0, 0, 0, 0);
  }
  tc::fence_proxy_async_smem();
}

// Warp rw: rows 32 (rw % 4) .. + 31 (one a lane), output columns 256 (rw / 4) .. + 255, which are 128 channels
// from each CTA's half.
template <bool kJoin>
__device__ inline void output_role(const WindowArgs& a, LongSmall& sm, uint8_t* base, int part, int rw, int lane, uint32_t tmem) {
  const int wq = rw & 3, col0 = 256 * (rw >> 2), r = 32 * wq + lane;
  const uint32_t lanes = tmem + (uint32_t(32 * wq) << 16) + uint32_t(col0);
  const float c = score_to_log2(a);
  uint8_t* stage = base + kOutOff + rw * 4096;
  LongPiece p;
  uint32_t nu = 0, n = 0;
  while (next_piece(sm, nu, lane, a.ws, p)) {
    const int tr = kHalfRows * part + r, have = p.t.have - (tr - lane);   // rows from the warp's first on that exist
    const int64_t g0 = int64_t(p.t.row) + tr - lane;
    float prev = -INFINITY;
    if (kJoin && lane < have) prev = a.prev_lse[g0 + lane];
    // (Read before any of the tile's lse is written, which may be the same place: that comes after all warps'
    // corr.  Where there are no blocks, what is written is what was read.)
    if (kJoin) prev = __shfl_sync(0xFFFFFFFFu, prev, lane);
    const int ch = lane & 7;
    const int64_t at = g0 * kLatent + 8 * ch;
    // the other attention's outputs, whole rows of 128 bytes an instruction, a step ahead (not those of rows of
    // which it has seen nothing, or that do not exist: their bit in `use` is 0)
    const auto channel_of = [&](int col) { return (col0 >> 1) + (col & 127) + ((col & 128) << 1); };
    const uint32_t use = kJoin ? __ballot_sync(0xFFFFFFFFu, prev != -INFINITY) : 0;
    uint4 ahead[kJoin ? 8 : 1];
    const auto fetch = [&](int col) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int row = 4 * i + lane / 8;
        uint4 v = make_uint4(0, 0, 0, 0);
        if (use >> row & 1) v = *reinterpret_cast<const uint4*>(a.prev_out + at + int64_t(row) * kLatent + channel_of(col));
        ahead[kJoin ? i : 0] = v;
      }
    };
    if (kJoin) fetch(0);
    // sums of the even and the odd blocks, each under the reference of its last block
    float sum = 0.0f, sub = 0.0f, sum_b = 0.0f, sub_b = 0.0f;
#pragma unroll 1
    for (int j = 0; j < p.n; ++j, ++n) {
      const uint32_t slot = n % kPSlots, st = n % kStages;
      if (!wait_warp<true>(sm, &sm.p_full[slot], (n / kPSlots) & 1, a.ws)) return;
      const float alpha = sm.meta[slot][wq][0][lane];
      sum_b = sum;
      sub_b = sub;
      sum = sm.meta[slot][wq][1][lane];
      sub = sm.meta[slot][wq][2][lane];
      uint32_t h0 = 0, h1 = 0;
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        h0 |= __float_as_uint(sm.meta[slot][k][3][0]);
        h1 |= __float_as_uint(sm.meta[slot][k][3][1]);
      }
      if (!wait_warp(sm, &sm.full[st], (n / kStages) & 1, a.ws)) return;
      if (h0 | h1) hide_values(base + kRingOff + st * kVStage, uint64_t(h1) << 32 | h0, rw, lane);
      if (__any_sync(0xFFFFFFFFu, alpha != 1.0f)) {
        // the outputs so far, once their products are done, to the new reference
        const uint32_t m = n - 1;
        if (!wait_warp(sm, &sm.pv_done[m % kPSlots], (m / kPSlots) & 1, a.ws)) return;
        tc::tc_fence_after_sync();
#pragma unroll 1
        for (int col = 0; col < 256; col += 8) {
          float v[8];
          tc::tmem_ld8(lanes + col, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] *= alpha;
          tc::tmem_st8(lanes + col, v);
        }
        tc::tc_fence_before_sync();
      }
      __syncwarp();
      if (lane == 0) arrive_remote(peer_addr(&sm.corr[slot], 2));
    }
    if (p.n > 0) {
      const uint32_t m = n - 1;
      if (!wait_warp(sm, &sm.pv_done[m % kPSlots], (m / kPSlots) & 1, a.ws)) return;
      tc::tc_fence_after_sync();
    }
    if (sum_b != 0.0f) sum += sum_b * ex2((sub_b - sub) * c);
    float mine = sum != 0.0f ? 1.0f / sum : 0.0f, other = 0.0f;          // NaN stays NaN
    float lse = sum != 0.0f ? fmaf(sub, c, log2f(sum)) * 0.6931471805599453f : -INFINITY;
    if (kJoin && prev != -INFINITY) {
      const float most = fmaxf(lse, prev), x0 = expf(lse - most), x1 = expf(prev - most);
      mine *= x0 / (x0 + x1);
      other = x1 / (x0 + x1);
      lse = most + logf(x0 + x1);
    }
    if (col0 == 0 && lane < have) a.lse[g0 + lane] = lse;
    const auto chunk_at = [&](int row, int ch) { return row * 128 + ((ch ^ (row & 7)) << 4); };
#pragma unroll 1
    for (int col = 0; col < 256; col += 64) {
      const int channel = channel_of(col);
      if (kJoin) {
#pragma unroll
        for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(stage + chunk_at(4 * i + lane / 8, ch)) = ahead[i];
        if (col < 192) fetch(col + 64);
        __syncwarp();
      }
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float v[32];
        uint4 o[kJoin ? 4 : 1];
        if (kJoin) {
#pragma unroll
          for (int i = 0; i < 4; ++i) o[i] = *reinterpret_cast<const uint4*>(stage + chunk_at(lane, 4 * h + i));
        }
        if (p.n > 0) {
          tc::tmem_ld32(lanes + col + 32 * h, v);
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) v[i] = 0.0f;
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          uint32_t w[4] = {0, 0, 0, 0};
          if (kJoin) {
            const uint4 x = o[kJoin ? i : 0];
            w[0] = x.x; w[1] = x.y; w[2] = x.z; w[3] = x.w;
          }
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            float lo = v[8 * i + 2 * k] * mine, up = v[8 * i + 2 * k + 1] * mine;
            if (kJoin) {
              lo = fmaf(other, __uint_as_float(w[k] << 16), lo);
              up = fmaf(other, __uint_as_float(w[k] & 0xFFFF0000u), up);
            }
            w[k] = bf16x2_rn(lo, up);
          }
          *reinterpret_cast<uint4*>(stage + chunk_at(lane, 4 * h + i)) = make_uint4(w[0], w[1], w[2], w[3]);
        }
      }
      __syncwarp();
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const int row = 4 * i + lane / 8;
        if (row < have)
          *reinterpret_cast<uint4*>(a.out + at + int64_t(row) * kLatent + channel) = *reinterpret_cast<const uint4*>(stage + chunk_at(row, ch));
      }
      __syncwarp();
    }
    if (p.n > 0) {
      tc::tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) arrive_remote(peer_addr(&sm.o_free, 2));
    }
  }
}

template <bool kJoin>
__global__ void __cluster_dims__(4, 1, 1) __launch_bounds__(kLongThreads, 1)
    window_long_kernel(const __grid_constant__ WindowArgs a, const __grid_constant__ WindowLongMaps m) {
  extern __shared__ __align__(1024) uint8_t base[];  // 1024-byte aligned: checked below
  __shared__ LongSmall sm;
  const int tid = threadIdx.x, lane = tid & 31, wid = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);   // the same for the warp, to the compiler too
  const int rank = blockIdx.x % 4, part = rank % 2;
  const bool scores = rank < 2;
  if (tc::smem_u32(base) & 1023u) {                  // never, as laid out; the same in every CTA
    pdl_wait();
    if (tid == 0) raise_err(a.ws, CSA2_DEV_TIMEOUT);
    return;
  }
  if (wid == 0) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::smem_u32(&sm.tmem_slot)), "r"(512u) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
  if (tid == 0) {
    for (int i = 0; i < kStages; ++i) {
      tc::mbar_init(&sm.full[i], 1);
      tc::mbar_init(&sm.empty[i], 1);
      tc::mbar_init(&sm.k_ready[i], 1);
      tc::mbar_init(&sm.q_place[i], 1);
    }
    for (int i = 0; i < kSBufs; ++i) {
      tc::mbar_init(&sm.s_full[i], 1);
      tc::mbar_init(&sm.s_empty[i], 8);              // four warps in each CTA
    }
    tc::mbar_init(&sm.q_full, 8);
    tc::mbar_init(&sm.q_free, 1);
    for (int i = 0; i < 8; ++i) tc::mbar_init(&sm.ref_full[i >> 2][i & 3], 1);
    for (int i = 0; i < kPSlots; ++i) {
      tc::mbar_init(&sm.p_free[i], 1);
      tc::mbar_init(&sm.p_full[i], 1);
      tc::mbar_init(&sm.corr[i], 2 * kRowWarps);
      tc::mbar_init(&sm.pv_done[i], 1);
    }
    tc::mbar_init(&sm.o_free, 2 * kRowWarps);
    tc::mbar_init(&sm.drain, 1);
    // who follows the plan: scores: softmax, queries, copies, and products or the relay; values: outputs, copies, slots, products
    const uint32_t readers = scores ? kRowWarps + 4 + 2 : kRowWarps + 2 + (part == 0 ? 1 : 0);
    for (int i = 0; i < kPlanSlots; ++i) {
      tc::mbar_init(&sm.plan_full[i], 1);
      tc::mbar_init(&sm.plan_empty[i], readers);
    }
    sm.abort = 0;
    sm.bad = 0;
    sm.tiles = 0;
    tc::fence_mbar_init();
    if (!scores)
      for (int i = 0; i < kPSlots; ++i) tc::mbar_expect_tx(&sm.p_full[i], kPBytes + 4 * kMetaWarp);
  }
  pdl_wait();
  pdl_launch_dependents();
  __syncthreads();
  Sequences<kLongRows> first = {0, 0, 0, 0, 0, 0};
  if (wid == kPlanWarp) first.load(a, lane);         // on their way while the tiles are counted
  // Starts out of order are reported and the call writes nothing.
  {
    const bool paged = a.page_table != nullptr;
    int tiles = 0;
    bool bad = false;
    for (int b = tid; b < a.batch; b += kLongThreads) {
      const int s0 = __ldg(a.q_start + b), s1 = __ldg(a.q_start + b + 1);
      if (s0 < 0 || s1 < s0 || s1 > a.total_q) {
        bad = true;
        continue;
      }
      if (blockIdx.x == 0) check_ctx(__ldg(a.ctx_len + b), a.d, paged, a.ws);
      tiles += tiles_of<kLongRows>(a, s1 - s0);
    }
    if (bad) atomicOr(&sm.bad, 1);
    tiles = __reduce_add_sync(0xFFFFFFFFu, tiles);
    if (lane == 0 && tiles > 0) atomicAdd(&sm.tiles, tiles);
  }
  tc::tc_fence_before_sync();
  __syncthreads();
  tc::tc_fence_after_sync();
  // every CTA's barriers stand before another writes into it
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  const uint32_t tmem = sm.tmem_slot;
  const int tiles = sm.bad ? 0 : sm.tiles, cluster = blockIdx.x / 4, clusters = gridDim.x / 4;
  if (blockIdx.x == 0 && tid == 0 && sm.bad) raise_err(a.ws, CSA2_DEV_Q_START);
  if (wid == kPlanWarp) {
    plan_role(a, sm, cluster, tiles, clusters, scores ? -1 : part, first, lane);
  } else if (scores) {
    if (wid < kRowWarps) softmax_role(a, sm, base, part, wid, lane, tmem);
    else if (wid < kMmaWarp) query_role(a, sm, base, wid - kQueryWarp0, lane, tmem);
    else if (wid == kMmaWarp && part == 0) scores_mma_role(a, sm, base, lane, tmem);
    else if (wid == kLoadWarp) load_role<true>(a, sm, base, part, lane, &m.q, &m.keys);
    else if (wid == kAuxWarp && part == 1) relay_role(a, sm, lane);
  } else {
    if (wid < kRowWarps) output_role<kJoin>(a, sm, base, part, wid, lane, tmem);
    else if (wid == kMmaWarp && part == 0) values_mma_role(a, sm, base, lane, tmem);
    else if (wid == kLoadWarp) load_role<false>(a, sm, base, part, lane, nullptr, &m.values);
    else if (wid == kAuxWarp) slot_role(a, sm, part, lane);
  }
  // the thread that issued the MMAs sees them done (they are, unless a wait gave up)
  __syncwarp();
  if (wid == kMmaWarp && part == 0) {
    if (elect_one()) {
      commit_to(&sm.drain, uint16_t(1u << rank));
      wait_slow<false>(sm, &sm.drain, 0, a.ws);
    }
    __syncwarp();
  }
  // after a wait that gave up, copies may still be on their way: they land within microseconds
  if (*reinterpret_cast<volatile int*>(&sm.abort)) {
    const uint64_t t0 = tc::globaltimer_ns();
    while (tc::globaltimer_ns() - t0 < 2000000ull) {
    }
  }
  __syncwarp();
  tc::tc_fence_before_sync();
  __syncthreads();
  tc::tc_fence_after_sync();
  // no CTA leaves (or frees a pair's tensor memory) while another may still write into it
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (wid == 0) asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u));
}

}  // namespace

// Clusters that run at the same time on the current device, asked once per device.
int window_long_clusters(bool join) {
  static std::atomic<int> known[2][kMaxDevices];
  static KernelAttrs attrs[2];
  auto kernel = join ? window_long_kernel<true> : window_long_kernel<false>;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  const bool slot = dev >= 0 && dev < kMaxDevices;
  if (slot) {
    const int n = known[join][dev].load(std::memory_order_relaxed);
    if (n > 0) return n;
  }
  if (prepare_kernel(kernel, size_t(kLongSmem), false, attrs[join]) != cudaSuccess) return 0;
  const int most = device_sms() / 4;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(unsigned(4 * most));
  cfg.blockDim = dim3(kLongThreads);
  cfg.dynamicSmemBytes = size_t(kLongSmem);
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = 4;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();
    n = most;
  }
  n = n < 1 ? 1 : n > most ? most : n;
  if (slot) known[join][dev].store(n, std::memory_order_relaxed);
  return n;
}

cudaError_t launch_window_long(const WindowArgs& a, const WindowLongMaps& m, int64_t tiles, cudaStream_t st) {
  const int clusters = window_long_clusters(a.prev_out != nullptr);
  if (clusters < 1) return cudaErrorInvalidConfiguration;
  auto kernel = a.prev_out ? window_long_kernel<true> : window_long_kernel<false>;
  cudaError_t e;
  CSA2_PROFILED(st, "window_attn_long",
                (e = launch_pdl(kernel, dim3(unsigned(4 * min64(clusters, max64(tiles, 1)))), dim3(kLongThreads), size_t(kLongSmem), st, 1, a, m)));
  return e;
}

}  // namespace csa2
