// dense.cu -- dense attention of a chunk of new tokens over the (paged) FP4
// main-KV cache, on the tcgen05 tensor cores.
//
// Rows r = (query token, head) of a ragged batch; for every cache position t
// that row r sees (causal, optionally a window; or all positions):
//   s_rt = scale * q_r . [dq(latent_t) ; rope_t],  out_r = sum_t softmax_t(s_rt) dq(latent_t),
//   lse_r = log sum_t exp(s_rt).
// One latent row serves all heads (foosynaptic atlas "DeepSeek-V4.1-Flash 梗概",
// section 3.2: shared main KV), so the tokens and heads of a sequence are simply
// rows of one matrix, cut into tiles of 128.
//
// Scores and outputs on different SMs.  128 rows x 512 fp32 outputs fill the tensor memory
// of an SM, so scores and outputs cannot live on one.  A cluster divides the work by
// kind instead:
//   scores CTA   queries resident in tensor memory (288 columns); a block of 64 positions
//       is widened from FP4 to fp16 (exact: 6 significant bits, 2^-10 .. 2688) in shared
//       memory, its rope keys stay bf16; S[128 x 64] = Q . K^T (M 128, N 64, K 512 fp16 +
//       64 bf16 -> fp32); softmax, one thread a row; P as fp16 goes to the values CTA by
//       an asynchronous copy between their shared memories;
//   values CTA   widens the same block's latents to fp16,
//       O[128 x 512] += P . V (M 128, N 2 x 256, K 64).
// Data flow one way only, so each side runs ahead through its rings (raw bytes of the
// next blocks, 2 blocks of keys or values, 3 score buffers, 3 blocks of P).  Tensor work
// a block: 1,152 and 1,024 cycles; nothing is computed twice but the widening.
//   G = 1: clusters of 2 CTAs, tiles of 128 rows;
//   G = 2: clusters of 4, tiles of 256 rows: two scores and two values CTAs, each pair one
//       product (cta_group::2: own rows, shared keys or values, of which each CTA widens and
//       holds half).  Half of the widening per row, and half of the shared-memory reads for
//       the shared operand.
//
// Softmax reference: kept per row as an integer (base-2) and raised only when a
// block's maximum passes it by more than 8, so the outputs are rarely rescaled, and
// then by a power of two.  P = 2^(x - ref + 7) <= 2^15 fits fp16 (rounded to 11 bits where
// bf16 has 8); terms 2^-31 below the reference are the first to be lost.  Sums are
// fp32, of the unrounded P.  The rounding of P moves an output by at most 2^-11 of
// sum p |v|, its bf16 form by 2^-8 of itself: against 64 bits the error is that of
// unrounded P to two digits (1.7e-3 relative; 1e-5 more with few positions).  P in two
// parts would double the values product, 1,024 of a block's tensor cycles.
//
// Work division: the (tile, block) pairs of the call are counted by a plan kernel
// and cut into equal runs, one per cluster, whatever the shape: a decode batch splits
// its long contexts, a prompt gives each cluster whole tiles.  A tile cut by a
// boundary leaves partial outputs (fp32, at most two per cluster) that a merge kernel
// joins in a fixed order: results are the same from call to call.
//
// Roles of a CTA's 28 warps: 8 row warps (softmax / outputs), 16 widening warps (which also
// bring the queries into tensor memory), one that issues the MMAs, one that copies blocks
// from the cache, and in a values CTA one that hands slots of P back.
//
// Measured (GB300; 1,933 TFLOP/s measured bf16 rate, 2 * 1088 flop a visible (row, position)):
// 2,048 tokens x 64 heads on 32,768 positions 5.4-5.6 ms, 1.62-1.68 PFLOP/s (84-87 %); bound by the
// tensor pipe and the shared-memory bandwidth that feeds it.  8 contexts of 131,072 with
// one token 0.31 ms, 0.47 PFLOP/s (64 of 128 rows of each product are used, and both CTAs
// widen every block: a block every 2,800 cycles, of which its product takes 1,152).  Whole
// prompts of 509 to 1,310 tokens 0.42 ms, 0.5 PFLOP/s: a tile costs about 8,000 cycles
// before its first block (its queries, 147 KB a CTA, cannot come before the last product of
// the tile before it), and runs of equal blocks hold 9 to 67 tiles, so the call waits for the
// clusters that have the first, short tiles of the prompts.
#include <cooperative_groups.h>
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "common.cuh"
#include "dense.cuh"
#include "kernels.cuh"
#include "profile.cuh"
#include "tc.cuh"
#include "tmap.cuh"

namespace csa2 {

namespace {

constexpr int kRowWarps = 8;                        // lane quarter (w % 4) x (w / 4): the scores of every other block
                                                    // (scores CTA), half of the output channels (values CTA)
constexpr int kConvWarp0 = kRowWarps, kConvWarps = 16;   // two groups of 8, one for each ring stage
constexpr int kMmaWarp = kRowWarps + kConvWarps;
// warp kMmaWarp: query copies and MMAs (scores CTA), MMAs (values CTA); then copies from
// the cache, and rope keys (scores CTA, G 1) or slots of P (values CTA); one more makes
// them a warpgroup and only gives its registers
constexpr int kDenseThreads = (kMmaWarp + 4) * 32;

constexpr int kReg = kDenseBlk * 128;               // 64 channels x 64 positions of 16-bit: 8 KB
constexpr int kMaxPSlots = 3;
constexpr int kPBytes = kDenseTile * 128;           // P[128 x 64] fp16
constexpr int kKStages = 2;
constexpr int kKBytes = 9 * kReg;                   // 576 channels of a block's positions, or of 64 query rows
constexpr int kVBytes = 8 * kReg;                   // 512 channels

// Shared memory of a CTA: slots of P, the ring of keys or values, raw bytes of the
// blocks to widen as they come from the cache, in two stages (G 1: 32 rows, half a block;
// G 2: a block's 32 rows in a scores CTA, half of its codes in a values CTA).
template <int G>
struct Lay {
  static constexpr int kPSlots = 3;
  static constexpr int kRawStages = 2;
  static constexpr int kKvOff = kPSlots * kPBytes;
  static constexpr int kRawOff = kKvOff + kKStages * kKBytes;
  static constexpr int kRawRope = 32 * kRope * 2;                     // scores CTA only
  static constexpr int kRawCodes = 32 * kCodesPerRow;                 // (a values CTA at G 2: 64 rows x 128 bytes)
  static constexpr int kRawStage = kRawRope + kRawCodes + 32 * kScalesPerRow;   // (a values CTA at G 2: 64 rows of scales, no rope)
  // values CTA: output staging, 2 G KB a warp, behind the values (at G 2 they are half of a stage)
  static constexpr int kStageOff = G == 1 ? kKvOff + kKStages * kVBytes : kKvOff + (kKStages - 1) * kVBytes + kVBytes / 2;
  static constexpr int kSmem = kRawOff + kRawStages * kRawStage;
  static_assert(kStageOff + kRowWarps * 2048 * G <= kRawOff, "output staging of the values CTA");
  static_assert(G == 1 || kRawCodes + kDenseBlk * kScalesPerRow <= kRawStage, "raw bytes of a values CTA");
  // beside at most 8 KB of named variables; the dynamic part starts on a multiple of its alignment
  static_assert(kRawStage % 1024 == 0 && kSmem + 8192 <= 232448, "alignment and size of shared memory");
};

constexpr uint32_t kSCol = 320;                     // score buffers behind the 288 query columns
constexpr int kSBufs = 3;
constexpr int kMetaWarp = 3 * 32 * 4;               // alpha, sum, reference of a warp's rows

struct DenseSmall {
  uint64_t raw_full[2], raw_empty[2];
  uint64_t kv_full[kKStages], kv_empty[kKStages];
  uint64_t s_full[kSBufs], s_empty[kSBufs];
  uint64_t q_turn[kKStages], q_place[kKStages];     // a ring stage free for queries; holding them
  uint64_t q_full;
  uint64_t p_free[kMaxPSlots];                         // scores CTA: slot read by the values CTA (remote arrival)
  uint64_t p_full[kMaxPSlots];                         // values CTA: bytes of P and meta have arrived
  uint64_t corr[kMaxPSlots];                           // values CTA: outputs brought to the slot's reference
  uint64_t pv_done[kMaxPSlots];
  uint64_t o_free;
  uint64_t drain;
  uint32_t tmem_slot;
  int abort;
  int raw_rows[2];                                  // rows of the raw bytes before the context's end (0: bad page)
  __align__(16) float meta[kMaxPSlots][4][3][32];
  uint16_t swap[4][kDenseTile];                     // largest magnitudes of the queries, between a row's four warps
  int8_t q_shift[4][kDenseTile];                    // power of two each query row was scaled by, of four tiles in turn
  float ref[2][kDenseTile];                         // softmax reference, handed from block to block
};

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

// Arrival on another CTA's barrier.  What it hands over is never read by ordinary loads
// of that CTA: shared memory that the tensor cores read (made visible to them by the
// writer's proxy fence before this), tensor memory (ordered by the tcgen05 fences on
// both sides), or a place that is free.  A release at cluster scope, which waits for
// every earlier store of the thread, costs a fifth of the kernel's time instead
// (1.55 against 1.28 ms, 1,216 tokens over 9,408 positions).
__device__ inline void arrive_remote(uint32_t rbar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(rbar) : "memory");
}

__device__ inline void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(tc::smem_u32(bar)) : "memory");
}

// One try, which suspends the thread for a while the hardware chooses.  kCluster: acquires
// what another CTA wrote.
template <bool kCluster>
__device__ inline bool try_wait(uint64_t* bar, uint32_t parity) {
  uint32_t done;
  if constexpr (kCluster)
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done) : "r"(tc::smem_u32(bar)), "r"(parity) : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\t"
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
        "selp.u32 %0, 1, 0, p;\n\t}"
        : "=r"(done) : "r"(tc::smem_u32(bar)), "r"(parity) : "memory");
  return done != 0;
}

// Every wait of the kernel: bounded (200 ms against microseconds; the clock is only read
// after some tries, it takes longer than most waits), and cut short once another role
// of the CTA has given up.  False: the caller's role ends.  The hardware barriers between
// warps have no limit, so a role that ends early still takes part in all those left to it
// (labels `leave`): none of its partners waits there for ever.  (mbarriers in their place
// cost 4 to 12 % of a call: 128K decode batch 306 -> 342 us, prompts 422 -> 445; for the
// queries' barriers alone 1 to 7 %.)
template <bool kCluster>
__device__ __forceinline__ bool wait_slow(DenseSmall& sm, uint64_t* bar, uint32_t parity, uint8_t* ws) {
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
// For a converged warp: one answer for all lanes.  (128K decode batch, 310 us: one lane asking
// for the others 645; a time hint on the wait, of whatever length, 322; some tests without
// suspending before it 333.)
template <bool kCluster = false>
__device__ inline bool wait_warp(DenseSmall& sm, uint64_t* bar, uint32_t parity, uint8_t* ws) {
  return __all_sync(0xFFFFFFFFu, try_wait<kCluster>(bar, parity) || wait_slow<kCluster>(sm, bar, parity, ws));
}

// Arrive on a barrier of the pair's leading CTA (the one that issues its MMAs).
template <int G>
__device__ inline void arrive_leader(uint64_t* bar, int leader) {
  if constexpr (G == 1) arrive(bar);
  else arrive_remote(peer_addr(bar, uint32_t(leader)));
}

// D[tmem] (+)= A * B[smem]^T over one CTA (G 1) or a pair (G 2: rows of both, B
// shared, each CTA holding half of its columns); A in tensor or shared memory.
template <int G>
__device__ inline void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  if constexpr (G == 1)
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(uint32_t(acc)) : "memory");
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
        ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(uint32_t(acc)) : "memory");
}
template <int G>
__device__ inline void mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool acc) {
  if constexpr (G == 1) tc::mma_bf16(d, a, b, idesc, acc);
  else
    asm volatile(
        "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
        "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(uint32_t(acc)) : "memory");
}
// Arrive on `bar` of this CTA (G 1), or of both CTAs in `mask`, once the MMAs so far are done.
template <int G>
__device__ inline void commit_to(uint64_t* bar, uint16_t mask) {
  if constexpr (G == 1) tc::mma_commit(bar);
  else
    asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                 ::"r"(tc::smem_u32(bar)), "h"(mask) : "memory");
}
template <int G>
__device__ inline void tmem_alloc_all(uint32_t* slot) {
  if constexpr (G == 1) tc::tmem_alloc(slot, 512);
  else {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(tc::smem_u32(slot)), "r"(512u)
                 : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
  }
}
template <int G>
__device__ inline void tmem_free_all(uint32_t taddr) {
  if constexpr (G == 1) tc::tmem_dealloc(taddr, 512);
  else asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(512u) : "memory");
}

// Instruction descriptor with fp16 A/B and fp32 accumulation.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int a_mn, int b_mn) {
  return (1u << 4) | (uint32_t(a_mn) << 15) | (uint32_t(b_mn) << 16) | (uint32_t(N >> 3) << 17) |
         (uint32_t(M >> 4) << 24);
}

__device__ inline bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

// Hardware barriers, each for one lane quarter of the softmax warps: the hand-off of the
// reference from the even blocks' warp, from the odd blocks' warp, the start of a tile; and
// for one half of the queries, of the widening warps.
constexpr int kRefBar = 1, kTurnBar = 9, kQueryBar = 13;
__device__ inline void some_arrive(int id, int threads) { asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(threads) : "memory"); }
__device__ inline void some_sync(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }

__device__ inline void st_shared16(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}
__device__ inline uint32_t ld_shared_u16(uint32_t addr) {
  uint16_t v;
  asm volatile("ld.shared.u16 %0, [%1];" : "=h"(v) : "r"(addr) : "memory");
  return v;
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
__device__ inline uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
__device__ inline uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Registers a thread of the calling warpgroup.  72 a thread are launched (seven warps on
// a quarter of the SM allow no more): the widening warps give 16 each and the last
// warpgroup 32, the 8 row warps, which hold 64 scores a thread, take 48.
template <int n>
__device__ inline void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(n)); }
template <int n>
__device__ inline void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(n)); }
constexpr int kLaunchRegs = 72, kConvRegs = 56, kRowRegs = 120, kMmaRegs = 40;
static_assert(kConvWarps * kConvRegs + kRowWarps * kRowRegs + 4 * kMmaRegs <= kLaunchRegs * (kDenseThreads / 32),
              "a split above what was launched would wait for ever");

__device__ inline float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ inline uint32_t f16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ inline uint32_t bf16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// byte i of w: two E2M1 nibbles -> two fp16, exact
template <int i>
__device__ inline uint32_t e2m1_byte_f16x2(uint32_t w) {
  uint32_t h;
  asm("{\n\t.reg .b8 b0, b1, b2, b3;\n\tmov.b32 {b0, b1, b2, b3}, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, b%2;\n\t}"
      : "=r"(h) : "r"(w), "n"(i));
  return h;
}
__device__ inline uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ inline uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// ---------------------------------------------------------------------------
// The blocks of a cluster's run, walked alike by every role.
// ---------------------------------------------------------------------------
struct Item {
  int4 a;             // seq, first row in the sequence, first query token, query tokens
  int4 b;             // context, first block, blocks of the tile, 0
  int blk, n;         // first block (absolute) and blocks of this piece
  bool head, tail;    // the piece starts / ends inside the tile
};
struct Walk {
  const int4* tiles;
  int t, off, left;
  __device__ Walk(const DensePlan& p, int c) {
    const int4 r = __ldg(p.runs + c);
    tiles = p.tiles;
    t = r.x;
    off = r.y;
    left = r.z;
  }
  __device__ bool next(Item& it) {
    if (left <= 0) return false;
    do {
      it.a = __ldg(tiles + 2 * t);
      it.b = __ldg(tiles + 2 * t + 1);
      ++t;
    } while (it.b.z == 0);
    it.blk = it.b.y + off;
    it.n = min(it.b.z - off, left);
    it.head = off > 0;
    it.tail = off + it.n < it.b.z;
    left -= it.n;
    off = 0;
    return true;
  }
};

// The blocks of a run one after the other, with their cache rows.  A warp keeps the
// page ids of up to 32 blocks, one a lane.
struct Cursor {
  Walk walk;
  Item it;
  int i, pages, lane;
  __device__ Cursor(const DensePlan& p, int c, int lane_) : walk(p, c), it{}, i(0), pages(0), lane(lane_) {}
  __device__ void load_pages(const DenseArgs& a) {
    const int at = (i & ~31) + lane;
    if (a.page_table && at < it.n) pages = __ldg(a.page_table + int64_t(it.a.x) * a.d.max_pages + it.blk + at);
  }
  __device__ bool item(const DenseArgs& a, int first = 0) {
    if (!walk.next(it)) return false;
    i = first;
    load_pages(a);
    return true;
  }
  // `by` (1 or 2) blocks on within the item; false behind its end
  __device__ bool step(const DenseArgs& a, int by) {
    const int was = i;
    i += by;
    if (i >= it.n) return false;
    if ((i ^ was) & 32) load_pages(a);
    return true;
  }
  // first cache row of the block, -1 for a page id out of range (all lanes)
  __device__ int64_t row0(const DenseArgs& a) const {
    if (!a.page_table) return int64_t(it.a.x) * a.d.max_ctx + (it.blk + i) * kDenseBlk;
    const int pg = __shfl_sync(0xFFFFFFFFu, pages, i & 31);
    return pg < 0 || pg >= a.d.num_pages ? -1 : int64_t(pg) * kPage;
  }
};

// ---------------------------------------------------------------------------
// A block's bytes come from the cache by TMA, asked for by a warp that runs ahead
// (raw_role), so the widening warps hold no addresses and wait for no loads.  (The same
// bytes by the widening threads' own loads, into registers or by cp.async, 16 bytes
// each: the SM's load path takes half of the kernel's time; 387 against 229 us without
// any loads, 128K decode batch.)
//
// Widening warps (every CTA): E2M1 x E4M3 -> fp16, exact (6 significant bits, 2^-10 ..
// 2688).  A lane takes 16 bytes of codes (32 channels) of one row at a time, lane = 8 *
// piece + row: a quarter-warp reads and stores one 16-byte chunk of 8 rows (all 32 banks,
// 128-byte swizzle).  The rope keys are copied along:
//   G 1: the 16 warps take half a block, 32 rows x 512 channels, together, one piece each;
//   G 2: 8 warps take every other block (those of one ring stage), two pieces each; a
//        scores CTA has 32 of the 64 rows, a values CTA its half of the 512 channels.
// (128K decode batch, kernel alone: 303 us.  Whole blocks in one raw stage, the rope keys
// copied straight into the ring and awaited there: 323; halves, but the rope keys so: 314;
// rows as they lie in the cache by untiled copies: 307; 8 warps on every other block at G 1,
// too: 332.)
// ---------------------------------------------------------------------------
// Copies the run's blocks into the raw stages: boxes of 128 bytes x 32 rows (64-byte boxes
// take the copy engine nearly twice as long), scales in one piece.
template <int G, bool kScores>
__device__ inline void raw_role(const DenseArgs& a, DenseSmall& sm, uint8_t* base, int cl, int part, int lane,
                                const CUtensorMap* codes, const CUtensorMap* rope) {
  constexpr bool kColumns = G == 2 && !kScores;
  constexpr int kRows = kColumns ? 64 : 32;                           // of a raw stage
  constexpr int kStages = Lay<G>::kRawStages;
  constexpr int kCodesAt = kScores ? Lay<G>::kRawRope : 0, kScalesAt = kCodesAt + Lay<G>::kRawCodes;
  constexpr uint32_t kBytes = kScalesAt;
  Cursor cur(a.plan, cl, lane);
  uint32_t n = 0;                                                     // raw stages filled
  for (bool more = cur.item(a); more; more = cur.step(a, 1) || cur.item(a)) {
    const int64_t row0 = cur.row0(a);
    if (kScores && part == 0 && row0 < 0 && lane == 0) raise_err(a.ws, CSA2_DEV_PAGE_ID);
    const int valid = row0 < 0 ? 0 : cur.it.b.x - (cur.it.blk + cur.i) * kDenseBlk;   // of the block
#pragma unroll 1
    for (int half = 0; half < (G == 1 ? 2 : 1); ++half, ++n) {
      const uint32_t st = n % kStages;
      const int first = G == 1 ? 32 * half : kScores ? 32 * part : 0;   // first of the stage's rows in the block
      const int rows = max(0, min(kRows, valid - first));
      const int64_t row = (row0 < 0 ? 0 : row0) + first;
      if (!wait_warp(sm, &sm.raw_empty[st], ((n / kStages) & 1) ^ 1, a.ws)) return;
      if (lane == 0) {
        uint8_t* raw = base + Lay<G>::kRawOff + st * Lay<G>::kRawStage;
        uint64_t* bar = &sm.raw_full[st];
        sm.raw_rows[st] = rows;
        tc::mbar_expect_tx(bar, kBytes + uint32_t(rows * kScalesPerRow));
        uint8_t* c = raw + kCodesAt;
        if (kColumns) {
          tc::tma_load_2d(codes, c, 128 * part, int(row), bar);
          tc::tma_load_2d(codes, c + 4096, 128 * part, int(row) + 32, bar);
        } else {
          tc::tma_load_2d(codes, c, 0, int(row), bar);
          tc::tma_load_2d(codes, c + 4096, 128, int(row), bar);
        }
        if (kScores) tc::tma_load_2d(rope, raw, 0, int(row), bar);
        // valid rows only: the plane may end behind them
        if (rows > 0)
          asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                       ::"r"(tc::smem_u32(raw + kScalesAt)), "l"(a.scales + row * kScalesPerRow), "r"(rows * kScalesPerRow),
                         "r"(tc::smem_u32(bar))
                       : "memory");
      }
      __syncwarp();
    }
  }
}

// 0xFF in each of two scale codes that is a NaN.  Such a scale makes NaN of the scores of the
// rows that see its position, by the keys; taken as 0 among the values it leaves the others
// alone (0 * P).
__device__ inline uint32_t nan_scales(uint32_t two) { return (((two & 0x7F7Fu) + 0x0101u) >> 7 & 0x0101u) * 0xFFu; }

// One 4-byte word of codes: 8 channels under one scale (twice in sc2).
__device__ inline uint4 widen8(uint32_t w, uint32_t sc2) {
  return make_uint4(mul_f16x2(e2m1_byte_f16x2<0>(w), sc2), mul_f16x2(e2m1_byte_f16x2<1>(w), sc2),
                    mul_f16x2(e2m1_byte_f16x2<2>(w), sc2), mul_f16x2(e2m1_byte_f16x2<3>(w), sc2));
}

// The tile's queries, in the ring as two halves of 64 rows, into tensor memory as fp16
// (latent channels) and bf16 (rope): lane quarter w % 4 has the row, its four warps the
// channels.  Each row is scaled by the power of two that brings its largest value into
// [2^14, 2^15): the 8 bits of bf16 are kept for all values down to 2^-28 of the largest,
// smaller ones are off by 2^-39 of it; the softmax takes the power back.  The widening
// warps do this, idle at that time, while the row warps finish the tile before.
template <int G>
__device__ inline bool queries_to_tmem(const DenseArgs& a, DenseSmall& sm, uint8_t* base, int w, int lane, uint32_t tmem,
                                       uint32_t k_item, int place) {
  const int wq = w & 3, part4 = w >> 2, half = wq >> 1, r = wq * 32 + lane, st = (place + half) & 1;
  // both halves: then the products that read the tile before are done, too (both stages were free)
  if (!wait_warp(sm, &sm.q_place[0], k_item & 1, a.ws)) return false;
  if (!wait_warp(sm, &sm.q_place[1], k_item & 1, a.ws)) return false;
  // from here on no way out: a warp takes part in both hardware barriers, or has left before them
  tc::tc_fence_after_sync();
  const uint32_t src = tc::smem_u32(base) + Lay<G>::kKvOff + st * kKBytes;
  const uint32_t row = tc::sw128_offset(r & 63, 0), turn = (r & 7) << 4;       // chunk c of a row: row's base + (c << 4 ^ turn)
  const uint32_t at = src + (row ^ turn);
  uint32_t big[2] = {0, 0};
#pragma unroll 1
  for (int q = part4; q < 18; q += 4)
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 x = ld_shared16(at + (q >> 1) * kReg + ((((q & 1) * 4 + i) << 4) ^ turn));
      big[i & 1] = __vmaxu2(big[i & 1], __vmaxu2(__vmaxu2(x.x & 0x7FFF7FFFu, x.y & 0x7FFF7FFFu), __vmaxu2(x.z & 0x7FFF7FFFu, x.w & 0x7FFF7FFFu)));
    }
  const uint32_t b2 = __vmaxu2(big[0], big[1]);
  sm.swap[part4][r] = uint16_t(max(b2 & 0xFFFFu, b2 >> 16));
  some_sync(kQueryBar + half, 256);
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) top = max(top, uint32_t(sm.swap[i][r]));
  const int k = min(14 + 127 - int(top >> 7), 126);                            // top >> 7: biased exponent of the largest
  const float up = __uint_as_float(uint32_t(127 + k) << 23) * (a.scale < 0.0f ? -1.0f : 1.0f);   // a negative scale negates the queries
  const uint32_t up2 = (__float_as_uint(up) >> 16) * 0x10001u;
  if (part4 == 0) sm.q_shift[k_item & 3][r] = int8_t(k);
#pragma unroll 1
  for (int q = part4; q < 18; q += 4) {
    uint32_t v[16];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 x = ld_shared16(at + (q >> 1) * kReg + ((((q & 1) * 4 + i) << 4) ^ turn));
      v[4 * i] = x.x; v[4 * i + 1] = x.y; v[4 * i + 2] = x.z; v[4 * i + 3] = x.w;
    }
    if (q < 16) {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = f16x2_rn(__uint_as_float(v[i] << 16) * up, __uint_as_float(v[i] & 0xFFFF0000u) * up);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) v[i] = mul_bf16x2(v[i], up2);
    }
    tmem_st16_nowait(tmem + (uint32_t(wq * 32) << 16) + q * 16, v);
  }
  tmem_wait_st();
  tc::tc_fence_before_sync();
  some_sync(kQueryBar + half, 256);
  if (lane == 0) {
    if ((wq & 1) == 0 && part4 == 0) arrive(&sm.kv_empty[st]);                 // the half has been read
    arrive_leader<G>(&sm.q_full, 0);
  }
  __syncwarp();
  return true;
}

template <int G, bool kScores>
__device__ inline void widen_role(const DenseArgs& a, DenseSmall& sm, uint8_t* base, int cl, int part, int w, int lane,
                                  uint32_t tmem) {
  constexpr int kLead = kScores ? 2 : 0;       // ring places of a tile's queries before its blocks
  constexpr uint32_t kStageBytes = kScores ? kKBytes : kVBytes;
  const uint32_t raw0 = tc::smem_u32(base) + Lay<G>::kRawOff, ring = tc::smem_u32(base) + Lay<G>::kKvOff;
  const int p = lane >> 3;
  Walk walk(a.plan, cl);
  Item it = {};
  int place = 0;                               // ring place (mod 2) of the item's start
  if constexpr (G == 1) {
    // a raw stage is 32 rows: one piece a lane, a block in two turns
    const int row = 8 * (w & 3) + (lane & 7), group = w >> 2;         // in the stage; 64 of a row's 256 code bytes
    constexpr uint32_t kCodesAt = kScores ? Lay<1>::kRawRope : 0;
    const bool with_rope = kScores && w < 8;
    const uint32_t o_rope = tc::sw128_offset(row, (w >> 2) * 4 + p);
    const uint32_t src = kCodesAt + (group >> 1) * 4096 + tc::sw128_offset(row, (group & 1) * 4 + p);
    const uint32_t ssrc = kCodesAt + Lay<1>::kRawCodes + row * kScalesPerRow + 2 * (4 * group + p);
    const uint32_t dst = ring + (2 * group + (p >> 1)) * kReg + tc::sw128_offset(row, (p & 1) * 4);
    uint32_t u = 0, v = 0;                     // ring places passed, raw stages used
    for (uint32_t k_item = 0; walk.next(it); ++k_item) {
      // the tile's queries come through the same ring
#pragma unroll 1
      for (int k = 0; k < kLead; ++k, ++u) {
        if (!wait_warp(sm, &sm.kv_empty[u % kKStages], ((u / kKStages) & 1) ^ 1, a.ws)) goto leave_queries;
        if (lane == 0) arrive(&sm.q_turn[u % kKStages]);
      }
      if (kScores && !queries_to_tmem<1>(a, sm, base, w, lane, tmem, k_item, place)) goto leave_queries;
#pragma unroll 1
      for (int i = 0; i < it.n; ++i, ++u) {
        const uint32_t st = u % kKStages;
#pragma unroll 1
        for (int half = 0; half < 2; ++half, ++v) {
          const uint32_t rs = v % Lay<1>::kRawStages, raw = raw0 + rs * Lay<1>::kRawStage;
          if (!wait_warp(sm, &sm.raw_full[rs], (v / Lay<1>::kRawStages) & 1, a.ws)) goto leave;
          const bool have = row < sm.raw_rows[rs];
          const uint4 cw = ld_shared16(raw + src);
          const uint32_t sc = ld_shared_u16(raw + ssrc);
          uint4 rp;
          if (with_rope) rp = ld_shared16(raw + o_rope);
          __syncwarp();
          if (lane == 0) arrive(&sm.raw_empty[rs]);
          // rows behind the context hold anything: their scale is taken as 0 (0 * P stays 0; their scores are masked)
          uint32_t code = have ? sc : 0u;
          if (!kScores) code &= ~nan_scales(code);
          const uint32_t two = e4m3x2_to_f16x2(uint16_t(code));
          const uint32_t s0 = __byte_perm(two, 0, 0x1010), s1 = __byte_perm(two, 0, 0x3232);
          const uint4 w0 = widen8(cw.x, s0), w1 = widen8(cw.y, s0), w2 = widen8(cw.z, s1), w3 = widen8(cw.w, s1);
          if (half == 0 && !wait_warp(sm, &sm.kv_empty[st], ((u / kKStages) & 1) ^ 1, a.ws)) goto leave;
          const uint32_t d = dst + st * kStageBytes + half * 4096;    // 32 rows on; a row's swizzle repeats every 8
          st_shared16(d, w0);
          st_shared16(d ^ 16, w1);
          st_shared16(d ^ 32, w2);
          st_shared16(d ^ 48, w3);
          if (with_rope) st_shared16(ring + st * kStageBytes + 8 * kReg + half * 4096 + o_rope, rp);
        }
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) arrive(&sm.kv_full[st]);
      }
      place = (place + kLead + it.n) & 1;
    }
  } else {
    constexpr int kPieces = 2;
    constexpr int kLeader = kScores ? 0 : G;
    constexpr bool kColumns = !kScores;
    constexpr int kRows = kScores ? 32 : 64;
    constexpr int kRegion = kRows * 128;
    const int g = w >> 3, w8 = w & 7;          // the warp's ring and raw stage
    const int hi = kScores ? w8 >> 2 : 0;      // half of the channels (256) this warp takes
    const int row = 8 * (kScores ? w8 & 3 : w8) + (lane & 7);          // in the stage
    // raw codes (128 bytes of a row; the second piece is 64 bytes on), its scales, first region (the next is two on)
    constexpr uint32_t kCodesAt = kScores ? Lay<G>::kRawRope : 0;
    const uint32_t raw = raw0 + g * Lay<G>::kRawStage;
    const uint32_t src = raw + kCodesAt + hi * kRows * 128 + tc::sw128_offset(row, p);
    const uint32_t ssrc = raw + kCodesAt + Lay<G>::kRawCodes + row * kScalesPerRow + 2 * (8 * (kColumns ? part : hi) + p);
    const uint32_t o_rope = tc::sw128_offset(row, hi * 4 + p);        // rope: one 16-byte chunk a lane
    const uint32_t dst = ring + g * kStageBytes + (4 * hi + (p >> 1)) * kRegion + tc::sw128_offset(row, (p & 1) * 4);
    uint32_t u = 0, v = 0;                     // uses of the ring stage and of the raw stage
    for (uint32_t k_item = 0; walk.next(it); ++k_item) {
      // the tile's queries come through the same ring
      if (kScores) {
        if (!wait_warp(sm, &sm.kv_empty[g], (u & 1) ^ 1, a.ws)) goto leave_queries;
        if (lane == 0) arrive(&sm.q_turn[g]);
        ++u;
        if (!queries_to_tmem<G>(a, sm, base, w, lane, tmem, k_item, place)) goto leave_queries;
      }
#pragma unroll 1
      for (int i = (g - place) & 1; i < it.n; i += 2, ++u, ++v) {
        if (!wait_warp(sm, &sm.raw_full[g], v & 1, a.ws)) goto leave;
        uint4 cw[kPieces], rp;
        uint32_t sc[kPieces];
        const bool have = row < sm.raw_rows[g];
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
          cw[j] = ld_shared16(src ^ (64 * j));
          sc[j] = ld_shared_u16(ssrc + 8 * j);
        }
        if (kScores) rp = ld_shared16(raw + o_rope);
        __syncwarp();
        if (lane == 0) arrive(&sm.raw_empty[g]);
        if (!wait_warp(sm, &sm.kv_empty[g], (u & 1) ^ 1, a.ws)) goto leave;
#pragma unroll
        for (int j = 0; j < kPieces; ++j) {
          uint32_t code = have ? sc[j] : 0u;
          if (!kScores) code &= ~nan_scales(code);
          const uint32_t two = e4m3x2_to_f16x2(uint16_t(code));
          const uint32_t s0 = __byte_perm(two, 0, 0x1010), s1 = __byte_perm(two, 0, 0x3232);
          const uint32_t d = dst + 2 * j * kRegion;
          st_shared16(d, widen8(cw[j].x, s0));
          st_shared16(d ^ 16, widen8(cw[j].y, s0));
          st_shared16(d ^ 32, widen8(cw[j].z, s1));
          st_shared16(d ^ 48, widen8(cw[j].w, s1));
        }
        if (kScores) st_shared16(ring + g * kStageBytes + 8 * kRegion + o_rope, rp);
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) arrive_leader<G>(&sm.kv_full[g], kLeader);
      }
      place = (place + kLead + it.n) & 1;
    }
  }
  return;
  // a wait has given up: the hardware barriers of this tile's queries, unless they are through, and of the tiles to come
leave_queries:
  __syncwarp();
  if (kScores) {
    some_sync(kQueryBar + ((w & 3) >> 1), 256);
    some_sync(kQueryBar + ((w & 3) >> 1), 256);
  }
leave:
  __syncwarp();
  while (kScores && walk.next(it)) {
    some_sync(kQueryBar + ((w & 3) >> 1), 256);
    some_sync(kQueryBar + ((w & 3) >> 1), 256);
  }
}

// ---------------------------------------------------------------------------
// Scores CTA
// ---------------------------------------------------------------------------
// Copies a tile's queries by TMA into the ring, as two places of 64 rows from place m
// on, once the widening warps, which follow the ring place by place, have found them free.
template <int G>
__device__ inline bool copy_queries(const DenseArgs& a, DenseSmall& sm, uint8_t* base, const Item& it, int part, uint32_t m,
                                    uint32_t k_item, bool one, const CUtensorMap* qmap) {
  const int y = it.a.z * a.d.heads + it.a.y + kDenseTile * part;
#pragma unroll 1
  for (int k = 0; k < 2; ++k, ++m) {
    const uint32_t st = m % kKStages;
    if (!wait_warp(sm, &sm.q_turn[st], k_item & 1, a.ws)) return false;
    if (one) {
      tc::mbar_expect_tx(&sm.q_place[st], kKBytes);
#pragma unroll 1
      for (int kb = 0; kb < 9; ++kb)
        tc::tma_load_2d(qmap, base + Lay<G>::kKvOff + st * kKBytes + kb * kReg, 64 * kb, y + 64 * k, &sm.q_place[st]);
    }
    __syncwarp();
  }
  return true;
}

// Asks L2 for the rows of the next tile's queries (one piece of memory).
__device__ inline void prefetch_queries(const DenseArgs& a, Walk walk, int part) {
  Item it = {};
  if (!walk.next(it)) return;
  const int64_t row = int64_t(it.a.z) * a.d.heads + it.a.y + kDenseTile * part;
  const int rows = min(kDenseTile, it.a.w * a.d.heads - it.a.y - kDenseTile * part);
  if (rows > 0)
    asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;" ::"l"(a.q + row * kDqk), "r"(rows * kDqk * 2) : "memory");
}

// The copying and issuing warp; in the second CTA of a pair it only copies.
template <int G>
__device__ inline void scores_mma_role(const DenseArgs& a, DenseSmall& sm, uint8_t* base, int cl, int part, uint32_t tmem,
                                       const CUtensorMap* qmap) {
  // latents are fp16, rope keys bf16 (each with queries of its type; one accumulator)
  constexpr uint32_t id_lat = idesc_f16(kDenseTile * G, kDenseBlk, 0, 0);
  constexpr uint32_t id_rope = tc::idesc_bf16(kDenseTile * G, kDenseBlk, 0, 0);
  constexpr int kRegion = kReg / G;                  // 64 channels of the 64 / G positions of a CTA
  constexpr uint16_t kBoth = 0x3;
  Walk walk(a.plan, cl);
  Item it = {};
  uint32_t n = 0;
  const bool leader = elect_one();
  for (uint32_t k = 0; walk.next(it); ++k) {
    if (!copy_queries<G>(a, sm, base, it, part, n, k, leader, qmap)) return;      // two places a tile: place and block number have one parity
    if (leader) prefetch_queries(a, walk, part);
    if (part != 0) {
      n += it.n;
      continue;
    }
    if (!wait_warp(sm, &sm.q_full, k & 1, a.ws)) return;
    for (int j = 0; j < it.n; ++j, ++n) {
      const uint32_t st = n % kKStages, buf = n % kSBufs;
      if (!wait_warp(sm, &sm.kv_full[st], (n / kKStages) & 1, a.ws)) return;
      if (!wait_warp(sm, &sm.s_empty[buf], ((n / kSBufs) & 1) ^ 1, a.ws)) return;
      tc::tc_fence_after_sync();
      if (leader) {
        const uint64_t bd = tc::smem_desc(tc::smem_u32(base + Lay<G>::kKvOff + st * kKBytes), 16, 1024, 2);
        const uint32_t d = tmem + kSCol + buf * kDenseBlk;
#pragma unroll 1
        for (int kb = 0; kb < 9; ++kb)
#pragma unroll
          for (int k4 = 0; k4 < 4; ++k4)
            mma_ts<G>(d, tmem + kb * 32 + k4 * 8, bd + ((kb * kRegion + k4 * 32) >> 4), kb < 8 ? id_lat : id_rope, kb + k4 > 0);
        commit_to<G>(&sm.kv_empty[st], kBoth);
        commit_to<G>(&sm.s_full[buf], kBoth);
      }
      __syncwarp();
    }
  }
}

// Warp rw: rows 32 (rw % 4) .. + 31 (one a lane) of every block n with n % 2 = rw / 4: the
// two warps of a row take turns, each with two block periods for the latencies of a
// block.  What must go in order is the reference: block n's warp takes it from block
// n - 1's as soon as that one has its maximum, and hands it on.
template <int G>
__device__ inline void softmax_role(const DenseArgs& a, DenseSmall& sm, uint8_t* base, int cl, int part, int rw, int lane,
                                    uint32_t tmem) {
  const int wq = rw & 3, half = rw >> 2;
  const uint32_t lanes = tmem + (uint32_t(wq * 32) << 16);
  const int r = wq * 32 + lane;
  const float c2 = a.scale * 1.4426950408889634f;
  uint32_t n = 0;
  uint32_t zeroed = 0;                               // slots in which this warp's rows of P are zeros
  uint32_t n0 = 0, n1 = 0;                           // blocks of the item
  bool live = false;                                 // some row of this warp (and of its other half) exists
  Cursor cur(a.plan, cl, lane);
  for (uint32_t k_item = 0; cur.item(a); ++k_item) {
    some_sync(kTurnBar + wq, 64);                    // both warps of a row are through the tile before
    float c = 0.0f;                                  // logits in base 2 per score; known with the first scores
    // positions this row sees: first .. last
    const int lr = cur.it.a.y + kDenseTile * part + r, tok = lr / a.d.heads;
    live = __any_sync(0xFFFFFFFFu, tok < cur.it.a.w);
    int last = -1, first = 0;
    if (tok < cur.it.a.w) {
      last = a.causal ? cur.it.b.x - cur.it.a.w + tok : cur.it.b.x - 1;
      if (a.window > 0) first = max(0, last - a.window + 1);
    }
    bool own_first = true;
    float own = -INFINITY, sum = 0.0f;               // reference of this warp's last block, its sum under it
    n0 = n;
    n1 = n + cur.it.n;
    cur.i = int((half ^ n0) & 1);
    n += uint32_t(cur.i);
#pragma unroll 1
    for (; n < n1; n += 2) {
      const uint32_t buf = n % kSBufs, slot = n % Lay<G>::kPSlots;
      const int t0 = (cur.it.blk + cur.i) * kDenseBlk;
      const int lo = first - t0, hi = cur.row0(a) < 0 ? -1 : last - t0;
      const bool edge = __any_sync(0xFFFFFFFFu, lo > 0 || hi < kDenseBlk - 1);
      uint8_t* ps = base + slot * kPBytes;
      if (!wait_warp(sm, &sm.s_full[buf], (n / kSBufs) & 1, a.ws)) goto leave;
      if (!live) {
        // no row at all (a decode tile of few heads): P stays zero
        if (!wait_warp(sm, &sm.p_free[slot], ((n / Lay<G>::kPSlots) & 1) ^ 1, a.ws)) goto leave;
        // Zeros once sent stand in the values CTA's slot as well: the bytes are only counted from
        // then on.  (What a later tile leaves there meets only rows that do not exist.)
        const bool sent = zeroed >> slot & 1;
        if (!sent) {
#pragma unroll
          for (int i = 0; i < 8; ++i) *reinterpret_cast<uint4*>(ps + wq * 4096 + i * 512 + lane * 16) = make_uint4(0, 0, 0, 0);
          sm.meta[slot][wq][0][lane] = 1.0f;
          sm.meta[slot][wq][1][lane] = 0.0f;
          sm.meta[slot][wq][2][lane] = 0.0f;
          tc::fence_proxy_async_smem();
          zeroed |= 1u << slot;
        }
        __syncwarp();
        if (lane == 0) {
          arrive_leader<G>(&sm.s_empty[buf], 0);
          const uint32_t bar = peer_addr(&sm.p_full[slot], uint32_t(G + part));
          if (sent) {
            asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cluster.b64 [%0], %1;" ::"r"(bar), "r"(4096 + kMetaWarp) : "memory");
          } else {
            copy_to_peer(peer_addr(ps + wq * 4096, uint32_t(G + part)), ps + wq * 4096, 4096, bar);
            copy_to_peer(peer_addr(&sm.meta[slot][wq][0][0], uint32_t(G + part)), &sm.meta[slot][wq][0][0], kMetaWarp, bar);
          }
        }
        __syncwarp();
        cur.step(a, 2);
        continue;
      }
      zeroed &= ~(1u << slot);
      tc::tc_fence_after_sync();
      if (own_first) {
        // the scores' queries were scaled by 2^k (of four tiles in turn: there are never scores of more than three unread)
        c = fmaxf(fabsf(c2) * __uint_as_float(uint32_t(127 - sm.q_shift[k_item & 3][r]) << 23), 1.17549435e-38f);
        own_first = false;
      }
      float x[64];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        float y[32];
        tc::tmem_ld32(lanes + kSCol + buf * kDenseBlk + 32 * h, y);
#pragma unroll
        for (int i = 0; i < 32; ++i) x[32 * h + i] = y[i];
      }
      tc::tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) arrive_leader<G>(&sm.s_empty[buf], 0);
      if (edge) {
#pragma unroll
        for (int i = 0; i < 64; ++i) x[i] = (i >= lo && i <= hi) ? x[i] : -INFINITY;
      }
      float t4[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
      for (int i = 4; i < 64; i += 8) {
#pragma unroll
        for (int k = 0; k < 4; ++k) t4[k] = i + 4 + k < 64 ? fmaxf(fmaxf(t4[k], x[i + k]), x[i + 4 + k]) : fmaxf(t4[k], x[i + k]);
      }
      const float top = fmaxf(fmaxf(t4[0], t4[1]), fmaxf(t4[2], t4[3])) * c;
      // the reference so far, from the other warp (each arrival is awaited before the next on
      // the same barrier)
      float before = -INFINITY;
      if (n != n0) {
        some_sync(kRefBar + 4 * (half ^ 1) + wq, 64);
        before = sm.ref[half ^ 1][r];
      }
      float ref = before, alpha = 1.0f;
      if (top > ref + 8.0f) {
        ref = ceilf(top);
        if (before != -INFINITY) alpha = ex2(before - ref);
      }
      if (n + 1 != n1) {
        sm.ref[half][r] = ref;
        some_arrive(kRefBar + 4 * half + wq, 64);
      }
      if (own != ref && own != -INFINITY) sum *= ex2(own - ref);     // (no reference yet: 0, or NaN)
      own = ref;
      const float sub = ref == -INFINITY ? 0.0f : ref - 7.0f;
      if (!wait_warp(sm, &sm.p_free[slot], ((n / Lay<G>::kPSlots) & 1) ^ 1, a.ws)) {
        n += 2;                                      // this block's hand-offs are done
        goto leave;
      }
      const uint64_t cc = pack2(c, c), ss = pack2(-sub, -sub);
      uint64_t acc[2] = {0, 0};                      // +0, +0
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        uint32_t pk[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          float p0, p1;
          unpack2(fma2(pack2(x[8 * i + 2 * k], x[8 * i + 2 * k + 1]), cc, ss), p0, p1);
          p0 = ex2(p0);
          p1 = ex2(p1);
          acc[k & 1] = add2(acc[k & 1], pack2(p0, p1));
          pk[k] = f16x2_rn(p0, p1);
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
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        const uint32_t bar = peer_addr(&sm.p_full[slot], uint32_t(G + part));
        copy_to_peer(peer_addr(ps + wq * 4096, uint32_t(G + part)), ps + wq * 4096, 4096, bar);
        copy_to_peer(peer_addr(&sm.meta[slot][wq][0][0], uint32_t(G + part)), &sm.meta[slot][wq][0][0], kMetaWarp, bar);
      }
      __syncwarp();
      cur.step(a, 2);
    }
    n = n1;
  }
  return;
  // a wait has given up: the hand-offs of the tile's blocks from n on, and of the tiles to come
leave:
  __syncwarp();
  for (;;) {
    for (; live && n < n1; n += 2) {
      if (n != n0) some_sync(kRefBar + 4 * (half ^ 1) + wq, 64);
      if (n + 1 != n1) some_arrive(kRefBar + 4 * half + wq, 64);
    }
    if (!cur.walk.next(cur.it)) return;
    some_sync(kTurnBar + wq, 64);
    live = __any_sync(0xFFFFFFFFu, (cur.it.a.y + kDenseTile * part + r) / a.d.heads < cur.it.a.w);
    n0 = n1;
    n1 += cur.it.n;
    n = n0 + ((half ^ n0) & 1);
  }
}

// ---------------------------------------------------------------------------
// Values CTA
// ---------------------------------------------------------------------------
// Hands each slot of P back once its products are done.
template <int G>
__device__ inline void slot_role(const DenseArgs& a, DenseSmall& sm, int cl, int part, int lane) {
  const int all = Walk(a.plan, cl).left;
  for (int n = 0; n + Lay<G>::kPSlots < all; ++n) {
    const uint32_t slot = uint32_t(n) % Lay<G>::kPSlots;
    if (!wait_warp(sm, &sm.pv_done[slot], (uint32_t(n) / Lay<G>::kPSlots) & 1, a.ws)) return;
    if (lane == 0) {
      tc::mbar_expect_tx(&sm.p_full[slot], kPBytes + 4 * kMetaWarp);
      arrive_remote(peer_addr(&sm.p_free[slot], uint32_t(part)));
    }
    __syncwarp();
  }
}

template <int G>
__device__ inline void values_mma_role(const DenseArgs& a, DenseSmall& sm, uint8_t* base, int cl, uint32_t tmem) {
  constexpr uint32_t id = idesc_f16(kDenseTile * G, 256, 0, 1);
  constexpr uint16_t kBoth = 0xC;
  Walk walk(a.plan, cl);
  Item it = {};
  uint32_t n = 0;
  const bool leader = elect_one();
  for (uint32_t k = 0; walk.next(it); ++k) {
    if (!wait_warp(sm, &sm.o_free, (k & 1) ^ 1, a.ws)) return;
    for (int j = 0; j < it.n; ++j, ++n) {
      const uint32_t st = n % kKStages, slot = n % Lay<G>::kPSlots, ph = (n / Lay<G>::kPSlots) & 1;
      if (!wait_warp(sm, &sm.kv_full[st], (n / kKStages) & 1, a.ws)) return;
      if (G == 1 && !wait_warp(sm, &sm.p_full[slot], ph, a.ws)) return;
      if (!wait_warp(sm, &sm.corr[slot], ph, a.ws)) return;       // of a pair: both have seen their P arrive
      tc::tc_fence_after_sync();
      if (leader) {
        const uint64_t ad = tc::smem_desc(tc::smem_u32(base + slot * kPBytes), 16, 1024, 2);
        const uint64_t bd = tc::smem_desc(tc::smem_u32(base + Lay<G>::kKvOff + st * kVBytes), kReg, 1024, 2);
#pragma unroll
        for (int ks = 0; ks < kDenseBlk / 16; ++ks)
#pragma unroll
          for (int h = 0; h < 2; ++h)
            mma_ss<G>(tmem + h * 256, ad + ((ks * 32) >> 4), bd + ((h * (4 / G) * kReg + ks * 2048) >> 4), id,
                      j > 0 || ks > 0);
        commit_to<G>(&sm.kv_empty[st], kBoth);
        commit_to<G>(&sm.pv_done[slot], kBoth);
      }
      __syncwarp();
    }
  }
}

// Warp rw: rows 32 (rw % 4) .. + 31 (one a lane), channels 256 (rw / 4) .. + 255.
template <int G>
__device__ inline void output_role(const DenseArgs& a, DenseSmall& sm, uint8_t* base, int cl, int part, int rw, int lane,
                                   uint32_t tmem) {
  const int wq = rw & 3, col0 = 256 * (rw >> 2);
  const uint32_t lanes = tmem + (uint32_t(wq * 32) << 16) + uint32_t(col0);
  const int r = wq * 32 + lane;
  constexpr int kCols = 32 * G;                      // columns staged at a time: 64 or 128 bytes of 32 rows
  uint8_t* stage = base + Lay<G>::kStageOff + rw * (2048 * G);
  // channel of output column col0 + c: in order at G 1; at G 2 a product's 256 columns are 128 channels from each CTA's half
  const auto channel = [&](int c) { return G == 1 ? col0 + c : (col0 >> 1) + (c & 127) + ((c & 128) << 1); };
  Walk walk(a.plan, cl);
  Item it = {};
  uint32_t n = 0;
  while (walk.next(it)) {
    // sums of the even and the odd blocks, each under the reference of its last block
    float sum = 0.0f, sub = 0.0f, sum_b = 0.0f, sub_b = 0.0f;
    for (int j = 0; j < it.n; ++j, ++n) {
      const uint32_t slot = n % Lay<G>::kPSlots;
      if (!wait_warp<true>(sm, &sm.p_full[slot], (n / Lay<G>::kPSlots) & 1, a.ws)) return;
      const float alpha = sm.meta[slot][wq][0][lane];
      sum_b = sum;
      sub_b = sub;
      sum = sm.meta[slot][wq][1][lane];
      sub = sm.meta[slot][wq][2][lane];
      if (__any_sync(0xFFFFFFFFu, alpha != 1.0f)) {
        // the outputs so far, once their products are done, to the new reference
        const uint32_t m = n - 1;
        if (!wait_warp(sm, &sm.pv_done[m % Lay<G>::kPSlots], (m / Lay<G>::kPSlots) & 1, a.ws)) return;
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
      if (lane == 0) arrive_leader<G>(&sm.corr[slot], G);
    }
    const uint32_t m = n - 1;
    if (!wait_warp(sm, &sm.pv_done[m % Lay<G>::kPSlots], (m / Lay<G>::kPSlots) & 1, a.ws)) return;
    tc::tc_fence_after_sync();
    if (sum_b != 0.0f) sum += sum_b * ex2(sub_b - sub);
    const float inv = sum != 0.0f ? 1.0f / sum : 0.0f;                 // NaN stays NaN
    const float lse = sum != 0.0f ? (sub + log2f(sum)) * 0.6931471805599453f : -INFINITY;
    const int lr = it.a.y + kDenseTile * part + r, rows = it.a.w * a.d.heads;
    if (it.head || it.tail) {
      const int slot = (2 * cl + (it.head ? 0 : 1)) * G + part;
      float* po = a.part_o + int64_t(slot) * kLatent * kDenseTile + r;
      if (col0 == 0) a.part_lse[slot * kDenseTile + r] = lse;
#pragma unroll 1
      for (int col = 0; col < 256; col += 32) {
        float v[32];
        tc::tmem_ld32(lanes + col, v);
#pragma unroll
        for (int i = 0; i < 32; ++i) po[(channel(col) + i) * kDenseTile] = v[i] * inv;
      }
    } else {
      const int64_t g0 = int64_t(it.a.z) * a.d.heads + lr - lane;           // the warp's first row
      const int have = rows - (lr - lane);                                  // rows from it on that exist
      if (col0 == 0 && lr < rows) a.lse[g0 + lane] = lse;
      constexpr int kChunks = kCols / 8;             // 16-byte chunks of a row
      const auto chunk_at = [&](int row, int ch) {   // 64- or 128-byte swizzle
        return G == 1 ? row * 64 + ((ch ^ ((row >> 1) & 3)) << 4) : row * 128 + ((ch ^ (row & 7)) << 4);
      };
      uint16_t* dst = a.out + g0 * kLatent + 8 * (lane % kChunks);
#pragma unroll 1
      for (int col = 0; col < 256; col += kCols) {
#pragma unroll
        for (int h = 0; h < G; ++h) {
          float v[32];
          tc::tmem_ld32(lanes + col + 32 * h, v);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4*>(stage + chunk_at(lane, 4 * h + i)) =
                make_uint4(bf16x2_rn(v[8 * i] * inv, v[8 * i + 1] * inv), bf16x2_rn(v[8 * i + 2] * inv, v[8 * i + 3] * inv),
                           bf16x2_rn(v[8 * i + 4] * inv, v[8 * i + 5] * inv),
                           bf16x2_rn(v[8 * i + 6] * inv, v[8 * i + 7] * inv));
        }
        __syncwarp();
        // whole rows of 64 or 128 bytes an instruction
#pragma unroll
        for (int i = 0; i < kChunks; ++i) {
          const int row = (32 / kChunks) * i + lane / kChunks;
          if (row < have)
            *reinterpret_cast<uint4*>(dst + int64_t(row) * kLatent + channel(col)) =
                *reinterpret_cast<const uint4*>(stage + chunk_at(row, lane % kChunks));
        }
        __syncwarp();
      }
    }
    tc::tc_fence_before_sync();
    __syncwarp();
    if (lane == 0) arrive_leader<G>(&sm.o_free, G);
  }
}

template <int G>
__device__ inline void dense_body(const DenseArgs& a, const CUtensorMap* qmap, const CUtensorMap* codes,
                                  const CUtensorMap* rope) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* base = smem_raw;                          // 1024-byte aligned: checked below
  __shared__ DenseSmall sm;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int rank = blockIdx.x % (2 * G), cl = blockIdx.x / (2 * G), part = rank % G;
  const bool scores = rank < G;
  if (tc::smem_u32(base) & 1023u) {                  // never, as laid out; the same in every CTA
    pdl_wait();
    if (tid == 0) raise_err(a.ws, CSA2_DEV_TIMEOUT);
    return;
  }
  if (wid == 0) tmem_alloc_all<G>(&sm.tmem_slot);
  if (tid == 0) {
    for (int i = 0; i < Lay<G>::kRawStages; ++i) {
      tc::mbar_init(&sm.raw_full[i], 1);
      tc::mbar_init(&sm.raw_empty[i], kConvWarps / G);
    }
    for (int i = 0; i < kKStages; ++i) {
      // G 1: all widening warps, and the rope keys' thread; G 2: 8 in each CTA of the pair
      tc::mbar_init(&sm.kv_full[i], kConvWarps);
      tc::mbar_init(&sm.kv_empty[i], 1);
      tc::mbar_init(&sm.q_turn[i], kConvWarps / G);
      tc::mbar_init(&sm.q_place[i], 1);
    }
    for (int i = 0; i < kSBufs; ++i) {
      tc::mbar_init(&sm.s_full[i], 1);
      tc::mbar_init(&sm.s_empty[i], 4 * G);
    }
    tc::mbar_init(&sm.q_full, kConvWarps * G);
    for (int i = 0; i < Lay<G>::kPSlots; ++i) {
      tc::mbar_init(&sm.p_free[i], 1);
      tc::mbar_init(&sm.p_full[i], 1);
      tc::mbar_init(&sm.corr[i], kRowWarps * G);
      tc::mbar_init(&sm.pv_done[i], 1);
    }
    tc::mbar_init(&sm.o_free, kRowWarps * G);
    tc::mbar_init(&sm.drain, 1);
    sm.abort = 0;
    tc::fence_mbar_init();
    if (!scores)
      for (int i = 0; i < Lay<G>::kPSlots; ++i) tc::mbar_expect_tx(&sm.p_full[i], kPBytes + 4 * kMetaWarp);
  }
  tc::tc_fence_before_sync();
  __syncthreads();
  tc::tc_fence_after_sync();
  // every CTA's barriers stand before another writes into it
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  const uint32_t tmem = sm.tmem_slot;
  pdl_wait();
  pdl_launch_dependents();
  if (scores) {
    if (wid < kRowWarps) {
      regs_up<kRowRegs>();
      softmax_role<G>(a, sm, base, cl, part, wid, lane, tmem);
    } else if (wid < kMmaWarp) {
      regs_down<kConvRegs>();
      widen_role<G, true>(a, sm, base, cl, part, wid - kConvWarp0, lane, tmem);
    } else {
      regs_down<kMmaRegs>();
      if (wid == kMmaWarp) scores_mma_role<G>(a, sm, base, cl, part, tmem, qmap);
      else if (wid == kMmaWarp + 1) raw_role<G, true>(a, sm, base, cl, part, lane, codes, rope);
    }
  } else {
    if (wid < kRowWarps) {
      regs_up<kRowRegs>();
      output_role<G>(a, sm, base, cl, part, wid, lane, tmem);
    } else if (wid < kMmaWarp) {
      regs_down<kConvRegs>();
      widen_role<G, false>(a, sm, base, cl, part, wid - kConvWarp0, lane, tmem);
    } else {
      regs_down<kMmaRegs>();
      if (wid == kMmaWarp && part == 0) values_mma_role<G>(a, sm, base, cl, tmem);
      else if (wid == kMmaWarp + 2) slot_role<G>(a, sm, cl, part, lane);
      else if (wid == kMmaWarp + 1) raw_role<G, false>(a, sm, base, cl, part, lane, codes, rope);
    }
  }
  // the thread that issued the MMAs sees them done (they are, unless a wait gave up)
  __syncwarp();
  if (wid == kMmaWarp && part == 0) {
    if (elect_one()) {
      commit_to<G>(&sm.drain, uint16_t(1u << rank));
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
  if (wid == 0) tmem_free_all<G>(tmem);
}

struct DenseMaps {
  CUtensorMap q, codes, rope;
};

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kDenseThreads, 1)
    dense_kernel(const __grid_constant__ DenseArgs a, const __grid_constant__ DenseMaps m) {
  dense_body<1>(a, &m.q, &m.codes, &m.rope);
}

__global__ void __cluster_dims__(4, 1, 1) __launch_bounds__(kDenseThreads, 1)
    dense_pair_kernel(const __grid_constant__ DenseArgs a, const __grid_constant__ DenseMaps m) {
  dense_body<2>(a, &m.q, &m.codes, &m.rope);
}

// ---------------------------------------------------------------------------
// Plan: one CTA.  Sequences -> tiles of 128 rows -> blocks each tile sees ->
// equal runs of blocks, one per cluster.
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;

// Exclusive sum over the block; buf: one value a warp.
__device__ inline int64_t block_scan_sum(int64_t v, int64_t* buf, int64_t& total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int64_t x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x += y;
  }
  __syncthreads();
  if (lane == 31) buf[w] = x;
  __syncthreads();
  const int64_t mine = lane < int(blockDim.x >> 5) ? buf[lane] : 0;
  int64_t z = mine;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int64_t y = __shfl_up_sync(0xFFFFFFFFu, z, o);
    if (lane >= o) z += y;
  }
  total = __shfl_sync(0xFFFFFFFFu, z, 31);
  return __shfl_sync(0xFFFFFFFFu, z - mine, w) + x - v;
}

// Inclusive maximum over the block.
__device__ inline int block_scan_max(int v, int64_t* buf, int& total) {
  const int lane = threadIdx.x & 31, w = threadIdx.x >> 5;
  int x = v;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
    if (lane >= o) x = max(x, y);
  }
  __syncthreads();
  if (lane == 31) buf[w] = x;
  __syncthreads();
  const int warps = int(blockDim.x >> 5);
  int before = INT32_MIN, all = INT32_MIN;
  for (int i = 0; i < warps; ++i) {
    if (i < w) before = max(before, int(buf[i]));
    all = max(all, int(buf[i]));
  }
  total = all;
  return max(before, x);
}

// The last of n (at least 1) ascending values that is at most x.
template <typename F>
__device__ inline int last_at_most(int n, int64_t x, F value) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (value(mid) <= x) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

// Tile t of a sequence: its two records, and how many blocks it sees.
__device__ inline int make_tile(const DenseArgs& a, int t, int seq, int4 s, int4* out) {
  const int H = a.d.heads, row0 = (t - s.x) * a.tile;
  const int tok0 = row0 / H, tok1 = min(s.z - 1, (row0 + a.tile - 1) / H);
  int first = 0, last = s.w - 1, nb = 0, fb = 0;
  if (a.causal) {
    last = s.w - s.z + tok1;
    if (a.window > 0) first = max(0, s.w - s.z + tok0 - a.window + 1);
  }
  if (last >= first) {
    fb = first / kDenseBlk;
    nb = last / kDenseBlk - fb + 1;
  }
  out[2 * t] = make_int4(seq, row0, s.y, s.z);
  out[2 * t + 1] = make_int4(s.w, fb, nb, 0);
  return nb;
}

__device__ inline int active_runs(const DenseArgs& a, int64_t blocks) {
  const int64_t want = (blocks + kDenseMinBlocks - 1) / kDenseMinBlocks;
  return blocks > 0 ? int(min64(a.clusters, want)) : 0;
}

// Run c: first tile, blocks of it before the run, blocks.
template <typename F>
__device__ inline int4 make_run(int c, int active, int64_t blocks, int ntiles, F before) {
  if (c >= active) return make_int4(0, 0, 0, 0);
  const int64_t w0 = blocks * c / active, w1 = blocks * (c + 1) / active;
  const int t = last_at_most(ntiles, w0, before);
  return make_int4(t, int(w0 - before(t)), int(w1 - w0), 0);
}

__global__ void __launch_bounds__(kPlanThreads, 1) dense_plan_kernel(DenseArgs a) {
  __shared__ int64_t buf[32];
  __shared__ int4 s_seq[kPlanThreads];
  __shared__ int s_before[kPlanThreads];
  const int tid = threadIdx.x, H = a.d.heads, threads = int(blockDim.x);
  const bool paged = a.page_table != nullptr;
  pdl_wait();
  pdl_launch_dependents();
  // One sequence and one tile a thread, all in shared memory, where that is enough and
  // the starts are in order.
  if (a.batch <= threads && a.max_tiles <= threads) {
    const bool in = tid < a.batch;
    const int from = in ? __ldg(a.q_start + tid) : 0, end = in ? __ldg(a.q_start + tid + 1) : 0;
    const int len = end - from;
    const int64_t raw_ctx = in ? __ldg(a.ctx_len + tid) : 0;
    if (__syncthreads_and(from >= 0 && end >= from && end <= a.total_q)) {
      const int ctx = in ? int(check_ctx(raw_ctx, a.d, paged, a.ws)) : 0;
      int64_t all, blocks;
      const int64_t at = block_scan_sum((int64_t(len) * H + a.tile - 1) / a.tile, buf, all);
      if (in) s_seq[tid] = make_int4(int(at), from, len, ctx);
      __syncthreads();
      const int ntiles = int(all);
      int nb = 0;
      if (tid < ntiles) {
        const int b = last_at_most(a.batch, tid, [&](int i) { return int64_t(s_seq[i].x); });
        nb = make_tile(a, tid, b, s_seq[b], a.plan.tiles);
      }
      const int64_t before = block_scan_sum(nb, buf, blocks);
      s_before[tid] = int(before);                   // at most 1,024 tiles of 16,384 blocks
      __syncthreads();
      const int active = active_runs(a, blocks);
      if (tid == 0) *a.plan.head = make_int4(ntiles, active, int(blocks), int(blocks >> 32));
      if (tid < ntiles) a.plan.before[tid] = before;
      for (int c = tid; c < a.clusters; c += threads)
        a.plan.runs[c] = make_run(c, active, blocks, ntiles, [&](int i) { return int64_t(s_before[i]); });
      return;
    }
  }
  // Any number of them.  A q_start that falls back or leaves [0, total_q] is reported and
  // replaced by the nearest value that keeps the order.
  const int s0 = __ldg(a.q_start);
  int reach = min(max(s0, 0), a.total_q);
  if (tid == 0 && reach != s0) raise_err(a.ws, CSA2_DEV_Q_START);
  int ntiles = 0;
  __shared__ int edge[kPlanThreads / 32];
  for (int base = 0; base < a.batch; base += threads) {
    const int b = base + tid;
    int end = INT32_MIN, raw = 0;
    if (b < a.batch) {
      raw = __ldg(a.q_start + b + 1);
      end = min(max(raw, 0), a.total_q);
    }
    int top;
    const int upto = max(reach, block_scan_max(end, buf, top));
    if (b < a.batch && upto != raw) raise_err(a.ws, CSA2_DEV_Q_START);
    // this sequence's first query: the reach before it
    int from = __shfl_up_sync(0xFFFFFFFFu, upto, 1);
    __syncthreads();
    if ((tid & 31) == 31) edge[tid >> 5] = upto;
    __syncthreads();
    if ((tid & 31) == 0) from = tid == 0 ? reach : edge[(tid >> 5) - 1];
    const int len = b < a.batch ? upto - from : 0;
    int64_t all;
    const int64_t at = block_scan_sum((int64_t(len) * H + a.tile - 1) / a.tile, buf, all);
    if (b < a.batch)
      a.plan.seqs[b] = make_int4(ntiles + int(at), from, len, int(checked_ctx(a.ctx_len, a.d, b, paged, a.ws)));
    ntiles += int(all);
    reach = max(reach, top);
  }
  __syncthreads();
  int64_t blocks = 0;
  for (int base = 0; base < ntiles; base += threads) {
    const int t = base + tid;
    int nb = 0;
    if (t < ntiles) {
      const int b = last_at_most(a.batch, t, [&](int i) { return int64_t(a.plan.seqs[i].x); });
      nb = make_tile(a, t, b, a.plan.seqs[b], a.plan.tiles);
    }
    int64_t all;
    const int64_t at = block_scan_sum(nb, buf, all);
    if (t < ntiles) a.plan.before[t] = blocks + at;
    blocks += all;
  }
  __syncthreads();
  const int active = active_runs(a, blocks);
  if (tid == 0) *a.plan.head = make_int4(ntiles, active, int(blocks), int(blocks >> 32));
  for (int c = tid; c < a.clusters; c += threads)
    a.plan.runs[c] = make_run(c, active, blocks, ntiles, [&](int i) { return a.plan.before[i]; });
}

// ---------------------------------------------------------------------------
// Merge: a CTA joins 8 channels of a tile that was cut between runs.  Thread = row.  It
// also writes the rows of tiles that see nothing.  Bound by the latency of its loads, so
// as many as may be are in flight (48 a thread; 16.3 us with 16 on the 128K decode batch,
// where a tile has about ten pieces; 14.2).
//   kFew, where there are few tiles, of many pieces each: CTA (g, t) is for tile t, and a
//     row has four threads, which take a quarter of the pieces each;
//   else CTA (g, c) is for the tile that the boundary before run c cuts, if c is the first
//     boundary inside it.
// ---------------------------------------------------------------------------
constexpr int kMergeCh = 8;
constexpr int kMergeFew = 4;                        // threads a row where there are few tiles

template <bool kFew>
__global__ void __launch_bounds__(kDenseTile * (kFew ? kMergeFew : 1)) dense_merge_kernel(DenseArgs a) {
  constexpr int Y = kFew ? kMergeFew : 1;
  __shared__ float s_top[kFew ? Y : 1][kDenseTile], s_total[kFew ? Y : 1][kDenseTile];
  __shared__ float s_o[kFew ? Y : 1][kFew ? kMergeCh : 1][kDenseTile];
  pdl_wait();
  pdl_launch_dependents();
  const int r = threadIdx.x, y = kFew ? threadIdx.y : 0, g = blockIdx.x;
  const int G = a.tile / kDenseTile, part = blockIdx.z;
  const int ctas = gridDim.x * gridDim.y * gridDim.z;
  const int t0 = (blockIdx.z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x;
  // the tile and its pieces: runs first .. first + n - 1 (see make_run); n 0: none, or one
  const int4 head = __ldg(a.plan.head);
  const int64_t blocks = int64_t(uint32_t(head.z)) | int64_t(head.w) << 32;
  const auto run_of = [&](int64_t block) { return int(((block + 1) * head.y - 1) / blocks); };
  int4 ta = {};
  int first = 0, n = 0;
  if constexpr (kFew) {
    const int t = blockIdx.y;
    ta = __ldg(a.plan.tiles + 2 * t);
    const int4 tb = __ldg(a.plan.tiles + 2 * t + 1);
    const int64_t b0 = __ldg(a.plan.before + t);
    if (t < head.x && tb.z > 0) {
      first = run_of(b0);
      n = run_of(b0 + tb.z - 1) - first + 1;
    }
  } else {
    // independent loads first: each level of dependent ones is most of a microsecond
    const int c = blockIdx.y;
    const int4 run = __ldg(a.plan.runs + c), prev = __ldg(a.plan.runs + max(c - 1, 0));
    // a boundary inside a tile, the first there: the run before starts at or before the tile's first block
    if (c < head.y && run.y > 0 && (prev.x != run.x || prev.y == 0)) {
      ta = __ldg(a.plan.tiles + 2 * run.x);
      const int4 tb = __ldg(a.plan.tiles + 2 * run.x + 1);
      first = c - 1;
      n = run_of(__ldg(a.plan.before + run.x) + tb.z - 1) - first + 1;
    }
  }
  if (n > 1) {
    const int lr = ta.y + kDenseTile * part + r;
    const bool in = lr < ta.w * a.d.heads;
    const int mine = in ? n : 0;
    // the first piece ends its run (its tail); the others start theirs
    const auto slot = [&](int i) { return (i == 0 ? 2 * first + 1 : 2 * (first + i)) * G + part; };
    float top = -INFINITY;
#pragma unroll 4
    for (int i = y; i < mine; i += Y) top = fmaxf(top, __ldg(a.part_lse + slot(i) * kDenseTile + r));
    if (kFew) {
      s_top[y][r] = top;
      __syncthreads();
#pragma unroll
      for (int j = 0; j < Y; ++j) top = fmaxf(top, s_top[j][r]);
    }
    float o[kMergeCh], total = 0.0f;
#pragma unroll
    for (int k = 0; k < kMergeCh; ++k) o[k] = 0.0f;
#pragma unroll 6
    for (int i = y; i < mine; i += Y) {
      const int s = slot(i);
      const float l = __ldg(a.part_lse + s * kDenseTile + r);
      const float w = l == -INFINITY ? 0.0f : exp2f((l - top) * 1.4426950408889634f);
      total += w;
      const float* po = a.part_o + (int64_t(s) * kLatent + g * kMergeCh) * kDenseTile + r;
#pragma unroll
      for (int k = 0; k < kMergeCh; ++k) o[k] = fmaf(w, __ldg(po + k * kDenseTile), o[k]);
    }
    if (kFew) {
      s_total[y][r] = total;
#pragma unroll
      for (int k = 0; k < kMergeCh; ++k) s_o[y][kFew ? k : 0][r] = o[k];
      __syncthreads();
      if (y == 0) {
#pragma unroll
        for (int j = 1; j < Y; ++j) {
          total += s_total[j][r];
#pragma unroll
          for (int k = 0; k < kMergeCh; ++k) o[k] += s_o[j][kFew ? k : 0][r];
        }
      }
    }
    if (in && y == 0) {
      const float inv = total != 0.0f ? 1.0f / total : 0.0f;
      const int64_t row = int64_t(ta.z) * a.d.heads + lr;
      uint4* dst = reinterpret_cast<uint4*>(a.out + row * kLatent + g * kMergeCh);
#pragma unroll
      for (int k = 0; k < kMergeCh / 8; ++k)
        dst[k] = make_uint4(bf16x2_rn(o[8 * k] * inv, o[8 * k + 1] * inv), bf16x2_rn(o[8 * k + 2] * inv, o[8 * k + 3] * inv),
                            bf16x2_rn(o[8 * k + 4] * inv, o[8 * k + 5] * inv),
                            bf16x2_rn(o[8 * k + 6] * inv, o[8 * k + 7] * inv));
      if (g == 0) a.lse[row] = total != 0.0f ? top + logf(total) : -INFINITY;
    }
  }
  // tiles that see nothing
  for (int t = t0; t < head.x; t += ctas) {
    if (__ldg(a.plan.tiles + 2 * t + 1).z != 0) continue;
    const int4 ta = __ldg(a.plan.tiles + 2 * t);
    const int rows = min(a.tile, ta.w * a.d.heads - ta.y);
    const int64_t row = int64_t(ta.z) * a.d.heads + ta.y;
    for (int i = y * kDenseTile + r; i < rows * (kLatent / 8); i += Y * kDenseTile)
      reinterpret_cast<uint4*>(a.out + row * kLatent)[i] = make_uint4(0, 0, 0, 0);
    for (int i = y * kDenseTile + r; i < rows; i += Y * kDenseTile) a.lse[row + i] = -INFINITY;
  }
}

PFN_cuTensorMapEncodeTiled_v12000 tensor_map_encoder() {
  static std::once_flag once;
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  std::call_once(once, [] {
    void* p = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(p);
  });
  return fn;
}

// Clusters of 2 G CTAs that run at the same time on the current device (asked once per
// device): the runs of a call are cut for that many.  Fewer fit than SMs / (2 G) where
// a GPU processing cluster's SM count is no multiple of 2 G.  0: not to be launched.
int resident_clusters(void (*kernel)(const DenseArgs, const DenseMaps), int G, size_t smem) {
  static std::atomic<int> known[2][kMaxDevices];
  const int most = kDenseMaxClusters / G;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return 0;
  const bool slot = dev >= 0 && dev < kMaxDevices;
  if (slot) {
    const int n = known[G - 1][dev].load(std::memory_order_relaxed);
    if (n > 0) return n;
  }
  // the register split of the roles counts on this many a thread
  cudaFuncAttributes fa;
  if (cudaFuncGetAttributes(&fa, kernel) != cudaSuccess || fa.numRegs != kLaunchRegs) return 0;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  cfg.gridDim = dim3(unsigned(2 * G * most));
  cfg.blockDim = dim3(kDenseThreads);
  cfg.dynamicSmemBytes = smem;
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = unsigned(2 * G);
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  int n = 0;
  if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess || n < 1) {
    cudaGetLastError();
    n = int(min64(most, device_sms() / (2 * G)));
  }
  n = n < 1 ? 1 : n > most ? most : n;
  if (slot) known[G - 1][dev].store(n, std::memory_order_relaxed);
  return n;
}

}  // namespace

cudaError_t launch_dense(DenseArgs a, cudaStream_t st) {
  // Tiles of 128 rows on 2 SMs or of 256 rows on 4: the larger one widens each block
  // once for twice the rows, and wastes up to 255 rows of a sequence instead of 127.
  const int G = dense_pairs(a.d.heads, a.batch, a.total_q) ? 2 : 1;
  a.tile = kDenseTile * G;
  DenseMaps m;
  const auto enc = tensor_map_encoder();
  const uint64_t rows = a.page_table ? uint64_t(a.d.num_pages) * kPage : uint64_t(a.batch) * uint64_t(a.d.max_ctx);
  if (!encode_2d_cached(enc, &m.q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.q, kDqk, uint64_t(a.total_q) * a.d.heads, kDqk * 2,
                        64, 64, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B) ||
      !encode_2d_cached(enc, &m.codes, CU_TENSOR_MAP_DATA_TYPE_UINT8, a.codes, kCodesPerRow, rows, kCodesPerRow, 128, 32,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B) ||
      !encode_2d_cached(enc, &m.rope, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.rope, kRope, rows, kRope * 2, 64, 32,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B))
    return cudaErrorUnknown;
  static KernelAttrs attrs[2];
  const size_t smem = size_t(G == 2 ? Lay<2>::kSmem : Lay<1>::kSmem);
  auto kernel = G == 2 ? dense_pair_kernel : dense_kernel;
  cudaError_t e = prepare_kernel(kernel, smem, false, attrs[G - 1]);
  if (e != cudaSuccess) return e;
  a.clusters = resident_clusters(kernel, G, smem);
  if (a.clusters < 1) return cudaErrorInvalidConfiguration;
  a.max_tiles = int(min64((int64_t(a.total_q) * a.d.heads + a.tile - 1) / a.tile + a.batch, INT32_MAX));
  // no more clusters than there can be runs (one token over at most 256 positions: 16.3
  // instead of 20.7 us)
  const int64_t ctx = a.page_table ? min64(a.d.max_ctx, int64_t(a.d.max_pages) * kPage) : a.d.max_ctx;
  const int64_t most = (a.max_tiles * ((ctx + kDenseBlk - 1) / kDenseBlk) + kDenseMinBlocks - 1) / kDenseMinBlocks;
  a.clusters = int(min64(a.clusters, most));
  // as many threads as there can be sequences or tiles, up to the most
  const int64_t want = max64(max64(a.max_tiles, a.batch), 128);
  const unsigned threads = want >= kPlanThreads ? kPlanThreads : unsigned((want + 31) / 32 * 32);
  CSA2_PROFILED(st, "dense_plan", (e = launch_pdl(dense_plan_kernel, dim3(1), dim3(threads), 0, st, 1, a)));
  if (e != cudaSuccess) return e;
  CSA2_PROFILED(st, "dense_attn",
                (e = launch_pdl(kernel, dim3(unsigned(2 * G * a.clusters)), dim3(kDenseThreads), smem, st, 1, a, m)));
  if (e != cudaSuccess) return e;
  // Few tiles, up to one for four clusters: four threads a row in the merge.  Measured, with and
  // without (graph): one token on 131,072 positions 60 / 88 us, on 16,000 28 / 51; 8 on 4,000
  // 35.5 / 38.1; 4 x 4 tokens on 2,000 25.1 / 26.9.  With up to one for two clusters: 16 tokens on
  // 1,000 (32 heads) 28.1 instead of 25.5.
  const bool few = int64_t(a.max_tiles) * 4 <= a.clusters;
  CSA2_PROFILED(st, "dense_merge",
                (e = few ? launch_pdl(dense_merge_kernel<true>, dim3(kLatent / kMergeCh, unsigned(a.max_tiles), unsigned(G)),
                                      dim3(kDenseTile, kMergeFew), 0, st, 1, a)
                         : launch_pdl(dense_merge_kernel<false>, dim3(kLatent / kMergeCh, unsigned(a.clusters), unsigned(G)),
                                      dim3(kDenseTile), 0, st, 1, a)));
  return e;
}

}  // namespace csa2
