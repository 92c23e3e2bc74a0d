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
// Split over a pair of SMs.  128 rows x 512 fp32 outputs fill the tensor memory
// of an SM, so scores and outputs cannot live on one SM.  A cluster of two CTAs
// divides the work by kind instead:
//   scores CTA (rank 0)   queries resident in tensor memory (288 columns); a block of
//       64 positions is widened from FP4 to bf16 (exact) in shared memory,
//       S[128 x 64] = Q . K^T (M 128, N 64, K 576, bf16 -> fp32); softmax, one thread a
//       row; P as fp16 goes to the other CTA by an asynchronous shared-memory copy;
//   values CTA (rank 1)   widens the same block's latents to fp16 (exact: 6
//       significant bits, 2^-10 .. 2688), O[128 x 512] += P . V (M 128, N 2 x 256, K 64).
// Data flow one way only, so each side runs ahead through its rings (2 blocks of
// keys, 2 score buffers, 3 blocks of P, 2 blocks of values).  Tensor work a block:
// 1,152 and 1,024 cycles; the halves are balanced and nothing is computed twice but
// the widening.
//
// Softmax reference: kept per row as an integer (base-2) and raised only when a
// block's maximum passes it by more than 8, so the outputs are rarely rescaled, and
// then by an exact power of two.  P = 2^(x - ref + 7) <= 2^15 fits fp16; terms
// 2^-31 below the reference are the first to be lost.  Sums are fp32, of the
// unrounded P.
//
// Work division: the (tile, block) pairs of the call are counted by a plan kernel
// and cut into equal runs, one per cluster, whatever the shape: a decode batch splits
// its long contexts, a prompt gives each cluster whole tiles.  A tile cut by a
// boundary leaves partial outputs (fp32, at most two per cluster) that a merge kernel
// joins in a fixed order: results are the same from call to call.
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

constexpr int kConvWarps = 8;
constexpr int kRowWarp0 = 8;                        // warps 8..11: one row a thread (lane quarters 0..3)
constexpr int kMmaWarp = 12;
constexpr int kAuxWarp = 13;
constexpr int kDenseThreads = 14 * 32;

constexpr int kReg = kDenseBlk * 128;               // 64 channels x 64 positions of 16-bit: 8 KB
constexpr int kPSlots = 3;
constexpr int kPBytes = kDenseTile * 128;           // P[128 x 64] fp16
constexpr int kKStages = 2;
constexpr int kKBytes = 9 * kReg;                   // 576 channels
constexpr int kVBytes = 8 * kReg;                   // 512 channels
constexpr int kQSlots = 3;
constexpr int kQPiece = kDenseTile * 64;            // 32 channels x 128 rows of bf16
constexpr int kQPieces = kDqk / 32;
constexpr int kPOff = 0;
constexpr int kKvOff = kPOff + kPSlots * kPBytes;
constexpr int kQOff = kKvOff + kKStages * kKBytes;  // scores CTA: query pieces; values CTA: output staging
constexpr int kDenseSmem = kQOff + kQSlots * kQPiece;
static_assert(4 * 4096 <= kQSlots * kQPiece, "output staging of the values CTA");

constexpr uint32_t kSCol = 320;                     // score buffers behind the 288 query columns
constexpr uint32_t kTmemAll = 512;
constexpr int kMetaWarp = 3 * 32 * 4;               // alpha, sum, reference of a warp's rows

struct DenseSmall {
  uint64_t kv_full[kKStages], kv_empty[kKStages];
  uint64_t s_full[2], s_empty[2];
  uint64_t q_full;
  uint64_t qc_full[kQSlots], qc_empty[kQSlots];
  uint64_t p_free[kPSlots];                         // scores CTA: slot read by the values CTA (remote arrival)
  uint64_t p_full[kPSlots];                         // values CTA: bytes of P and meta have arrived
  uint64_t corr[kPSlots];                           // values CTA: outputs brought to the slot's reference
  uint64_t pv_done[kPSlots];
  uint64_t o_free;
  uint64_t drain;
  uint32_t tmem_slot;
  int abort;
  int page_ok[4];                                   // of the block n & 3
  __align__(16) float meta[kPSlots][4][3][32];
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

__device__ inline void arrive_remote(uint32_t rbar) {
  asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" ::"r"(rbar) : "memory");
}

__device__ inline void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(tc::smem_u32(bar)) : "memory");
}

__device__ inline bool try_wait_cluster(uint64_t* bar, uint32_t parity, uint32_t hint_ns) {
  uint32_t done;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2, %3;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(done)
      : "r"(tc::smem_u32(bar)), "r"(parity), "r"(hint_ns)
      : "memory");
  return done != 0;
}

// Every wait of the kernel: bounded (200 ms against microseconds), and cut short
// once another role of the CTA has given up.  False: the caller's role ends.
__device__ __noinline__ bool wait_slow(DenseSmall& sm, uint64_t* bar, uint32_t parity, uint8_t* ws) {
  const uint64_t t0 = tc::globaltimer_ns();
  while (true) {
    if (try_wait_cluster(bar, parity, 20000u)) return true;
    if (*reinterpret_cast<volatile int*>(&sm.abort)) return false;
    if (tc::globaltimer_ns() - t0 > 200ull * 1000 * 1000) {
      *reinterpret_cast<volatile int*>(&sm.abort) = 1;
      raise_err(ws, CSA2_DEV_TIMEOUT);
      return false;
    }
  }
}
__device__ inline bool wait_on(DenseSmall& sm, uint64_t* bar, uint32_t parity, uint8_t* ws) {
  return try_wait_cluster(bar, parity, 0u) || wait_slow(sm, bar, parity, ws);
}
// the same for a converged warp: one answer for all lanes
__device__ inline bool wait_warp(DenseSmall& sm, uint64_t* bar, uint32_t parity, uint8_t* ws) {
  return __all_sync(0xFFFFFFFFu, wait_on(sm, bar, parity, ws));
}

// D[tmem] (+)= A[tmem] * B[smem]^T
__device__ inline void mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}"
      ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(uint32_t(acc))
      : "memory");
}

// Instruction descriptor with fp16 A/B and fp32 accumulation.
__host__ __device__ constexpr uint32_t idesc_f16(int M, int N, int a_mn, int b_mn) {
  return (1u << 4) | (uint32_t(a_mn) << 15) | (uint32_t(b_mn) << 16) | (uint32_t(N >> 3) << 17) |
         (uint32_t(M >> 4) << 24);
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
// fp16 values (normal or zero) as the bf16 of 2^-112 times them: the 5-bit
// exponent moved into the 8-bit field, the top 7 mantissa bits kept
__device__ inline uint32_t f16x2_as_bf16x2(uint32_t h) { return ((h >> 3) & 0x0FFF0FFFu) | (h & 0x80008000u); }

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

// ---------------------------------------------------------------------------
// Widening warps (both CTAs).  Warp w takes the block's rows 8 w .. 8 w + 7, lane
// = 8 * piece + row: a quarter-warp stores one 16-byte chunk of 8 rows (all 32 banks,
// 128-byte swizzle), a load instruction reads 64 contiguous bytes of 8 rows.
// The next block is loaded before the current one waits for its stage.
// ---------------------------------------------------------------------------
struct Raw {
  uint4 cw[4];
  uint32_t sc[2];     // four pairs of E4M3 scales
  uint4 rp[2];
  int ok;             // the page is valid
};

template <bool kScores>
__device__ inline void load_raw(const DenseArgs& a, int4 ta, int4 tb, int blk, int w, int lane, Raw& r) {
  const int b = ta.x, t = blk * kDenseBlk + 8 * w + (lane & 7), p = lane >> 3;
  int64_t row = -1;
  r.ok = 1;
  if (a.page_table) {
    const int pg = __ldg(a.page_table + int64_t(b) * a.d.max_pages + blk);
    if (pg < 0 || pg >= a.d.num_pages) {
      r.ok = 0;
      if (kScores && lane == 0 && w == 0) raise_err(a.ws, CSA2_DEV_PAGE_ID);
    } else {
      row = int64_t(pg) * kPage + (t & (kPage - 1));
    }
  } else {
    row = int64_t(b) * a.d.max_ctx + t;
  }
  // rows behind the context hold anything: they are zeros (0 * P stays 0)
  if (t >= tb.x || row < 0) {
#pragma unroll
    for (int j = 0; j < 4; ++j) r.cw[j] = make_uint4(0, 0, 0, 0);
    r.sc[0] = r.sc[1] = 0;
    if (kScores) r.rp[0] = r.rp[1] = make_uint4(0, 0, 0, 0);
    return;
  }
  const uint4* cp = reinterpret_cast<const uint4*>(a.codes + row * kCodesPerRow);
  const uint16_t* sp = reinterpret_cast<const uint16_t*>(a.scales + row * kScalesPerRow);
#pragma unroll
  for (int j = 0; j < 4; ++j) r.cw[j] = __ldg(cp + 4 * j + p);
  r.sc[0] = uint32_t(__ldg(sp + p)) | uint32_t(__ldg(sp + 4 + p)) << 16;
  r.sc[1] = uint32_t(__ldg(sp + 8 + p)) | uint32_t(__ldg(sp + 12 + p)) << 16;
  if (kScores) {
    const uint4* rp = reinterpret_cast<const uint4*>(a.rope + row * kRope);
    r.rp[0] = __ldg(rp + p);
    r.rp[1] = __ldg(rp + 4 + p);
  }
}

// Four FP4 words' worth of one 16-byte chunk: 8 channels under one scale.
template <bool kScores>
__device__ inline uint4 widen8(uint32_t w, uint32_t sc2) {
  uint32_t h[4] = {e2m1_byte_f16x2<0>(w), e2m1_byte_f16x2<1>(w), e2m1_byte_f16x2<2>(w), e2m1_byte_f16x2<3>(w)};
#pragma unroll
  for (int i = 0; i < 4; ++i) h[i] = kScores ? mul_bf16x2(f16x2_as_bf16x2(h[i]), sc2) : mul_f16x2(h[i], sc2);
  return make_uint4(h[0], h[1], h[2], h[3]);
}

template <bool kScores>
__device__ inline void store_wide(uint8_t* dst, const Raw& r, int w, int lane) {
  const int row = 8 * w + (lane & 7), p = lane >> 3;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int piece = 4 * j + p;                     // 16 code bytes: channels 32 piece .. + 31
    const uint32_t two = e4m3x2_to_f16x2(uint16_t(r.sc[j >> 1] >> (16 * (j & 1))));
    uint32_t s0, s1;
    if (kScores) {
      // scale * 2^112 in bf16 (exact: 4 significant bits, below 2^121), twice
      const __half2 hh = *reinterpret_cast<const __half2*>(&two);
      const float f0 = __low2float(hh) * 5.192296858534828e33f, f1 = __high2float(hh) * 5.192296858534828e33f;
      s0 = __byte_perm(__float_as_uint(f0), 0, 0x3232);
      s1 = __byte_perm(__float_as_uint(f1), 0, 0x3232);
    } else {
      s0 = __byte_perm(two, 0, 0x1010);
      s1 = __byte_perm(two, 0, 0x3232);
    }
    uint8_t* reg = dst + (piece >> 1) * kReg;
    const int c0 = (piece & 1) * 4;
    const uint32_t w4[4] = {r.cw[j].x, r.cw[j].y, r.cw[j].z, r.cw[j].w};
#pragma unroll
    for (int i = 0; i < 4; ++i)
      *reinterpret_cast<uint4*>(reg + tc::sw128_offset(row, c0 + i)) = widen8<kScores>(w4[i], i < 2 ? s0 : s1);
  }
  if (kScores) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
      *reinterpret_cast<uint4*>(dst + 8 * kReg + tc::sw128_offset(row, 4 * j + p)) = r.rp[j];
  }
}

template <bool kScores>
__device__ inline void widen_role(const DenseArgs& a, DenseSmall& sm, uint8_t* base, int cl, int w, int lane) {
  Walk walk(a.plan, cl);
  Item it;
  if (!walk.next(it)) return;
  Raw cur;
  load_raw<kScores>(a, it.a, it.b, it.blk, w, lane, cur);
  for (uint32_t n = 0;; ++n) {
    // the next block's loads
    Raw nxt;
    bool more = true;
    ++it.blk;
    if (--it.n == 0) more = walk.next(it);
    if (more) load_raw<kScores>(a, it.a, it.b, it.blk, w, lane, nxt);
    const uint32_t st = n % kKStages;
    if (!wait_warp(sm, &sm.kv_empty[st], ((n / kKStages) & 1) ^ 1, a.ws)) return;
    store_wide<kScores>(base + kKvOff + st * (kScores ? kKBytes : kVBytes), cur, w, lane);
    if (kScores && w == 0 && lane == 0) sm.page_ok[n & 3] = cur.ok;
    tc::fence_proxy_async_smem();
    __syncwarp();
    if (lane == 0) arrive(&sm.kv_full[st]);
    if (!more) return;
    cur = nxt;
  }
}

// ---------------------------------------------------------------------------
// Scores CTA
// ---------------------------------------------------------------------------
__device__ inline void scores_mma_role(const DenseArgs& a, DenseSmall& sm, uint8_t* base, int cl, uint32_t tmem) {
  constexpr uint32_t id = tc::idesc_bf16(kDenseTile, kDenseBlk, 0, 0);
  Walk walk(a.plan, cl);
  Item it;
  uint32_t n = 0;
  for (uint32_t k = 0; walk.next(it); ++k) {
    if (!wait_on(sm, &sm.q_full, k & 1, a.ws)) return;
    for (int j = 0; j < it.n; ++j, ++n) {
      const uint32_t st = n % kKStages, buf = n & 1;
      if (!wait_on(sm, &sm.kv_full[st], (n / kKStages) & 1, a.ws)) return;
      if (!wait_on(sm, &sm.s_empty[buf], ((n >> 1) & 1) ^ 1, a.ws)) return;
      tc::tc_fence_after_sync();
      const uint64_t bd = tc::smem_desc(tc::smem_u32(base + kKvOff + st * kKBytes), 16, 1024, 2);
      const uint32_t d = tmem + kSCol + buf * kDenseBlk;
#pragma unroll
      for (int ks = 0; ks < kDqk / 16; ++ks)
        mma_ts(d, tmem + ks * 8, bd + (((ks >> 2) * kReg + (ks & 3) * 32) >> 4), id, ks > 0);
      tc::mma_commit(&sm.kv_empty[st]);
      tc::mma_commit(&sm.s_full[buf]);
    }
  }
}

__device__ inline void query_tma_role(const DenseArgs& a, DenseSmall& sm, uint8_t* base, int cl, const CUtensorMap* map) {
  Walk walk(a.plan, cl);
  Item it;
  uint32_t n = 0;
  while (walk.next(it)) {
    const int y = it.a.z * a.d.heads + it.a.y;
    for (int c = 0; c < kQPieces; ++c, ++n) {
      const uint32_t s = n % kQSlots;
      if (!wait_on(sm, &sm.qc_empty[s], ((n / kQSlots) & 1) ^ 1, a.ws)) return;
      tc::mbar_expect_tx(&sm.qc_full[s], kQPiece);
      tc::tma_load_2d(map, base + kQOff + s * kQPiece, 32 * c, y, &sm.qc_full[s]);
    }
  }
}

__device__ inline void softmax_role(const DenseArgs& a, DenseSmall& sm, uint8_t* base, int cl, int wq, int lane,
                                    uint32_t tmem) {
  const uint32_t lanes = tmem + (uint32_t(wq * 32) << 16);
  const int r = wq * 32 + lane;
  const float c2 = a.scale * 1.4426950408889634f;
  const bool neg = c2 < 0.0f;
  const float c = fmaxf(fabsf(c2), 1.17549435e-38f);
  uint32_t n = 0, nq = 0;
  Walk walk(a.plan, cl);
  Item it;
  uint32_t peer_p[kPSlots], peer_meta[kPSlots], peer_bar[kPSlots];
#pragma unroll
  for (int s = 0; s < kPSlots; ++s) {
    peer_p[s] = peer_addr(base + kPOff + s * kPBytes + wq * 4096, 1);
    peer_meta[s] = peer_addr(&sm.meta[s][wq][0][0], 1);
    peer_bar[s] = peer_addr(&sm.p_full[s], 1);
  }
  while (walk.next(it)) {
    // the tile's queries into tensor memory, 32 channels (16 columns) at a time; the
    // MMAs that read the previous tile's are done (their scores have been read)
    for (int q = 0; q < kQPieces; ++q, ++nq) {
      const uint32_t s = nq % kQSlots;
      if (!wait_warp(sm, &sm.qc_full[s], (nq / kQSlots) & 1, a.ws)) return;
      uint32_t v[16];
      const uint8_t* src = base + kQOff + s * kQPiece + r * 64;      // 64-byte swizzle: chunk ^ (row / 2) % 4
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const uint4 x = *reinterpret_cast<const uint4*>(src + ((i ^ ((r >> 1) & 3)) << 4));
        v[4 * i] = x.x; v[4 * i + 1] = x.y; v[4 * i + 2] = x.z; v[4 * i + 3] = x.w;
      }
      tmem_st16_nowait(lanes + q * 16, v);
      __syncwarp();
      if (lane == 0) arrive(&sm.qc_empty[s]);
    }
    tmem_wait_st();
    tc::tc_fence_before_sync();
    __syncwarp();
    if (lane == 0) arrive(&sm.q_full);

    // positions this row sees: first .. last
    const int lr = it.a.y + r, tok = lr / a.d.heads;
    int last = -1, first = 0;
    if (tok < it.a.w) {
      last = a.causal ? it.b.x - it.a.w + tok : it.b.x - 1;
      if (a.window > 0) first = max(0, last - a.window + 1);
    }
    float ref = -INFINITY, sum = 0.0f;
    for (int j = 0; j < it.n; ++j, ++n) {
      const uint32_t buf = n & 1, slot = n % kPSlots;
      if (!wait_warp(sm, &sm.s_full[buf], (n >> 1) & 1, a.ws)) return;
      tc::tc_fence_after_sync();
      float x[64];
      {
        float h[32];
        tc::tmem_ld32(lanes + kSCol + buf * kDenseBlk, h);
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = h[i];
        tc::tmem_ld32(lanes + kSCol + buf * kDenseBlk + 32, h);
#pragma unroll
        for (int i = 0; i < 32; ++i) x[32 + i] = h[i];
      }
      const int t0 = (it.blk + j) * kDenseBlk;
      int lo = first - t0, hi = last - t0;
      if (!sm.page_ok[n & 3]) hi = -1;
      tc::tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) arrive(&sm.s_empty[buf]);
      if (neg) {
#pragma unroll
        for (int i = 0; i < 64; ++i) x[i] = -x[i];
      }
      if (__any_sync(0xFFFFFFFFu, lo > 0 || hi < kDenseBlk - 1)) {
#pragma unroll
        for (int i = 0; i < 64; ++i) x[i] = (i >= lo && i <= hi) ? x[i] : -INFINITY;
      }
      float m[4] = {x[0], x[1], x[2], x[3]};
#pragma unroll
      for (int i = 4; i < 64; ++i) m[i & 3] = fmaxf(m[i & 3], x[i]);
      const float top = fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3])) * c;
      float alpha = 1.0f;
      if (top > ref + 8.0f) {
        const float now = ceilf(top);
        if (ref != -INFINITY) alpha = ex2(ref - now);
        sum *= alpha;
        ref = now;
      }
      const float sub = ref == -INFINITY ? 0.0f : ref - 7.0f;
      uint32_t pk[32];
      float s4[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float p0 = ex2(__fmaf_rn(x[2 * i], c, -sub)), p1 = ex2(__fmaf_rn(x[2 * i + 1], c, -sub));
        s4[(2 * i) & 3] += p0;
        s4[(2 * i + 1) & 3] += p1;
        pk[i] = f16x2_rn(p0, p1);
      }
      sum += (s4[0] + s4[1]) + (s4[2] + s4[3]);
      if (!wait_warp(sm, &sm.p_free[slot], ((n / kPSlots) & 1) ^ 1, a.ws)) return;
      uint8_t* ps = base + kPOff + slot * kPBytes;
#pragma unroll
      for (int i = 0; i < 8; ++i)
        *reinterpret_cast<uint4*>(ps + tc::sw128_offset(r, i)) =
            make_uint4(pk[4 * i], pk[4 * i + 1], pk[4 * i + 2], pk[4 * i + 3]);
      sm.meta[slot][wq][0][lane] = alpha;
      sm.meta[slot][wq][1][lane] = sum;
      sm.meta[slot][wq][2][lane] = sub;
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) {
        copy_to_peer(peer_p[slot], ps + wq * 4096, 4096, peer_bar[slot]);
        copy_to_peer(peer_meta[slot], &sm.meta[slot][wq][0][0], kMetaWarp, peer_bar[slot]);
      }
      __syncwarp();
    }
  }
}

// ---------------------------------------------------------------------------
// Values CTA
// ---------------------------------------------------------------------------
__device__ inline void values_mma_role(const DenseArgs& a, DenseSmall& sm, uint8_t* base, int cl, uint32_t tmem) {
  constexpr uint32_t id = idesc_f16(kDenseTile, 256, 0, 1);
  Walk walk(a.plan, cl);
  Item it;
  uint32_t n = 0;
  for (uint32_t k = 0; walk.next(it); ++k) {
    if (!wait_on(sm, &sm.o_free, (k & 1) ^ 1, a.ws)) return;
    for (int j = 0; j < it.n; ++j, ++n) {
      const uint32_t st = n % kKStages, slot = n % kPSlots, ph = (n / kPSlots) & 1;
      if (!wait_on(sm, &sm.kv_full[st], (n / kKStages) & 1, a.ws)) return;
      if (!wait_on(sm, &sm.p_full[slot], ph, a.ws)) return;
      if (!wait_on(sm, &sm.corr[slot], ph, a.ws)) return;
      tc::tc_fence_after_sync();
      const uint64_t ad = tc::smem_desc(tc::smem_u32(base + kPOff + slot * kPBytes), 16, 1024, 2);
      const uint64_t bd = tc::smem_desc(tc::smem_u32(base + kKvOff + st * kVBytes), kReg, 1024, 2);
#pragma unroll
      for (int ks = 0; ks < kDenseBlk / 16; ++ks)
#pragma unroll
        for (int h = 0; h < 2; ++h)
          tc::mma_bf16(tmem + h * 256, ad + ((ks * 32) >> 4), bd + ((h * 4 * kReg + ks * 2048) >> 4), id, j > 0 || ks > 0);
      tc::mma_commit(&sm.kv_empty[st]);
      tc::mma_commit(&sm.pv_done[slot]);
    }
  }
}

// Hands each slot of P back once its products are done.
__device__ inline void slot_role(const DenseArgs& a, DenseSmall& sm, int cl) {
  Walk walk(a.plan, cl);
  for (int n = 0, all = walk.left; n < all; ++n) {
    const uint32_t slot = uint32_t(n) % kPSlots;
    if (!wait_on(sm, &sm.pv_done[slot], (uint32_t(n) / kPSlots) & 1, a.ws)) return;
    if (n + kPSlots < all) {
      tc::mbar_expect_tx(&sm.p_full[slot], kPBytes + 4 * kMetaWarp);
      arrive_remote(peer_addr(&sm.p_free[slot], 0));
    }
  }
}

__device__ inline void output_role(const DenseArgs& a, DenseSmall& sm, uint8_t* base, int cl, int wq, int lane,
                                   uint32_t tmem) {
  const uint32_t lanes = tmem + (uint32_t(wq * 32) << 16);
  const int r = wq * 32 + lane;
  uint8_t* stage = base + kQOff + wq * 4096;
  Walk walk(a.plan, cl);
  Item it;
  uint32_t n = 0;
  while (walk.next(it)) {
    float sum = 0.0f, sub = 0.0f;
    for (int j = 0; j < it.n; ++j, ++n) {
      const uint32_t slot = n % kPSlots;
      if (!wait_warp(sm, &sm.p_full[slot], (n / kPSlots) & 1, a.ws)) return;
      const float alpha = sm.meta[slot][wq][0][lane];
      sum = sm.meta[slot][wq][1][lane];
      sub = sm.meta[slot][wq][2][lane];
      if (__any_sync(0xFFFFFFFFu, alpha != 1.0f)) {
        // the outputs so far, once their products are done, to the new reference
        const uint32_t m = n - 1;
        if (!wait_warp(sm, &sm.pv_done[m % kPSlots], (m / kPSlots) & 1, a.ws)) return;
        tc::tc_fence_after_sync();
#pragma unroll 1
        for (int col = 0; col < kLatent; col += 8) {
          float v[8];
          tc::tmem_ld8(lanes + col, v);
#pragma unroll
          for (int i = 0; i < 8; ++i) v[i] *= alpha;
          tc::tmem_st8(lanes + col, v);
        }
        tc::tc_fence_before_sync();
      }
      __syncwarp();
      if (lane == 0) arrive(&sm.corr[slot]);
    }
    const uint32_t m = n - 1;
    if (!wait_warp(sm, &sm.pv_done[m % kPSlots], (m / kPSlots) & 1, a.ws)) return;
    tc::tc_fence_after_sync();
    const float inv = sum > 0.0f ? 1.0f / sum : 0.0f;
    const float lse = sum > 0.0f ? (sub + log2f(sum)) * 0.6931471805599453f : -INFINITY;
    const int lr = it.a.y + r, rows = it.a.w * a.d.heads;
    if (it.head || it.tail) {
      const int slot = 2 * cl + (it.head ? 0 : 1);
      float* po = a.part_o + int64_t(slot) * kLatent * kDenseTile + r;
      a.part_lse[slot * kDenseTile + r] = lse;
#pragma unroll 1
      for (int col = 0; col < kLatent; col += 32) {
        float v[32];
        tc::tmem_ld32(lanes + col, v);
#pragma unroll
        for (int i = 0; i < 32; ++i) po[(col + i) * kDenseTile] = v[i] * inv;
      }
    } else {
      const int64_t g0 = int64_t(it.a.z) * a.d.heads + it.a.y + wq * 32;    // the warp's first row
      const int have = min(32, rows - it.a.y - wq * 32);                    // rows of it that exist
      if (lr < rows) a.lse[g0 + lane] = lse;
#pragma unroll 1
      for (int col = 0; col < kLatent; col += 64) {
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          float v[32];
          tc::tmem_ld32(lanes + col + 32 * half, v);
#pragma unroll
          for (int i = 0; i < 4; ++i)
            *reinterpret_cast<uint4*>(stage + tc::sw128_offset(lane, 4 * half + i)) =
                make_uint4(bf16x2_rn(v[8 * i] * inv, v[8 * i + 1] * inv), bf16x2_rn(v[8 * i + 2] * inv, v[8 * i + 3] * inv),
                           bf16x2_rn(v[8 * i + 4] * inv, v[8 * i + 5] * inv),
                           bf16x2_rn(v[8 * i + 6] * inv, v[8 * i + 7] * inv));
        }
        __syncwarp();
        // four rows of 128 bytes an instruction
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int row = 4 * i + (lane >> 3);
          if (row < have)
            *reinterpret_cast<uint4*>(a.out + (g0 + row) * kLatent + col + 8 * (lane & 7)) =
                *reinterpret_cast<const uint4*>(stage + tc::sw128_offset(row, lane & 7));
        }
        __syncwarp();
      }
    }
    tc::tc_fence_before_sync();
    __syncwarp();
    if (lane == 0) arrive(&sm.o_free);
  }
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kDenseThreads, 1)
    dense_kernel(DenseArgs a, const __grid_constant__ CUtensorMap qmap) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  uint8_t* base = smem_raw + ((1024u - (tc::smem_u32(smem_raw) & 1023u)) & 1023u);
  __shared__ DenseSmall sm;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  const int rank = blockIdx.x & 1, cl = blockIdx.x >> 1;
  if (wid == 0) tc::tmem_alloc(&sm.tmem_slot, kTmemAll);
  if (tid == 0) {
    for (int i = 0; i < kKStages; ++i) {
      tc::mbar_init(&sm.kv_full[i], kConvWarps);
      tc::mbar_init(&sm.kv_empty[i], 1);
    }
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sm.s_full[i], 1);
      tc::mbar_init(&sm.s_empty[i], 4);
    }
    tc::mbar_init(&sm.q_full, 4);
    for (int i = 0; i < kQSlots; ++i) {
      tc::mbar_init(&sm.qc_full[i], 1);
      tc::mbar_init(&sm.qc_empty[i], 4);
    }
    for (int i = 0; i < kPSlots; ++i) {
      tc::mbar_init(&sm.p_free[i], 1);
      tc::mbar_init(&sm.p_full[i], 1);
      tc::mbar_init(&sm.corr[i], 4);
      tc::mbar_init(&sm.pv_done[i], 1);
    }
    tc::mbar_init(&sm.o_free, 4);
    tc::mbar_init(&sm.drain, 1);
    sm.abort = 0;
    tc::fence_mbar_init();
    if (rank == 1)
      for (int i = 0; i < kPSlots; ++i) tc::mbar_expect_tx(&sm.p_full[i], kPBytes + 4 * kMetaWarp);
  }
  tc::tc_fence_before_sync();
  __syncthreads();
  tc::tc_fence_after_sync();
  // both CTAs' barriers stand before either writes into the other
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  const uint32_t tmem = sm.tmem_slot;
  pdl_wait();
  pdl_launch_dependents();
  if (rank == 0) {
    if (wid < kConvWarps) widen_role<true>(a, sm, base, cl, wid, lane);
    else if (wid < kRowWarp0 + 4) softmax_role(a, sm, base, cl, wid - kRowWarp0, lane, tmem);
    else if (wid == kMmaWarp && lane == 0) scores_mma_role(a, sm, base, cl, tmem);
    else if (wid == kAuxWarp && lane == 0) query_tma_role(a, sm, base, cl, &qmap);
  } else {
    if (wid < kConvWarps) widen_role<false>(a, sm, base, cl, wid, lane);
    else if (wid < kRowWarp0 + 4) output_role(a, sm, base, cl, wid - kRowWarp0, lane, tmem);
    else if (wid == kMmaWarp && lane == 0) values_mma_role(a, sm, base, cl, tmem);
    else if (wid == kAuxWarp && lane == 0) slot_role(a, sm, cl);
  }
  // the thread that issued the MMAs sees them done (they are, unless a wait gave up)
  if (wid == kMmaWarp && lane == 0) {
    tc::mma_commit(&sm.drain);
    wait_slow(sm, &sm.drain, 0, a.ws);
  }
  __syncwarp();
  tc::tc_fence_before_sync();
  __syncthreads();
  tc::tc_fence_after_sync();
  // neither CTA leaves while the other may still write into it
  asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
  asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (wid == 0) tc::tmem_dealloc(tmem, kTmemAll);
}

// ---------------------------------------------------------------------------
// Plan: one CTA.  Sequences -> tiles of 128 rows -> blocks each tile sees ->
// equal runs of blocks, one per cluster.
// ---------------------------------------------------------------------------
constexpr int kPlanThreads = 1024;

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
  int64_t before = 0, all = 0;
  for (int i = 0; i < kPlanThreads / 32; ++i) {
    if (i < w) before += buf[i];
    all += buf[i];
  }
  total = all;
  return before + x - v;      // exclusive
}

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
  int before = INT32_MIN, all = INT32_MIN;
  for (int i = 0; i < kPlanThreads / 32; ++i) {
    if (i < w) before = max(before, int(buf[i]));
    all = max(all, int(buf[i]));
  }
  total = all;
  return max(before, x);      // inclusive
}

__global__ void __launch_bounds__(kPlanThreads, 1) dense_plan_kernel(DenseArgs a) {
  __shared__ int64_t buf[kPlanThreads / 32];
  const int tid = threadIdx.x, H = a.d.heads;
  pdl_wait();
  pdl_launch_dependents();
  // sequences: a q_start that falls back or leaves [0, total_q] is reported and
  // replaced by the nearest value that keeps the order
  const int s0 = __ldg(a.q_start);
  int reach = min(max(s0, 0), a.total_q);
  if (tid == 0 && reach != s0) raise_err(a.ws, CSA2_DEV_Q_START);
  int ntiles = 0;
  for (int base = 0; base < a.batch; base += kPlanThreads) {
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
    __shared__ int edge[kPlanThreads / 32];
    __syncthreads();
    if ((tid & 31) == 31) edge[tid >> 5] = upto;
    __syncthreads();
    if ((tid & 31) == 0) from = tid == 0 ? reach : edge[(tid >> 5) - 1];
    const int len = b < a.batch ? upto - from : 0;
    const int64_t tiles = (int64_t(len) * H + kDenseTile - 1) / kDenseTile;
    int64_t all;
    const int64_t at = block_scan_sum(tiles, buf, all);
    if (b < a.batch) {
      const int64_t ctx = checked_ctx(a.ctx_len, a.d, b, a.page_table != nullptr, a.ws);
      a.plan.seqs[b] = make_int4(ntiles + int(at), from, len, int(ctx));
    }
    ntiles += int(all);
    reach = max(reach, top);
  }
  __syncthreads();
  // tiles
  int64_t blocks = 0;
  for (int base = 0; base < ntiles; base += kPlanThreads) {
    const int t = base + tid;
    int nb = 0, fb = 0;
    if (t < ntiles) {
      int lo = 0, hi = a.batch - 1;                  // the last sequence whose first tile is <= t
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.plan.seqs[mid].x <= t) lo = mid;
        else hi = mid - 1;
      }
      const int4 s = a.plan.seqs[lo];
      const int row0 = (t - s.x) * kDenseTile;
      const int tok0 = row0 / H, tok1 = min(s.z - 1, (row0 + kDenseTile - 1) / H);
      int first = 0, last = s.w - 1;
      if (a.causal) {
        last = s.w - s.z + tok1;
        if (a.window > 0) first = max(0, s.w - s.z + tok0 - a.window + 1);
      }
      if (last >= first) {
        fb = first / kDenseBlk;
        nb = last / kDenseBlk - fb + 1;
      }
      a.plan.tiles[2 * t] = make_int4(lo, row0, s.y, s.z);
      a.plan.tiles[2 * t + 1] = make_int4(s.w, fb, nb, 0);
    }
    int64_t all;
    const int64_t at = block_scan_sum(nb, buf, all);
    if (t < ntiles) a.plan.before[t] = blocks + at;
    blocks += all;
  }
  __syncthreads();
  const int64_t want = (blocks + kDenseMinBlocks - 1) / kDenseMinBlocks;
  const int active = int(min64(a.clusters, max64(want, 1)));
  if (tid == 0) *a.plan.head = make_int4(ntiles, blocks > 0 ? active : 0, 0, 0);
  for (int c = tid; c < a.clusters; c += kPlanThreads) {
    int4 run = make_int4(0, 0, 0, 0);
    const int64_t w0 = c < active ? blocks * c / active : blocks, w1 = c < active ? blocks * (c + 1) / active : blocks;
    if (w1 > w0) {
      int lo = 0, hi = ntiles - 1;                   // the last tile whose first block is <= w0
      while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (a.plan.before[mid] <= w0) lo = mid;
        else hi = mid - 1;
      }
      run = make_int4(lo, int(w0 - a.plan.before[lo]), int(w1 - w0), 0);
    }
    a.plan.runs[c] = run;
  }
}

// ---------------------------------------------------------------------------
// Merge: CTA (g, c) joins 16 channels of the tile that the boundary before run c
// cuts, if c is the first boundary inside it.  Thread = row.  It also writes the
// rows of tiles that see nothing.
// ---------------------------------------------------------------------------
constexpr int kMergeCh = 16;

__global__ void __launch_bounds__(kDenseTile) dense_merge_kernel(DenseArgs a) {
  pdl_wait();
  pdl_launch_dependents();
  const int r = threadIdx.x, g = blockIdx.x, c = blockIdx.y;
  const int4 head = __ldg(a.plan.head);
  if (c < head.y) {
    const int4 run = __ldg(a.plan.runs + c);
    const int64_t w0 = run.y;                        // blocks of the tile before this run
    if (w0 > 0) {
      const int4 ta = __ldg(a.plan.tiles + 2 * run.x), tb = __ldg(a.plan.tiles + 2 * run.x + 1);
      const int64_t before = __ldg(a.plan.before + run.x);
      const int4 prev = __ldg(a.plan.runs + c - 1);
      // first boundary inside: the run before starts at or before the tile's first block
      const bool mine = prev.x != run.x || prev.y == 0;
      const int lr = ta.y + r;
      if (mine && lr < ta.w * a.d.heads) {
        // last run that touches the tile
        int c1 = c;
        int64_t done = w0 + run.z;
        while (done < tb.z) {
          ++c1;
          done += __ldg(a.plan.runs + c1).z;
        }
        (void)before;
        const int n = c1 - c + 2;                    // pieces: runs c - 1 .. c1
        // the first piece ends the run before (its tail); the others start theirs
        const auto slot = [&](int i) { return i == 0 ? 2 * (c - 1) + 1 : 2 * (c - 1 + i); };
        float top = -INFINITY;
        for (int i = 0; i < n; ++i) top = fmaxf(top, a.part_lse[slot(i) * kDenseTile + r]);
        float o[kMergeCh], total = 0.0f;
#pragma unroll
        for (int k = 0; k < kMergeCh; ++k) o[k] = 0.0f;
        for (int i = 0; i < n; ++i) {
          const int s = slot(i);
          const float l = a.part_lse[s * kDenseTile + r];
          const float w = l == -INFINITY ? 0.0f : exp2f((l - top) * 1.4426950408889634f);
          total += w;
          const float* po = a.part_o + (int64_t(s) * kLatent + g * kMergeCh) * kDenseTile + r;
#pragma unroll
          for (int k = 0; k < kMergeCh; ++k) o[k] = fmaf(w, po[k * kDenseTile], o[k]);
        }
        const float inv = total > 0.0f ? 1.0f / total : 0.0f;
        const int64_t row = int64_t(ta.z) * a.d.heads + lr;
        uint4* dst = reinterpret_cast<uint4*>(a.out + row * kLatent + g * kMergeCh);
#pragma unroll
        for (int k = 0; k < kMergeCh / 8; ++k)
          dst[k] = make_uint4(bf16x2_rn(o[8 * k] * inv, o[8 * k + 1] * inv), bf16x2_rn(o[8 * k + 2] * inv, o[8 * k + 3] * inv),
                              bf16x2_rn(o[8 * k + 4] * inv, o[8 * k + 5] * inv),
                              bf16x2_rn(o[8 * k + 6] * inv, o[8 * k + 7] * inv));
        if (g == 0) a.lse[row] = total > 0.0f ? top + logf(total) : -INFINITY;
      }
    }
  }
  const int ctas = gridDim.x * gridDim.y;
  for (int t = blockIdx.y * gridDim.x + blockIdx.x; t < head.x; t += ctas) {
    if (__ldg(a.plan.tiles + 2 * t + 1).z != 0) continue;
    const int4 ta = __ldg(a.plan.tiles + 2 * t);
    const int rows = min(kDenseTile, ta.w * a.d.heads - ta.y);
    const int64_t row = int64_t(ta.z) * a.d.heads + ta.y;
    for (int i = r; i < rows * (kLatent / 8); i += kDenseTile)
      reinterpret_cast<uint4*>(a.out + row * kLatent)[i] = make_uint4(0, 0, 0, 0);
    if (r < rows) a.lse[row + r] = -INFINITY;
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

}  // namespace

cudaError_t launch_dense(DenseArgs a, cudaStream_t st) {
  a.clusters = int(min64(kDenseMaxClusters, device_sms() / 2));
  if (a.clusters < 1) a.clusters = 1;
  CUtensorMap qmap;
  if (!encode_2d_cached(tensor_map_encoder(), &qmap, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.q, kDqk,
                        uint64_t(a.total_q) * a.d.heads, kDqk * 2, 32, kDenseTile, CU_TENSOR_MAP_SWIZZLE_64B,
                        CU_TENSOR_MAP_L2_PROMOTION_L2_256B))
    return cudaErrorUnknown;
  static KernelAttrs attrs;
  constexpr size_t smem = size_t(kDenseSmem) + 1024;
  cudaError_t e = prepare_kernel(dense_kernel, smem, false, attrs);
  if (e != cudaSuccess) return e;
  CSA2_PROFILED(st, "dense_plan", (e = launch_pdl(dense_plan_kernel, dim3(1), dim3(kPlanThreads), 0, st, 1, a)));
  if (e != cudaSuccess) return e;
  CSA2_PROFILED(st, "dense_attn",
                (e = launch_pdl(dense_kernel, dim3(unsigned(2 * a.clusters)), dim3(kDenseThreads), smem, st, 1, a, qmap)));
  if (e != cudaSuccess) return e;
  CSA2_PROFILED(st, "dense_merge",
                (e = launch_pdl(dense_merge_kernel, dim3(kLatent / kMergeCh, unsigned(a.clusters)), dim3(kDenseTile), 0,
                                st, 1, a)));
  return e;
}

}  // namespace csa2
