// window.cu -- attention of new tokens over a sliding window of exact bf16 rows, with the
// first positions that stay visible, on the tcgen05 tensor cores.
//
// Rows r = (query token, head) of a ragged batch; the token at position p sees the positions
// t <= p with t > p - window or t < sinks:
//   s_rt = scale * q_r . kv_t (576),  out_r = sum_t softmax_t(s_rt) kv_t[0:512],
//   lse_r = log sum_t exp(s_rt),
// and, joined with another attention's (out', lse') over other positions of the same rows
// (the layer's FP4 entries: one softmax over main KV and exact SWA rows, foosynaptic atlas
// "DeepSeek-V4.1-Flash 梗概", section 3.2, figure "异构 KV"):
//   lse = log(e^l + e^l'),  out = e^(l - lse) out + e^(l' - lse) out'.
//
// Tiles of 64 rows, one SM each: with transposed products the rows are the MMAs' columns, so that a single
// token of 64 heads wastes nothing (S^T [128 positions x 64 rows] = K . Q^T, O^T [4 x 128 channels x 64 rows] =
// V^T . P^T, both from one copy of the cache rows in shared memory: 128 x 1,152 B, with the queries' 72 KB
// all that an SM has).  A position is a tensor-memory lane: the softmax's maxima and sums go across lanes.
// The rows of a window of 128 are copied once for a run of tiles and then row by row (compact calls); longer
// windows go through the same memory block by block, and where there are few tiles their blocks are shared
// out among the SMs and merged.  (Many tokens over long windows: window_long.cu.)
//
// Roles of a CTA's 24 warps: 8 softmax, 8 outputs, one that issues the MMAs, 5 that copy a channel group
// each, one that plans.  They meet at mbarriers, group by group, so that the next tile's queries and rows come
// while this one's outputs are formed.
//
// P is rounded to bf16, as a product's operands have one type and the rows are bf16: outputs are off by 1.8-2.0e-3
// relative against 64 bits, of which their own rounding to bf16 is 1.65e-3.  (P in two parts would take the second products
// twice: 1,900 cycles more in the chain below.)  The largest weight of a row is 1, which bf16 holds exactly.
//
// What bounds it: the chain of a tile, about 8,000 cycles: scores 3,000 (2,100 of products at the rate at which
// shared memory feeds 64 columns, 5/6 of its bandwidth), softmax 2,200, outputs 1,900, and the hand-overs
// between.  Measured (GB300, 64 heads): whole prompts of 8,872 tokens, window 128, 260 us (0.71 of the copy rate
// on queries and outputs); 64 decode tokens joined with another attention 11.9 us, one token 9.4-10 us (launch,
// plan, copies, products, outputs one after the other); 8 tokens over 2,048 positions 18.5 us.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <atomic>
#include <mutex>
#include <type_traits>

#include "common.cuh"
#include "kernels.cuh"
#include "profile.cuh"
#include "tc.cuh"
#include "window.cuh"
#include "window_tiles.cuh"

namespace csa2 {

namespace {

constexpr int kRowWarps = 8;                         // softmax: lane quarter w % 4, half of the rows w / 4
constexpr int kOutWarp0 = kRowWarps, kOutWarps = 8;  // outputs: likewise
constexpr int kMmaWarp = kOutWarp0 + kOutWarps;
constexpr int kGroups = 5;                           // channel groups, a copying warp each: 4 x 128 latent, 64 rope
constexpr int kLoadWarp0 = kMmaWarp + 1;
constexpr int kPlanWarp = kLoadWarp0 + kGroups;      // (one more makes them a warpgroup)
constexpr int kWinThreads = (kMmaWarp + 8) * 32;
constexpr int kReaders = kPlanWarp;                  // warps that follow the plan

constexpr int kKReg = kWinPos * 128;                 // 64 channels of a block's positions: 16 KB
constexpr int kQReg = kWinRows * 128;                // 64 channels of a tile's rows: 8 KB
constexpr int kKBytes = 9 * kKReg, kQBytes = 9 * kQReg;
constexpr int kPHalf = 64 * 128;                     // P of 64 positions: 8 KB
constexpr int kQOff = kKBytes, kPOff = kQOff + kQBytes;
constexpr int kWinSmem = kPOff + kPHalf;
constexpr uint32_t kOCol = 64;                       // tensor memory: S^T 64 columns, O^T 4 x 64
constexpr uint32_t kCols = 512;
// Least blocks a tile's positions are split from, into three pieces or more; into two, as many as here.
// Measured, 64 heads, single tokens, split / whole: 1 sequence over 300, 500, 2,000 positions 13.8 / 15.0,
// 14.2 / 17.4, 15.8 / 50.2 us; 32 sequences 15.8 / 15.3, 16.2 / 17.7, 29.6 / 54.9; 70 sequences, in two pieces,
// 21.0 / 16.0, 22.1 / 19.5, 53.8 / 62.4 (1,000 positions, 8 or 9 blocks: 35.4 / 33.5).
__host__ __device__ inline bool splits(int64_t tiles, int64_t blocks, int64_t grid) {
  return blocks >= 3 && (3 * tiles <= grid || (2 * tiles <= grid && blocks >= 12));
}
constexpr int kPlanSlots = 3;

// One piece of a tile's work.  Its tokens see the positions lo .. last and the sinks before lo.
//   Compact calls: all of them fit a block of 128 places.  Position t has place t (t < sinks) or
//     sinks + (t - sinks) % (128 - sinks), so that the rows of consecutive tiles stay where they are and
//     a tile's new positions take the places of those that the window has left.
//   Other calls: whole pages of 64 positions, the sinks' (sp of them) and then the window's, two a block.
struct __align__(16) Piece {
  int n;                        // blocks, -1 behind the last piece
  int row, have;                // first row of q, rows (64, or what is left of the sequence)
  int seq;
  int lo, last;
  int pos, rem;                 // the first row's token position and head
  int blk, np;                  // first block; pages (sinks' and window's)
  int sp;                       // sinks' pages
  int unit;
  // compact calls have in place of the last four:
  __device__ int& fresh() { return blk; }            // first position that the tile before has not left in its place (0: none left)
  __device__ int& turn() { return np; }              // (last - sinks) % (128 - sinks), -1 where last < sinks
  __device__ int turn() const { return np; }
};

struct WinSmall {
  uint64_t q_full[2], q_empty[kGroups];              // queries and cache rows by channel group (full: latent, rope channels)
  uint64_t k_full[kGroups], k_empty[kGroups];
  uint64_t s_full, p_full, o_full, o_empty, drain;
  uint64_t stat_full, stat_empty;
  uint64_t meet[2], out_meet[2];                     // the four warps of a half
  uint64_t plan_full[kPlanSlots], plan_empty[kPlanSlots];
  uint32_t tmem_slot;
  int abort;
  int bad;                                           // q_start out of order
  uint32_t hidden;                                   // 1 + the last block in which hide_values has changed the places
  int tiles, tokens, most;                           // tiles of the call; most tokens of one, most positions that one sees
  Piece plan[kPlanSlots];
  __align__(16) float factor[kRowWarps][32];         // of a warp's weights, by row; at the end of a piece the first warp's of a half: reference
  __align__(16) float own[2][32], other[2][32];      // of the outputs of a half's rows, of the other attention's (its four warps write the same values)
  __align__(16) float top[4][kWinRows];              // maxima of a block by lane quarter; at the end of a piece the sums
};
static_assert(kWinSmem + (sizeof(WinSmall) + 1023) / 1024 * 1024 <= 232448, "shared memory; the dynamic part starts on a multiple of its alignment");

// Every wait is bounded (200 ms against microseconds) and cut short once another role has given up.
__device__ __forceinline__ bool wait_slow(WinSmall& sm, uint64_t* bar, uint32_t parity, uint8_t* ws) {
  uint64_t t0 = 0;
  for (uint32_t i = 1;; ++i) {
    if (tc::mbar_try_wait(bar, parity)) return true;
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
__device__ inline bool wait_warp(WinSmall& sm, uint64_t* bar, uint32_t parity, uint8_t* ws) {
  return __all_sync(0xFFFFFFFFu, tc::mbar_try_wait(bar, parity) || wait_slow(sm, bar, parity, ws));
}

__device__ inline void arrive(uint64_t* bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(tc::smem_u32(bar)) : "memory");
}
__device__ inline bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xFFFFFFFF;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}

struct WindowMaps {
  CUtensorMap q;
  CUtensorMap kv[7];                                 // boxes of 64 channels x 2^i rows
};

// Registers a thread of the calling warpgroup: what a role gives below the launch's 80, another takes.
template <int n>
__device__ inline void regs_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(n)); }
template <int n>
__device__ inline void regs_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(n)); }
constexpr int kWinRegs = 80, kRowRegs = 96, kOutRegs = 96, kMoveRegs = 48;
static_assert(kRowWarps * kRowRegs + kOutWarps * kOutRegs + 8 * kMoveRegs <= kWinRegs * (kWinThreads / 32),
              "a split above what was launched would wait for ever");

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

__device__ inline float max_over_warp(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
// 32 values a lane summed over the warp: lane l gets the sum of value l (31 shuffles).
__device__ inline float butterfly_sum(const float (&x)[32], int lane) {
  float v[16];
#pragma unroll
  for (int half = 16; half >= 1; half >>= 1) {
    const bool up = lane & half;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float lo = half == 16 ? x[i] : v[i], hi = half == 16 ? x[half + i] : v[half + i];
      const float keep = up ? hi : lo, give = up ? lo : hi;
      v[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, half);
    }
  }
  return v[0];
}

// Position of place e of block j of a piece (-1: none).
template <bool kCompact>
__device__ inline int place_position(const WindowArgs& a, const Piece& p, int j, int e) {
  if (kCompact) {
    if (e < a.sinks) return e <= p.last ? e : -1;
    int d = p.turn() - (e - a.sinks);                  // places from e on to the last position's
    if (d < 0) d += kWinPos - a.sinks;
    const int t = p.last - d;
    return p.turn() >= 0 && t >= max(p.lo, a.sinks) ? t : -1;
  }
  const int i = 2 * (p.blk + j) + (e >> 6);
  const int t = (i < p.sp ? i : p.lo / kPage + i - p.sp) * kPage + (e & (kPage - 1));
  return i < p.np && t <= p.last ? t : -1;
}

// For a position whose scores are no numbers, of cache row `row`, at place e, which the rows `see` of the warp's see.
// Its values, if an infinity or NaN is among them, become 0 where a row does not see them: the weight there is 0, and
// so must be 0 times its values.  Returns the rows that do see such values.  (Looked up in the cache, as the other
// half's warp may have hidden them.)
__device__ __noinline__ uint32_t hide_values(const WindowArgs& a, WinSmall& sm, uint8_t* base, uint32_t see, int row, int e, uint32_t block) {
  uint32_t lost = 0;
  if (see != 0u) {
    const uint4* at = reinterpret_cast<const uint4*>(a.kv + int64_t(row) * kDqk);
#pragma unroll 1
    for (int c = 0; c < 64; ++c)
      if (!bf16x8_finite(__ldg(at + c))) lost = see;
  }
  if (see == ~0u) return lost;
  bool whole = true;
#pragma unroll 1
  for (int c = 0; c < 64; ++c)
    whole = whole && bf16x8_finite(*reinterpret_cast<const uint4*>(base + (c >> 3) * kKReg + tc::sw128_offset(e, c & 7)));
  if (whole) return lost;
  *reinterpret_cast<volatile uint32_t*>(&sm.hidden) = block + 1;
#pragma unroll 1
  for (int c = 0; c < 64; ++c)
    *reinterpret_cast<uint4*>(base + (c >> 3) * kKReg + tc::sw128_offset(e, c & 7)) = make_uint4(0, 0, 0, 0);
  return lost;
}

// ---------------------------------------------------------------------------
// Plan: one warp walks the CTA's tiles and tells the others what to do, a few pieces ahead.
// ---------------------------------------------------------------------------
// A CTA's units of work (pieces of tiles): first, first + step, ... below units.
struct Span {
  int first, units, step, pieces;
};

// `q`: the first 32 sequences, loaded.
template <bool kCompact, bool kJoin>
__device__ inline void plan_role(const WindowArgs& a, WinSmall& sm, const Span& w, Sequences<kWinRows>& q, int lane) {
  q.count(lane);
  int was_seq = -1, was_last = 0;
  uint32_t k = 0;
  for (int u = w.first;; u += w.step, ++k) {
    Piece p = {};
    p.n = -1;
    if (u < w.units) {
      const int t = w.pieces == 1 ? u : u / w.pieces, s = u - t * w.pieces;
      const Tile tile = find_tile(a, q, t, lane);
      p.row = tile.row;
      p.have = tile.have;
      p.seq = tile.seq;
      p.pos = tile.pos;
      p.rem = tile.rem;
      p.last = tile.last;
      p.lo = tile.lo;
      p.unit = u;
      if (kCompact) {
        p.n = p.last >= 0;
        p.fresh() = p.seq == was_seq ? was_last + 1 : 0;
        p.turn() = p.last >= a.sinks ? (p.last - a.sinks) % (kWinPos - a.sinks) : -1;
        if (p.n > 0) {
          was_seq = p.seq;
          was_last = p.last;
        }
      } else {
        const TilePages pages = pages_of(a, p.lo, p.last);
        p.sp = pages.sinks;
        p.np = pages.all;
        const int nb = (p.np + 1) / 2;
        p.blk = w.pieces == 1 ? 0 : nb * s / w.pieces;
        p.n = w.pieces == 1 ? nb : nb * (s + 1) / w.pieces - p.blk;
      }
    }
    const uint32_t slot = k % kPlanSlots;
    if (!wait_warp(sm, &sm.plan_empty[slot], ((k / kPlanSlots) & 1) ^ 1, a.ws)) return;
    if (lane == 0) {
      sm.plan[slot] = p;
      arrive(&sm.plan_full[slot]);
      // the other attention's outputs of a later tile (one piece of memory) to L2
      if (kJoin && k > 0 && p.n >= 0 && p.have > 0 && w.pieces == 1)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;"
                     ::"l"(a.prev_out + int64_t(p.row) * kLatent), "r"(uint32_t(p.have * kLatent * 2)) : "memory");
    }
    __syncwarp();
    if (p.n < 0) return;
  }
}

// The next piece, for a converged warp; false behind the last.
__device__ inline bool next_piece(WinSmall& sm, uint32_t& k, int lane, uint8_t* ws, Piece& p) {
  const uint32_t slot = k % kPlanSlots;
  if (!wait_warp(sm, &sm.plan_full[slot], (k / kPlanSlots) & 1, ws)) return false;
  p = sm.plan[slot];
  __syncwarp();
  if (lane == 0) arrive(&sm.plan_empty[slot]);
  ++k;
  return p.n >= 0;
}

// The four warps of a half meet (bounded, unlike a hardware barrier), in two steps.
__device__ inline void meet_arrive(uint64_t* bar, int lane) {
  __syncwarp();
  if (lane == 0) arrive(bar);
}
__device__ inline bool meet_wait(WinSmall& sm, uint64_t* bar, uint32_t& n, uint8_t* ws) { return wait_warp(sm, bar, n++ & 1, ws); }

// ---------------------------------------------------------------------------
// Copies
// ---------------------------------------------------------------------------
// A box of 2^lg rows (lg -1: none) from cache row `row` on, for the places from `slot` on.
struct Box {
  int slot, row, lg;
};

// The positions first .. last (at most 128) of a sequence as boxes, one a lane: they are cut where
// pages end and at `turn` (where the places come round) into up to four runs, each of them a sum of
// powers of two; lane = 8 * run + 6 - power.  The place of a position is `shift` more than it before
// `turn`, `shift - back` from there on.
__device__ inline Box make_box(const WindowArgs& a, int seq, int first, int last, int turn, int shift, int back, int lane, bool& lost) {
  const int end = last + 1, c1 = min((first / kPage + 1) * kPage, end), c2 = min(c1 + kPage, end);
  const int c3 = min(max(turn, first), end);         // cuts: first, c1, c2, c3, end
  const int lo = min(c1, c3), hi = max(c2, c3), mid = c1 + c2 + c3 - lo - hi;
  const int r = lane >> 3, lg = 6 - (lane & 7);
  const int from = r == 0 ? first : r == 1 ? lo : r == 2 ? mid : hi, to = r == 0 ? lo : r == 1 ? mid : r == 2 ? hi : end;
  const int n = to - from;
  Box box = {0, 0, -1};
  if (n > 0 && lg >= 0 && (n >> lg & 1)) {
    const int t = from + (n & ~((2 << lg) - 1));     // behind the larger powers
    box.row = row_of(a, seq, t);
    box.slot = t + shift - (t >= turn ? back : 0);
    if (box.row >= 0) box.lg = lg;
    else lost = true;
  }
  return box;
}

// Where P of a block's first and last 64 positions goes: over the block's rope channels, which only
// the scores need; in a compact call, whose rows stay, into a place of its own and over the queries'
// rope channels, which no other block of the tile needs.
template <bool kCompact>
__device__ inline uint32_t p_offset(int half) {
  return kCompact ? (half == 0 ? kPOff : kQOff + 8 * kQReg) : 8 * kKReg + half * kPHalf;
}

// Copies channel group g of the queries and the cache rows.  (One warp for all groups takes 650 cycles
// for the few copies of one: what it waits for is the issue, not the copies.)
//
// A few rows are fetched into registers while their places are still in use, and stored when they are
// free: a copy by TMA from then on takes 700 cycles of the chain.  More rows go as boxes.
constexpr int kFewRows = 4, kFewChunks = kFewRows * 16 / 32;

template <bool kCompact>
__device__ inline void load_role(const WindowArgs& a, WinSmall& sm, uint8_t* base, int g, int lane, const WindowMaps& m) {
  const int regions = g < 4 ? 2 : 1, shift = g < 4 ? 4 : 3;            // (16-byte pieces of a row: 1 << shift)
  uint64_t* const q_full = &sm.q_full[g == 4];
  Piece p;
  uint32_t nu = 0, nq = 0, nk = 0;
  while (next_piece(sm, nu, lane, a.ws, p)) {
    if (p.n == 0) continue;
    Box box[2];                                      // the window's, the sinks'
    int rows = 0;
    bool lost = false, few = false;
    uint4 v[kFewChunks];
    uint32_t to[kFewChunks];                         // offsets in the block, ~0: none
    const auto whole = [&]() {
      const int first = max(p.lo, a.sinks), c = kWinPos - a.sinks;
      // the last position has place sinks + turn(): `turn()` positions before it is the first place
      box[0] = make_box(a, p.seq, first, max(p.last, first - 1), p.last - p.turn(), a.sinks + p.turn() - p.last + c, c, lane, lost);
      box[1].lg = -1;
      if (a.sinks > 0) box[1] = make_box(a, p.seq, 0, min(a.sinks - 1, p.last), 1 << 30, 0, 0, lane, lost);
      rows = __reduce_add_sync(0xFFFFFFFFu, (box[0].lg >= 0 ? 1 << box[0].lg : 0) + (box[1].lg >= 0 ? 1 << box[1].lg : 0));
    };
    if (kCompact) {
      few = p.fresh() > 0 && p.last - p.fresh() < kFewRows;
      if (few) {
#pragma unroll
        for (int i = 0; i < kFewChunks; ++i) {
          const int c = lane + 32 * i, t = p.fresh() + (c >> shift), r = 2 * g + (c >> 3 & (regions - 1));
          to[i] = ~0u;
          if (t > p.last) continue;
          const int row = row_of(a, p.seq, t);
          if (row < 0) {
            lost = true;
            continue;
          }
          int d = p.turn() - (p.last - t);
          if (d < 0) d += kWinPos - a.sinks;
          to[i] = r * kKReg + tc::sw128_offset(t < a.sinks ? t : a.sinks + d, c & 7);
          v[i] = __ldg(reinterpret_cast<const uint4*>(a.kv + int64_t(row) * kDqk + 64 * r) + (c & 7));
        }
      } else {
        whole();
      }
    }
    if (!wait_warp(sm, &sm.q_empty[g], (nq++ & 1) ^ 1, a.ws)) return;
    if (lane == 0) {
      tc::mbar_expect_tx(q_full, uint32_t(regions * kQReg));
#pragma unroll 1
      for (int r = 2 * g; r < 2 * g + regions; ++r)
        tc::tma_load_2d(&m.q, base + kQOff + r * kQReg, 64 * r, p.row, q_full);
      // the next tile's queries are the next rows: to L2
      const int64_t more = min64(kWinRows, int64_t(a.total_q) * a.d.heads - p.row - kWinRows);
      if (kCompact && g == 4 && more > 0)
        asm volatile("cp.async.bulk.prefetch.L2.global [%0], %1;"
                     ::"l"(a.q + (int64_t(p.row) + kWinRows) * kDqk), "r"(uint32_t(more * kDqk * 2)) : "memory");
    }
    __syncwarp();
    if (kCompact) {
      if (!wait_warp(sm, &sm.k_empty[g], (nk & 1) ^ 1, a.ws)) return;
      // values of the tile before may have been taken out of their places
      if (few && g < 4 && nk > 0 && *reinterpret_cast<volatile uint32_t*>(&sm.hidden) == nk) {
        few = false;
        whole();
      }
      if (few) {
#pragma unroll
        for (int i = 0; i < kFewChunks; ++i)
          if (to[i] != ~0u) *reinterpret_cast<uint4*>(base + to[i]) = v[i];
        tc::fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) arrive(&sm.k_full[g]);
      } else {
        if (lane == 0) tc::mbar_expect_tx(&sm.k_full[g], uint32_t(regions * rows * 128));
        __syncwarp();
#pragma unroll 1
        for (int part = 0; part < 2; ++part) {
          const Box b = part == 0 ? box[0] : box[1];
          if (b.lg >= 0)
#pragma unroll 1
            for (int r = 2 * g; r < 2 * g + regions; ++r)
              tc::tma_load_2d(&m.kv[b.lg], base + r * kKReg + b.slot * 128, 64 * r, b.row, &sm.k_full[g]);
        }
      }
      ++nk;
    } else {
#pragma unroll 1
      for (int j = 0; j < p.n; ++j, ++nk) {
        // lane: half of the block (lane & 1), region
        const int h = lane & 1, r = 2 * g + (lane >> 1), t = place_position<false>(a, p, j, kPage * h);
        const int row = t >= 0 ? row_of(a, p.seq, t) : -1;
        lost = lost || (t >= 0 && row < 0);
        const int halves = __popc(__ballot_sync(0xFFFFFFFFu, row >= 0) & 3u);
        if (!wait_warp(sm, &sm.k_empty[g], (nk & 1) ^ 1, a.ws)) return;
        if (lane == 0) tc::mbar_expect_tx(&sm.k_full[g], uint32_t(regions * halves * (kKReg / 2)));
        __syncwarp();
        if (lane < 2 * regions && row >= 0)
          tc::tma_load_2d(&m.kv[6], base + r * kKReg + h * (kKReg / 2), 64 * r, row, &sm.k_full[g]);
      }
    }
    if (g == 0 && lost) raise_err(a.ws, CSA2_DEV_PAGE_ID);
  }
}

// ---------------------------------------------------------------------------
// Products
// ---------------------------------------------------------------------------
// tc::mma_bf16 with descriptors as low words (address, leading offset); their high words are one
// constant: rows of 8 are 1,024 bytes apart, 128-byte swizzle.  Called by the whole warp, done by
// the thread with `leader`: what the operands are formed from is then the same for the warp to the
// compiler, which keeps it in uniform registers.
__device__ inline void mma_lo(uint32_t leader, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, uint32_t add) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 x, y;\n\t"
      "mov.b64 x, {%1, %5};\n\tmov.b64 y, {%2, %5};\n\t"
      "setp.ne.b32 p, %6, 0;\n\tsetp.ne.b32 q, %4, 0;\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}"
      ::"r"(d), "r"(a), "r"(b), "r"(idesc), "r"(leader), "n"((1024 >> 4) | 1 << 14 | 2 << 29), "r"(add)
      : "memory");
}
__device__ inline void commit_lo(uint32_t leader, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}"
      ::"r"(tc::smem_u32(bar)), "r"(leader) : "memory");
}

template <bool kCompact>
__device__ inline void mma_role(const WindowArgs& a, WinSmall& sm, uint8_t* base, int lane, uint32_t tmem) {
  constexpr uint32_t id_s = tc::idesc_bf16(kWinPos, kWinRows, 0, 0);
  constexpr uint32_t id_o = tc::idesc_bf16(kWinPos, kWinRows, 1, 1);
  const uint32_t at = tc::smem_u32(base);
  const uint32_t k_lo = uint32_t(tc::smem_desc(at, 16, 1024, 2)), q_lo = uint32_t(tc::smem_desc(at + kQOff, 16, 1024, 2));
  const uint32_t v_lo = uint32_t(tc::smem_desc(at, kKReg, 1024, 2));
  const uint32_t p_lo[2] = {uint32_t(tc::smem_desc(at + p_offset<kCompact>(0), kPHalf, 1024, 2)),
                            uint32_t(tc::smem_desc(at + p_offset<kCompact>(1), kPHalf, 1024, 2))};
  const uint32_t leader = elect_one();
  Piece p;
  uint32_t nu = 0, nq = 0, nk = 0;
  bool more = next_piece(sm, nu, lane, a.ws, p);
  while (more) {
    const int n = p.n;
    if (n == 0) more = next_piece(sm, nu, lane, a.ws, p);
#pragma unroll 1
    for (int j = 0; j < n; ++j, ++nk) {
      const bool end = j == n - 1;
#pragma unroll 1
      for (int t = 0; t < 9; ++t) {                  // regions of 64 channels
        const int g = t >> 1;
        if ((t & 1) == 0) {
          if (j == 0 && (t == 0 || t == 8) && !wait_warp(sm, &sm.q_full[t >> 3], nq & 1, a.ws)) return;
          if (!wait_warp(sm, &sm.k_full[g], nk & 1, a.ws)) return;
          tc::tc_fence_after_sync();
        }
        const uint32_t x = k_lo + t * (kKReg >> 4), y = q_lo + t * (kQReg >> 4);
        mma_lo(leader, tmem, x, y, id_s, t);
#pragma unroll
        for (int k = 1; k < 4; ++k) mma_lo(leader, tmem, x + k * (32 >> 4), y + k * (32 >> 4), id_s, 1);
        // the next tile's queries come group by group (P goes over the rope channels in a compact call)
        if (end && ((t & 1) || (t == 8 && !kCompact))) commit_lo(leader, &sm.q_empty[g]);
      }
      commit_lo(leader, &sm.s_full);
      if (kCompact) commit_lo(leader, &sm.k_empty[4]);
      if (end) more = next_piece(sm, nu, lane, a.ws, p);                    // ahead: nothing between this piece's last product and its scores
      if (!wait_warp(sm, &sm.p_full, nk & 1, a.ws)) return;
      if (j == 0 && !wait_warp(sm, &sm.o_empty, (nq & 1) ^ 1, a.ws)) return;
      tc::tc_fence_after_sync();
#pragma unroll 1
      for (int mt = 0; mt < 4; ++mt) {
        const uint32_t vs = v_lo + mt * (2 * kKReg >> 4), d = tmem + kOCol + 64 * mt;
        mma_lo(leader, d, vs, p_lo[0], id_o, j);
#pragma unroll
        for (int k = 1; k < 8; ++k) mma_lo(leader, d, vs + (k * 2048 >> 4), p_lo[k >> 2] + ((k & 3) * 2048 >> 4), id_o, 1);
        commit_lo(leader, &sm.k_empty[mt]);
      }
      commit_lo(leader, kCompact ? &sm.q_empty[4] : &sm.k_empty[4]);
      if (end) commit_lo(leader, &sm.o_full);
    }
    if (n > 0) ++nq;
  }
}

// ---------------------------------------------------------------------------
// Softmax
// ---------------------------------------------------------------------------
// Which of the warp's 32 rows see position t (bit i: row i), and whether all 64 rows of the tile do, of which
// `before` come before the warp's.  `pos`, `rem`: the first row's token position and head; tokens are `heads` rows
// each.  (Rows that do not exist take part as if they did: nothing of theirs is used.)
__device__ inline uint32_t seen_by(const WindowArgs& a, int t, int pos, int rem, int before, bool& all) {
  all = false;
  if (t < 0) return 0u;
  // rows from the first of token t on, to the last of token t + window - 1 (any, for a sink)
  const int lo = (t - pos) * a.d.heads - rem, hi = t < a.sinks ? kWinRows : lo + a.window * a.d.heads;
  all = lo <= -before && hi >= kWinRows - before;
  if (lo >= 32 || hi <= 0) return 0u;
  const uint32_t from = lo <= 0 ? ~0u : ~0u << lo;
  return hi >= 32 ? from : from & ((1u << hi) - 1u);
}

// The scores of rows that do not see the lane's position become -inf.  `row`: its cache row.
__device__ inline void mask_scores(const WindowArgs& a, WinSmall& sm, uint8_t* base, float (&x)[32], uint32_t see, int row, int e,
                                   uint32_t block) {
  float any = 0.0f;                                  // 0, or NaN where a score is no number
#pragma unroll
  for (int i = 0; i < 32; ++i) {
    any = fmaf(x[i], 0.0f, any);
    x[i] = see >> i & 1 ? x[i] : -INFINITY;
  }
  if (any == 0.0f) return;
  // An infinity or NaN: values that are no numbers go where a row does not see them, and the rows that do become NaN.
  // (Of values that are numbers a score of -inf, by the rotary channels alone, is weight 0, and one of +inf makes NaN
  // by itself.)
  const uint32_t lost = hide_values(a, sm, base, see, row, e, block);
#pragma unroll
  for (int i = 0; i < 32; ++i) x[i] = lost >> i & 1 ? NAN : x[i];
}

// Two scores as weights under their rows' maxima (a pair, low half first).
__device__ inline void weights2(float& x, float& y, uint64_t m, float c) {
  asm("{\n\t.reg .b64 v, k;\n\t"
      "mov.b64 v, {%0, %1};\n\tmov.b64 k, {%3, %3};\n\t"
      "fma.rn.f32x2 v, %2, k, v;\n\tmov.b64 k, {%4, %4};\n\tmul.rn.f32x2 v, v, k;\n\tmov.b64 {%0, %1}, v;\n\t}"
      : "+f"(x), "+f"(y) : "l"(m), "f"(-1.0f), "f"(c));
  x = ex2(x);
  y = ex2(y);
}

// Softmax over a block's positions (tensor-memory lanes).  Warp rw has the lanes 32 (rw % 4) .. + 31
// and the rows 32 (rw / 4) .. + 31; lane i keeps the state of row i of these (alike in the four warps
// of a half, but for the sum, which is of its own lanes).  A warp's weights are formed under its own
// maxima while it waits for the other warps', and then brought to the common reference.
// Maxima and references are scores, not yet times `c`: the difference of two scores is exact where it matters, and 0
// for the largest, whatever their size.  (c x less a rounded c x is not: half a unit of it, past any weight from 2^31 on.)
constexpr float kNone = -3.402823466e38f;            // maximum of no scores
template <bool kCompact>
__device__ inline void row_role(const WindowArgs& a, WinSmall& sm, uint8_t* base, int rw, int lane, uint32_t tmem) {
  const int quarter = rw & 3, half = rw >> 2, e = 32 * quarter + lane;
  const uint32_t lanes = tmem + (uint32_t(32 * quarter) << 16) + uint32_t(32 * half);
  const float c = score_to_log2(a);
  uint8_t* const p_at = base + p_offset<kCompact>(quarter >> 1);
  Piece p;
  uint32_t nu = 0, nk = 0, nm = 0;
  while (next_piece(sm, nu, lane, a.ws, p)) {
    // the warp's first row: its token's position, its head
    const int r0 = p.rem + 32 * half, tok = over_heads(a, r0), rem = r0 - tok * a.d.heads, pos = p.pos + tok;
    float ref = kNone, sum = 0.0f;
    int t, row;
    const auto look = [&](int j) {
      t = place_position<kCompact>(a, p, j, e);
      row = t >= 0 ? row_of(a, p.seq, t) : -1;
    };
    look(0);
    // the last piece's sums, which stand where the maxima go, have been read
    if (!wait_warp(sm, &sm.stat_empty, nu & 1, a.ws)) return;
#pragma unroll 1
    for (int j = 0; j < p.n; ++j, ++nk) {
      if (row < 0) t = -1;
      bool all;
      const uint32_t see = seen_by(a, t, pos, rem, 32 * half, all);
      const bool edge = !__all_sync(0xFFFFFFFFu, all);     // the same for both halves: what one hides, the other must know of
      if (!wait_warp(sm, &sm.s_full, nk & 1, a.ws)) return;
      tc::tc_fence_after_sync();
      float x[32];
      tc::tmem_ld32(lanes, x);
      if (a.scale < 0.0f) {
#pragma unroll
        for (int i = 0; i < 32; ++i) x[i] = -x[i];
      }
      if (edge) {
        mask_scores(a, sm, base, x, see, row, e, nk);
        __syncwarp();
      }
      float top = kNone;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float m = max_over_warp(x[i]);
        if (lane == i) top = m;
      }
      top = fmaxf(top, kNone);
      sm.top[quarter][32 * half + lane] = top;       // (read before the other warps' P, which these scores came after)
      meet_arrive(&sm.meet[half], lane);
#pragma unroll
      for (int i4 = 0; i4 < 8; ++i4) {
        const ulonglong2 m = reinterpret_cast<const ulonglong2*>(&sm.top[quarter][32 * half])[i4];
        weights2(x[4 * i4], x[4 * i4 + 1], m.x, c);
        weights2(x[4 * i4 + 2], x[4 * i4 + 3], m.y, c);
      }
      if (!meet_wait(sm, &sm.meet[half], nm, a.ws)) return;
      float most = top;
#pragma unroll
      for (int k = 0; k < 4; ++k) most = fmaxf(most, sm.top[k][32 * half + lane]);
      float alpha = 1.0f;
      if ((most - ref) * c > kWinSlack || (ref == kNone && most > kNone)) {
        if (ref != kNone) alpha = ex2((ref - most) * c);
        ref = most;                                  // the largest weight is 1, which bf16 holds exactly
      }
      sm.factor[rw][lane] = ex2((top - ref) * c);
      __syncwarp();
      if (__any_sync(0xFFFFFFFFu, alpha != 1.0f)) {
        // the outputs so far to the new reference (this block's scores came after the last product: the
        // copies that they needed waited for it)
        sum *= alpha;
#pragma unroll 1
        for (int col = 0; col < 32; col += 8)
#pragma unroll 1
          for (int mt = 0; mt < 4; ++mt) {
            float o[8];
            tc::tmem_ld8(lanes + kOCol + 64 * mt + col, o);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] *= __shfl_sync(0xFFFFFFFFu, alpha, col + i);
            tc::tmem_st8(lanes + kOCol + 64 * mt + col, o);
          }
      }
#pragma unroll
      for (int i8 = 0; i8 < 4; ++i8) {
        uint32_t pk[4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float4 f = reinterpret_cast<const float4*>(sm.factor[rw])[2 * i8 + k];
          const int i = 8 * i8 + 4 * k;
          x[i] *= f.x;
          x[i + 1] *= f.y;
          x[i + 2] *= f.z;
          x[i + 3] *= f.w;
          pk[2 * k] = bf16x2_rn(x[i], x[i + 1]);
          pk[2 * k + 1] = bf16x2_rn(x[i + 2], x[i + 3]);
        }
        *reinterpret_cast<uint4*>(p_at + tc::sw128_offset(e & 63, 4 * half + i8)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
      }
      tc::fence_proxy_async_smem();
      tc::tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) arrive(&sm.p_full);
      sum += butterfly_sum(x, lane);
      if (j + 1 < p.n) look(j + 1);
    }
    // all have read the maxima: the sums go in their place
    meet_arrive(&sm.meet[half], lane);
    if (!meet_wait(sm, &sm.meet[half], nm, a.ws)) return;
    sm.top[quarter][32 * half + lane] = sum;
    if (quarter == 0) sm.factor[rw][lane] = ref * c;
    __syncwarp();
    if (lane == 0) arrive(&sm.stat_full);
  }
}

// ---------------------------------------------------------------------------
// Outputs, from tensor memory: lanes are channels, columns are rows.  The products take five sixths of
// shared memory's bandwidth, which shuffles share, so values go out as they lie, 64 bytes of a row an
// instruction.  (Eight channels of four rows a lane, by 32 shuffles for 32 x 32 values: as many lines
// for the stores, and the shuffles beside them.)
// ---------------------------------------------------------------------------
__device__ inline void load_factors(const float (&own)[32], float (&f)[32]) {
#pragma unroll
  for (int i4 = 0; i4 < 8; ++i4) {
    const float4 v = reinterpret_cast<const float4*>(own)[i4];
    f[4 * i4] = v.x;
    f[4 * i4 + 1] = v.y;
    f[4 * i4 + 2] = v.z;
    f[4 * i4 + 3] = v.w;
  }
}
template <bool kJoin>
__device__ inline void out_role(const WindowArgs& a, WinSmall& sm, int pieces, int ow, int lane, uint32_t tmem) {
  const int quarter = ow & 3, half = ow >> 2, e = 32 * quarter + lane;
  const uint32_t lanes = tmem + (uint32_t(32 * quarter) << 16) + uint32_t(32 * half);
  const bool whole = pieces == 1, join = kJoin && whole;
  Piece p;
  uint32_t nu = 0, nq = 0, nm = 0;
  while (next_piece(sm, nu, lane, a.ws, p)) {
    const int have = p.have - 32 * half;             // rows of this half
    const int64_t row0 = int64_t(p.row) + 32 * half;
    float prev = -INFINITY;
    if (join && lane < have) prev = a.prev_lse[row0 + lane];
    // Joined outputs go by pairs of lanes: of rows 2 i and 2 i + 1 the even lane takes both channels of the one,
    // the odd lane both of the other, so that loads and stores are 32 bits.  The other attention's come a step
    // ahead, the first while the scores and products are formed (but for rows of which it has seen nothing: they
    // may be anything).  4,000 tokens of 16 heads, joined: 61 us (41 alone); with values of 16 bits 66, and all
    // fetched ahead, which leaves too few registers to be on their way together, 127.
    const int odd = lane & 1;
    uint32_t raw[kJoin ? 16 : 1], use = 0;
    const uint32_t* src = nullptr;
    const auto fetch = [&]() {
#pragma unroll
      for (int i = 0; i < 16; ++i) raw[kJoin ? i : 0] = use >> (2 * i) & 1 ? src[i * kLatent] : 0;
    };
    if constexpr (kJoin) {
      use = __ballot_sync(0xFFFFFFFFu, prev != -INFINITY) >> odd;
      src = reinterpret_cast<const uint32_t*>(a.prev_out + (row0 + odd) * kLatent + (e - odd));
      fetch();
    }
    if (!wait_warp(sm, &sm.stat_full, (nu - 1) & 1, a.ws)) return;
    float total = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) total += sm.top[k][32 * half + lane];
    const float ref = sm.factor[4 * half][lane];
    float own = total != 0.0f ? 1.0f / total : 0.0f, other = 0.0f;
    float lse = total != 0.0f ? (ref + log2f(total)) * 0.6931471805599453f : -INFINITY;
    if (join && prev != -INFINITY) {
      const float most = fmaxf(lse, prev), x0 = expf(lse - most), x1 = expf(prev - most);
      own *= x0 / (x0 + x1);
      other = x1 / (x0 + x1);
      lse = most + logf(x0 + x1);
    }
    // all four have read prev_lse (lse may be the same place) and the last piece's factors
    meet_arrive(&sm.out_meet[half], lane);
    if (!meet_wait(sm, &sm.out_meet[half], nm, a.ws)) return;
    sm.own[half][lane] = own;
    if (kJoin) sm.other[half][lane] = other;
    __syncwarp();
    if (lane == 0) arrive(&sm.stat_empty);
    float f[kJoin ? 1 : 32];
    if constexpr (!kJoin) load_factors(sm.own[half], f);
    if (p.n > 0) {
      if (!wait_warp(sm, &sm.o_full, nq & 1, a.ws)) return;
      tc::tc_fence_after_sync();
    }
    if (whole) {
      if (quarter == 0 && lane < have) a.lse[row0 + lane] = lse;
      uint16_t* dst = a.out + row0 * kLatent + e;
      if constexpr (kJoin) {
        uint32_t* to = reinterpret_cast<uint32_t*>(dst + (odd ? kLatent - 1 : 0));
        float fo[16], go[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          fo[i] = sm.own[half][2 * i + odd];
          go[i] = sm.other[half][2 * i + odd];
        }
#pragma unroll 1
        for (int mt = 0; mt < 4; ++mt, to += 64) {
          uint32_t old[16];
#pragma unroll
          for (int i = 0; i < 16; ++i) old[i] = raw[i];
          src += 64;
          if (mt < 3) fetch();
#pragma unroll
          for (int i8 = 0; i8 < 32; i8 += 16) {
            float o[16];
            if (p.n > 0) {
              tc::tmem_ld16(lanes + kOCol + 64 * mt + i8, o);
            } else {
#pragma unroll
              for (int i = 0; i < 16; ++i) o[i] = 0.0f;
            }
#pragma unroll
            for (int i = 0; i < 16; i += 2) {
              const float got = __shfl_xor_sync(0xFFFFFFFFu, odd ? o[i] : o[i + 1], 1);
              const float f = fo[(i8 + i) / 2], g = go[(i8 + i) / 2];
              const uint32_t w = old[(i8 + i) / 2];
              const float x = fmaf(g, __uint_as_float(w << 16), (odd ? got : o[i]) * f);
              const float y = fmaf(g, __uint_as_float(w & 0xFFFF0000u), (odd ? o[i + 1] : got) * f);
              if (i8 + i + odd < have) to[(i8 + i) / 2 * kLatent] = bf16x2_rn(x, y);
            }
          }
        }
      } else {
#pragma unroll 1
        for (int mt = 0; mt < 4; ++mt, dst += 128) {
          float o[32];
          if (p.n > 0) {
            tc::tmem_ld32(lanes + kOCol + 64 * mt, o);
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i) o[i] = 0.0f;
          }
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] *= f[i];
          if (have >= 32) {
#pragma unroll
            for (int i = 0; i < 32; i += 2) {
              const uint32_t y = bf16x2_rn(o[i], o[i + 1]);
              dst[i * kLatent] = uint16_t(y);
              dst[(i + 1) * kLatent] = uint16_t(y >> 16);
            }
          } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (i < have) dst[i * kLatent] = uint16_t(bf16x2_rn(o[i], 0.0f));
          }
        }
      }
    } else {
      // a piece: its own softmax in fp32, for the merge
      const int u = p.unit;
      if (quarter == 0) {
        a.part_lse[u * kWinRows + 32 * half + lane] = lse;
        if (u % pieces == 0 && ow == 0 && lane == 0) a.tiles[u / pieces] = make_int2(p.row, p.have);
      }
      if (p.n > 0) {
#pragma unroll 1
        for (int mt = 0; mt < 4; ++mt) {
          float o[32];
          tc::tmem_ld32(lanes + kOCol + 64 * mt, o);
          float* dst = a.part_o + (int64_t(u) * kWinRows + 32 * half) * kLatent + 128 * mt + e;
#pragma unroll
          for (int i = 0; i < 32; ++i)
            if (i < have) dst[i * kLatent] = o[i] * sm.own[half][i];
        }
      }
    }
    if (p.n > 0) {
      tc::tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) arrive(&sm.o_empty);
      ++nq;
    }
  }
}

template <bool kJoin>
__global__ void __launch_bounds__(kWinThreads, 1)
    window_kernel(const __grid_constant__ WindowArgs a, const __grid_constant__ WindowMaps m) {
  extern __shared__ __align__(1024) uint8_t base[];  // 1024-byte aligned: checked below
  __shared__ WinSmall sm;
  const int tid = threadIdx.x, lane = tid & 31, wid = __shfl_sync(0xFFFFFFFFu, tid >> 5, 0);   // the same for the warp, to the compiler too
  if (tc::smem_u32(base) & 1023u) {                  // never, as laid out
    pdl_wait();
    if (tid == 0) raise_err(a.ws, CSA2_DEV_TIMEOUT);
    return;
  }
  if (wid == kMmaWarp) tc::tmem_alloc(&sm.tmem_slot, kCols);
  if (tid == 0) {
    tc::mbar_init(&sm.q_full[0], kGroups - 1);
    tc::mbar_init(&sm.q_full[1], 1);
    for (int g = 0; g < kGroups; ++g) {
      tc::mbar_init(&sm.q_empty[g], 1);
      tc::mbar_init(&sm.k_full[g], 1);
      tc::mbar_init(&sm.k_empty[g], 1);
    }
    tc::mbar_init(&sm.s_full, 1);
    tc::mbar_init(&sm.p_full, kRowWarps);
    tc::mbar_init(&sm.o_full, 1);
    tc::mbar_init(&sm.o_empty, kOutWarps);
    tc::mbar_init(&sm.drain, 1);
    tc::mbar_init(&sm.stat_full, kRowWarps);
    tc::mbar_init(&sm.stat_empty, kOutWarps);
    for (int i = 0; i < 2; ++i) {
      tc::mbar_init(&sm.meet[i], 4);
      tc::mbar_init(&sm.out_meet[i], 4);
    }
    for (int i = 0; i < kPlanSlots; ++i) {
      tc::mbar_init(&sm.plan_full[i], 1);
      tc::mbar_init(&sm.plan_empty[i], kReaders);
    }
    tc::fence_mbar_init();
    sm.abort = 0;
    sm.bad = 0;
    sm.hidden = 0;
    sm.tiles = 0;
    sm.tokens = 0;
    sm.most = 0;
  }
  // Places that no row is copied to (short contexts, a last block of one page) hold zeros: what else the
  // memory held might be no numbers, which costs a look through them (decode steps over windows of 300 to 400
  // positions 19 us in place of 14, 4 tokens over 64 positions 28 in place of 16).
  for (int i = tid; i < kKBytes / 16; i += kWinThreads) reinterpret_cast<uint4*>(base)[i] = make_uint4(0, 0, 0, 0);
  tc::fence_proxy_async_smem();
  pdl_wait();
  pdl_launch_dependents();
  __syncthreads();
  Sequences<kWinRows> first = {0, 0, 0, 0, 0, 0};
  if (wid == kPlanWarp) first.load(a, lane);         // on their way while the tiles are counted
  // Count the tiles, and what most their rows see.  Starts out of order are reported and the call
  // writes nothing.
  {
    const bool paged = a.page_table != nullptr;
    const int H = a.d.heads, span = tile_tokens(H, kWinRows);
    int tiles = 0, tokens = 0, most = 0;
    bool bad = false;
    for (int b = tid; b < a.batch; b += kWinThreads) {
      const int s0 = __ldg(a.q_start + b), s1 = __ldg(a.q_start + b + 1);
      if (s0 < 0 || s1 < s0 || s1 > a.total_q) {
        bad = true;
        continue;
      }
      if (blockIdx.x == 0) check_ctx(__ldg(a.ctx_len + b), a.d, paged, a.ws);
      tiles += tiles_of<kWinRows>(a, s1 - s0);
      tokens = max(tokens, min(span, s1 - s0));
      if (a.may_split && s1 > s0) most = max(most, int(min64(context(a, b), int64_t(a.window) + min(span, s1 - s0) - 1 + a.sinks)));
    }
    if (bad) atomicOr(&sm.bad, 1);
    tiles = __reduce_add_sync(0xFFFFFFFFu, tiles);
    tokens = __reduce_max_sync(0xFFFFFFFFu, tokens);
    most = __reduce_max_sync(0xFFFFFFFFu, most);
    if (lane == 0 && tiles > 0) {
      atomicAdd(&sm.tiles, tiles);
      atomicMax(&sm.tokens, tokens);
      if (a.may_split) atomicMax(&sm.most, most);
    }
  }
  tc::tc_fence_before_sync();
  __syncthreads();
  tc::tc_fence_after_sync();
  const uint32_t tmem = sm.tmem_slot;
  const int tiles = sm.bad ? 0 : sm.tiles, grid = gridDim.x;
  // Compact where a tile's positions fit a block.  As whole pages they might be three, in two blocks (window
  // 128, 64 heads: 8,000 tokens of prompts 233 us compact, 384 by pages; 64 sequences of 4 tokens 16.9, 20.9),
  // unless they are no more than a page and one: then one block by pages, too, which is copied without a look
  // at each position (window 64: 244, 229; 16.7, 14.3).
  const int64_t seen = int64_t(a.window) + sm.tokens - 1;
  const bool compact = seen + a.sinks <= kWinPos && (a.sinks > 0 || seen > kPage + 1);
  Span w;
  w.pieces = 1;
  if (compact) {
    // consecutive tiles share most of their rows
    w.first = int(int64_t(tiles) * blockIdx.x / grid);
    w.units = int(int64_t(tiles) * (blockIdx.x + 1) / grid);
    w.step = 1;
  } else {
    const int blocks = (sm.most + kWinPos - 1) / kWinPos;
    if (a.may_split && tiles > 0 && splits(tiles, blocks, grid)) w.pieces = min(grid / tiles, blocks);
    w.first = blockIdx.x;
    w.units = tiles * w.pieces;
    w.step = grid;
  }
  if (blockIdx.x == 0 && tid == 0) {
    if (sm.bad) raise_err(a.ws, CSA2_DEV_Q_START);
    if (a.may_split) {
      a.head[0] = tiles;
      a.head[1] = w.pieces;
    }
  }
  if (wid < kRowWarps) {
    regs_up<kRowRegs>();
    if (compact) row_role<true>(a, sm, base, wid, lane, tmem);
    else row_role<false>(a, sm, base, wid, lane, tmem);
  } else if (wid < kMmaWarp) {
    regs_up<kOutRegs>();
    out_role<kJoin>(a, sm, w.pieces, wid - kOutWarp0, lane, tmem);
  } else {
    regs_down<kMoveRegs>();
    if (wid == kMmaWarp) {
      if (compact) mma_role<true>(a, sm, base, lane, tmem);
      else mma_role<false>(a, sm, base, lane, tmem);
    } else if (wid < kPlanWarp) {
      if (compact) load_role<true>(a, sm, base, wid - kLoadWarp0, lane, m);
      else load_role<false>(a, sm, base, wid - kLoadWarp0, lane, m);
    } else if (wid == kPlanWarp) {
      if (compact) plan_role<true, kJoin>(a, sm, w, first, lane);
      else plan_role<false, kJoin>(a, sm, w, first, lane);
    }
  }
  // the thread that issued the MMAs sees them done (they are, unless a wait gave up)
  __syncwarp();
  if (wid == kMmaWarp) {
    if (elect_one()) {
      tc::mma_commit(&sm.drain);
      wait_slow(sm, &sm.drain, 0, a.ws);
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
  if (wid == kMmaWarp) tc::tmem_dealloc(tmem, kCols);
}

// ---------------------------------------------------------------------------
// Merge of the pieces of split tiles, and the join.  A CTA has four rows of a tile.
// ---------------------------------------------------------------------------
constexpr int kMergeRows = 4, kMergeThreads = kMergeRows * kLatent / 8;

__global__ void __launch_bounds__(kMergeThreads) window_merge_kernel(const __grid_constant__ WindowArgs a) {
  __shared__ float s_part[kMergeRows][kWinMaxCtas];
  pdl_launch_dependents();
  const int tiles = __ldg(a.head), n = __ldg(a.head + 1), t = blockIdx.y;
  if (n <= 1 || t >= tiles) return;
  const int2 tile = __ldg(a.tiles + t);
  const int y = threadIdx.x / (kLatent / 8), r = blockIdx.x * kMergeRows + y, x = threadIdx.x % (kLatent / 8);
  const bool have = r < tile.y;
  const int64_t row = int64_t(tile.x) + r;
  if (blockIdx.x * kMergeRows >= tile.y) return;
  // weights of the pieces and of the other attention, by row
  for (int s = x; s < n; s += kLatent / 8) s_part[y][s] = __ldg(a.part_lse + (t * n + s) * kWinRows + r);
  const float prev = have && a.prev_out ? a.prev_lse[row] : -INFINITY;
  uint4 old = make_uint4(0, 0, 0, 0);
  if (prev != -INFINITY) old = *reinterpret_cast<const uint4*>(a.prev_out + row * kLatent + 8 * x);
  __syncthreads();                                   // (and every row's prev_lse has been read: lse may be the same place)
  if (!have) return;
  float most = prev;
  for (int s = 0; s < n; ++s) most = fmaxf(most, s_part[y][s]);
  float o[8], total = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) o[k] = 0.0f;
  const float* src = a.part_o + (int64_t(t) * n * kWinRows + r) * kLatent + 8 * x;
#pragma unroll 8
  for (int s = 0; s < n; ++s) {
    const float l = s_part[y][s];
    float4 u = make_float4(0.0f, 0.0f, 0.0f, 0.0f), v = u;
    if (l != -INFINITY) {                            // (else that piece has written no outputs)
      u = __ldg(reinterpret_cast<const float4*>(src + int64_t(s) * kWinRows * kLatent));
      v = __ldg(reinterpret_cast<const float4*>(src + int64_t(s) * kWinRows * kLatent) + 1);
    }
    const float f = l != -INFINITY ? expf(l - most) : 0.0f;
    total += f;
    o[0] = fmaf(f, u.x, o[0]);
    o[1] = fmaf(f, u.y, o[1]);
    o[2] = fmaf(f, u.z, o[2]);
    o[3] = fmaf(f, u.w, o[3]);
    o[4] = fmaf(f, v.x, o[4]);
    o[5] = fmaf(f, v.y, o[5]);
    o[6] = fmaf(f, v.z, o[6]);
    o[7] = fmaf(f, v.w, o[7]);
  }
  if (prev != -INFINITY) {
    const float f = expf(prev - most);
    total += f;
    const uint32_t z[4] = {old.x, old.y, old.z, old.w};
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      o[2 * k] = fmaf(f, __uint_as_float(z[k] << 16), o[2 * k]);
      o[2 * k + 1] = fmaf(f, __uint_as_float(z[k] & 0xFFFF0000u), o[2 * k + 1]);
    }
  }
  const float inv = total != 0.0f ? 1.0f / total : 0.0f;
  *reinterpret_cast<uint4*>(a.out + row * kLatent + 8 * x) =
      make_uint4(bf16x2_rn(o[0] * inv, o[1] * inv), bf16x2_rn(o[2] * inv, o[3] * inv), bf16x2_rn(o[4] * inv, o[5] * inv),
                 bf16x2_rn(o[6] * inv, o[7] * inv));
  if (x == 0) a.lse[row] = total != 0.0f ? most + logf(total) : -INFINITY;
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

// The maps of a call, a pure function of the arguments here: encoding them takes longer than the call's
// other work on the host, so the last ones are remembered (as tmap.cuh does for single maps).
bool window_maps(const void* q, uint64_t q_rows, const void* kv, uint64_t kv_rows, WindowMaps* out, WindowLongMaps* out_long) {
  struct Entry {
    bool used;
    const void *q, *kv;
    uint64_t q_rows, kv_rows;
    WindowMaps maps;
    WindowLongMaps longs;
  };
  constexpr int kEntries = 16;
  static std::mutex mu;
  static Entry cache[kEntries];
  static int next = 0;
  std::lock_guard<std::mutex> lk(mu);
  for (const Entry& e : cache)
    if (e.used && e.q == q && e.kv == kv && e.q_rows == q_rows && e.kv_rows == kv_rows) {
      *out = e.maps;
      *out_long = e.longs;
      return true;
    }
  const auto enc = tensor_map_encoder();
  if (!enc) return false;
  const auto encode = [&](CUtensorMap* map, const void* base, uint64_t rows, uint32_t box_rows) {
    const cuuint64_t dim[2] = {kDqk, rows}, stride[1] = {kDqk * 2};
    const cuuint32_t box[2] = {64, box_rows}, step[2] = {1, 1};
    return enc(map, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dim, stride, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
               CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
  };
  bool ok = encode(&out->q, q, q_rows, kWinRows);
  for (int i = 0; i < 7; ++i) ok = ok && encode(&out->kv[i], kv, kv_rows, 1u << i);
  ok = ok && encode(&out_long->q, q, q_rows, 32);
  if (!ok) return false;
  out_long->keys = out->kv[5];
  out_long->values = out->kv[6];
  Entry& e = cache[next];
  next = (next + 1) % kEntries;
  e = {true, q, kv, q_rows, kv_rows, *out, *out_long};
  return true;
}

// Whether a call takes window_long.cu's tiles of 256 rows on four SMs.  Measured, 64 heads, these tiles / those:
//   more rows than one tile of 64 an SM: 10,240 rows over windows of 129, 256, 512, 2,048 positions 19.9 / 19.0,
//     25.9 / 21.8, 37.2 / 27.4, 104 / 58 us; 81,920 rows 73 / 60, 99 / 72, 150 / 96, 473 / 235 us;
//   fewer, where tiles take many blocks: 4,096 rows 24.0 / 19.2 us over 512 positions, 42 / 33 over 2,048
//     (256: 16.0 / 16.8); 2,560 rows 20.3 / 18.2, 32.0 / 32.8;
//   joined, where the longer pass over the outputs holds up the next tile: 64,000 rows over windows of 128, 192,
//     256, 512 positions 71 / 83, 71 / 88, 90 / 89, 128 / 108 us;
//   sequences of fewer rows than a tile: 64 of 128 rows 14 / 20, 17 / 24, 24 / 31, 67 / 73 us.
bool window_is_long(const WindowArgs& a, int span) {
  const int64_t rows = int64_t(a.total_q) * a.d.heads, see = int64_t(a.window) + a.sinks;
  if (a.prev_out && see < 200) return false;
  return see + span - 1 > kWinPos && rows >= int64_t(kLongRows) * a.batch && (rows > int64_t(device_sms()) * kWinRows || (rows >= 4096 && see >= 512));
}

}  // namespace

cudaError_t launch_window(WindowArgs a, cudaStream_t st) {
  const int H = a.d.heads, span = tile_tokens(H, kWinRows);
  a.by_heads = H > 1 ? ~uint64_t(0) / H + 1 : 0;     // (for powers of two, too: 2^64 / H)
  WindowMaps m;
  WindowLongMaps ml;
  const uint64_t rows = a.page_table ? uint64_t(a.d.num_pages) * kPage : uint64_t(a.batch) * uint64_t(a.d.max_ctx);
  if (!window_maps(a.q, uint64_t(a.total_q) * a.d.heads, a.kv, rows, &m, &ml)) return cudaErrorUnknown;
  if (window_is_long(a, span)) {
    a.may_split = 0;
    return launch_window_long(a, ml, (int64_t(a.total_q) * H + kLongRows - 1) / kLongRows + a.batch, st);
  }
  static KernelAttrs attrs[2];
  auto kernel = a.prev_out ? window_kernel<true> : window_kernel<false>;
  cudaError_t e = prepare_kernel(kernel, size_t(kWinSmem), false, attrs[a.prev_out ? 1 : 0]);
  if (e != cudaSuccess) return e;
  static std::atomic<bool> split[2];                 // the register split of the roles counts on this many a thread
  if (!split[a.prev_out ? 1 : 0].load(std::memory_order_relaxed)) {
    cudaFuncAttributes fa;
    if ((e = cudaFuncGetAttributes(&fa, kernel)) != cudaSuccess) return e;
    if (fa.numRegs != kWinRegs) return cudaErrorInvalidConfiguration;
    split[a.prev_out ? 1 : 0].store(true, std::memory_order_relaxed);
  }
  // bounds of what the device will find: tiles, and blocks of one
  int odd = H;                                       // 64 less the greatest common divisor: what a sequence's last tile may lack
  for (int b = kWinRows; b != 0;) {
    const int r = odd % b;
    odd = b;
    b = r;
  }
  const int64_t seqs = min64(a.batch, a.total_q);
  const int64_t tiles = (int64_t(a.total_q) * H + (kWinRows - odd) * seqs) / kWinRows;
  const int64_t ctx = a.page_table ? min64(a.d.max_ctx, int64_t(a.d.max_pages) * kPage) : a.d.max_ctx;
  const int64_t see = min64(ctx, int64_t(a.window) + span - 1 + a.sinks), blocks = (see + kWinPos - 1) / kWinPos;
  const int64_t grid = min64(min64(device_sms(), kWinMaxCtas), max64(1, tiles * blocks));
  // (By the tokens of the call: of padding tokens, which make no tiles, it would be seen on the device only.)
  a.may_split = splits(int64_t(a.total_q) * H / kWinRows, blocks, grid);
  CSA2_PROFILED(st, "window_attn",
                (e = launch_pdl(kernel, dim3(unsigned(grid)), dim3(kWinThreads), size_t(kWinSmem), st, 1, a, m)));
  if (e != cudaSuccess || !a.may_split) return e;
  // Launched only when the pieces are done.  (Ahead of that, by pdl_launch_dependents, its CTAs all go to the
  // few SMs that the attention leaves free and stay there: 24.0 us in place of 18.6 for 8 tokens over 2,048 positions.)
  CSA2_PROFILED(st, "window_merge",
                (window_merge_kernel<<<dim3(kWinRows / kMergeRows, unsigned(min64(tiles, grid / 2))), dim3(kMergeThreads), 0, st>>>(a),
                 e = cudaGetLastError()));
  return e;
}

}  // namespace csa2
