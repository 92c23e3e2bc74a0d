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
#include <cuda.h>
#include <cudaTypedefs.h>

#include <mutex>

#include "common.cuh"
#include "kernels.cuh"
#include "profile.cuh"
#include "tc.cuh"
#include "tmap.cuh"
#include "window.cuh"

namespace csa2 {

namespace {

constexpr int kRowWarps = 8;                         // softmax and outputs: lane quarter w % 4, half of the rows w / 4
constexpr int kMmaWarp = kRowWarps;
constexpr int kGroups = 5;                           // channel groups, a copying warp each: 4 x 128 latent, 64 rope
constexpr int kLoadWarp0 = kMmaWarp + 1;
constexpr int kWinThreads = (kLoadWarp0 + kGroups) * 32;

constexpr int kKReg = kWinPos * 128;                 // 64 channels of a block's positions: 16 KB
constexpr int kQReg = kWinRows * 128;                // 64 channels of a tile's rows: 8 KB
constexpr int kKBytes = 9 * kKReg, kQBytes = 9 * kQReg;
constexpr int kPHalf = 64 * 128;                     // P of 64 positions: 8 KB
constexpr int kQOff = kKBytes, kPOff = kQOff + kQBytes;
constexpr int kWinSmem = kPOff + kPHalf;
constexpr uint32_t kOCol = 64;                       // tensor memory: S^T 64 columns, O^T 4 x 64
constexpr uint32_t kCols = 512;
constexpr int kMinSplit = 3;                         // least blocks a tile's positions are split from

struct WinSmall {
  uint64_t q_full, q_empty, q8_full, q8_empty;       // queries: latent channels, rope channels
  uint64_t k_full[kGroups], k_empty[kGroups];
  uint64_t s_full, p_full, o_full, o_empty, drain;
  uint32_t tmem_slot;
  int abort;
  int bad;                                           // q_start out of order
  uint32_t hidden;                                   // 1 + the last block in which hide_values has changed the places
  int tiles, blocks;                                 // tiles of the call; most blocks of one
  // of the rows of a half, for all lanes of its four warps, which write the same values
  __align__(16) float ref[2][32];                    // softmax reference
  __align__(16) float alpha[2][32];
  __align__(16) int pos[2][32];                      // positions (-1: no such row)
  __align__(16) float top[2][4][kWinRows];           // maxima of a block by lane quarter; sums at the end
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
__device__ inline void bar_sync(int id, int threads) { asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory"); }

struct WindowMaps {
  CUtensorMap q;
  CUtensorMap kv[7];                                 // boxes of 64 channels x 2^i rows
};

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

// 32 values a lane reduced over the warp: lane l gets the sum or maximum of value l (31 shuffles; 130
// cycles, where 32 reductions by redux take 2,950).
template <bool kMax>
__device__ inline float butterfly(const float (&x)[32], int lane) {
  float v[16];
#pragma unroll
  for (int half = 16; half >= 1; half >>= 1) {
    const bool up = lane & half;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float lo = half == 16 ? x[i] : v[i], hi = half == 16 ? x[half + i] : v[half + i];
      const float keep = up ? hi : lo, give = up ? lo : hi;
      const float got = __shfl_xor_sync(0xFFFFFFFFu, give, half);
      v[i] = kMax ? fmaxf(keep, got) : keep + got;
    }
  }
  return v[0];
}

// One step of a transposition: register bit K goes to lane bit B and back.
template <int N, int K, int B, typename T>
__device__ inline void exchange(T (&v)[N], int lane) {
  const bool up = lane >> B & 1;
#pragma unroll
  for (int i = 0; i < N; ++i) {
    if (i & K) continue;
    const T give = up ? v[i] : v[i | K];
    const T got = __shfl_xor_sync(0xFFFFFFFFu, give, 1 << B);
    if (up) v[i] = got;
    else v[i | K] = got;
  }
}

// ---------------------------------------------------------------------------
// Tiles: 64 rows of a sequence each, the sequences' tiles one after the other.
// ---------------------------------------------------------------------------
// Context of sequence b (bad ones are reported by the first CTA's count, and taken as 0).
__device__ inline int context(const WindowArgs& a, int b) {
  const int n = __ldg(a.ctx_len + b);
  return n < 0 || n > a.d.max_ctx || (a.page_table && n > int64_t(a.d.max_pages) * kPage) ? 0 : n;
}
__device__ inline int tiles_of(const WindowArgs& a, int len) { return (len * a.d.heads + kWinRows - 1) / kWinRows; }

// One piece of a tile's work.  Its tokens see the positions lo .. last and the sinks before lo.
//   Compact calls (`compact`, below): all of them fit a block of 128 places.  Position t has place
//     t (t < sinks) or sinks + (t - sinks) % (128 - sinks), so that the rows of consecutive tiles
//     stay where they are and a tile's new positions take the places of those that the window has left.
//   Other calls: whole pages of 64 positions, the sinks' (sp of them) and then the window's, two a block.
struct Piece {
  int seq, from, len, ctx;      // sequence: first query token, query tokens, context
  int row0;                     // first row in the sequence
  int lo, last;
  int sp, np;
  int blk, n;                   // blocks of this piece
};

// Position of place e of block j of a piece (-1: none).
__device__ inline int place_position(const WindowArgs& a, const Piece& p, int j, int e) {
  if (a.compact) {
    if (e < a.sinks) return e <= p.last ? e : -1;
    const int c = kWinPos - a.sinks, d = (p.last - a.sinks) % c - (e - a.sinks);      // places from e on to the last position's
    const int t = p.last - (d < 0 ? d + c : d);
    return t >= max(p.lo, a.sinks) ? t : -1;
  }
  const int i = 2 * (p.blk + j) + (e >> 6);
  const int t = (i < p.sp ? i : p.lo / kPage + i - p.sp) * kPage + (e & (kPage - 1));
  return i < p.np && t <= p.last ? t : -1;
}

// A warp's way through the tiles.  It keeps 32 sequences, one a lane.
struct Walk {
  const WindowArgs& a;
  int lane;
  int b0, base;                                      // first sequence kept, tiles before it
  int from, len, ctx, upto;                          // the lane's sequence; tiles up to its end from b0 on
  __device__ Walk(const WindowArgs& args, int l) : a(args), lane(l), b0(0), base(0) { load(); }
  __device__ void load() {
    const int i = b0 + lane;
    from = len = ctx = upto = 0;
    if (i < a.batch) {
      from = __ldg(a.q_start + i);
      len = __ldg(a.q_start + i + 1) - from;
      ctx = context(a, i);
      upto = tiles_of(a, len);
    }
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += y;
    }
  }
  // Piece s of n of tile t (not before the one asked for last); false behind the last.
  __device__ bool piece(int t, int s, int n, Piece& p) {
    uint32_t past;
    while ((past = __ballot_sync(0xFFFFFFFFu, base + upto > t)) == 0) {
      base += __shfl_sync(0xFFFFFFFFu, upto, 31);
      b0 += 32;
      if (b0 >= a.batch) return false;
      load();
    }
    const int w = __ffs(past) - 1;
    p.seq = b0 + w;
    p.from = __shfl_sync(0xFFFFFFFFu, from, w);
    p.len = __shfl_sync(0xFFFFFFFFu, len, w);
    p.ctx = __shfl_sync(0xFFFFFFFFu, ctx, w);
    const int before = __shfl_sync(0xFFFFFFFFu, upto, max(w - 1, 0));
    p.row0 = (t - base - (w > 0 ? before : 0)) * kWinRows;
    const int tok0 = p.row0 / a.d.heads, tok1 = min(p.len - 1, (p.row0 + kWinRows - 1) / a.d.heads);
    p.last = p.ctx - p.len + tok1;
    p.lo = max(0, p.ctx - p.len + tok0 - a.window + 1);
    p.sp = min((a.sinks + kPage - 1) / kPage, p.lo / kPage);
    p.np = p.last < 0 ? 0 : p.sp + p.last / kPage - p.lo / kPage + 1;
    const int nb = a.compact ? p.last >= 0 : (p.np + 1) / 2;
    p.blk = n == 1 ? 0 : nb * s / n;
    p.n = n == 1 ? nb : nb * (s + 1) / n - p.blk;
    return true;
  }
};

// Cache row of position t (-1: its page id is out of range).
__device__ inline int row_of(const WindowArgs& a, int seq, int t) {
  if (!a.page_table) return int(int64_t(seq) * a.d.max_ctx + t);
  const int pg = __ldg(a.page_table + int64_t(seq) * a.d.max_pages + t / kPage);
  return pg < 0 || pg >= a.d.num_pages ? -1 : pg * kPage + t % kPage;
}

// ---------------------------------------------------------------------------
// Roles
// ---------------------------------------------------------------------------
// The position's values, if an infinity or NaN is among them, become 0: its weight in the rows that
// do not see it is 0, and so must be 0 times its values.  The rows that do see it are NaN by its
// score, which holds the same channels.
__device__ __noinline__ void hide_values(WinSmall& sm, uint8_t* base, int e, uint32_t block) {
  bool whole = true;
#pragma unroll 1
  for (int c = 0; c < 64; ++c) {
    const uint4 x = *reinterpret_cast<const uint4*>(base + (c >> 3) * kKReg + tc::sw128_offset(e, c & 7));
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) whole = whole && (w[i] & 0x7F80u) != 0x7F80u && (w[i] & 0x7F800000u) != 0x7F800000u;
  }
  if (whole) return;
  *reinterpret_cast<volatile uint32_t*>(&sm.hidden) = block + 1;
#pragma unroll 1
  for (int c = 0; c < 64; ++c)
    *reinterpret_cast<uint4*>(base + (c >> 3) * kKReg + tc::sw128_offset(e, c & 7)) = make_uint4(0, 0, 0, 0);
}

struct Span {
  int first, units, step, pieces;                    // the CTA's units: first, first + step, ... below units
};

// A box of 2^lg rows (lg -1: none) from cache row `row` on, for the places from `slot` on.
struct Box {
  int slot, row, lg;
};

// The positions first .. last of a compact tile as boxes, one a lane from lane `k` on: runs of
// rows, cut at pages and where the places come round, in powers of two (a tile has at most 6 runs
// of 128 rows together: at most 23 boxes).  `page`: lane i has the page ids of the first two pages
// (lanes 0, 1) and of the window's (lanes 2 .. 5).  Returns their rows.
__device__ inline int boxes(const WindowArgs& a, const Piece& p, int first, int last, int page, int lane, int& k, Box& mine,
                            bool& lost) {
  int rows = 0;
  for (int t = first; t <= last;) {
    const int at = t / kPage;
    int slot = t < a.sinks ? t : a.sinks + (t - a.sinks) % (kWinPos - a.sinks);
    int n = min(last - t + 1, kWinPos - slot), row;
    if (a.page_table) {
      n = min(n, kPage - t % kPage);
      const int pg = __shfl_sync(0xFFFFFFFFu, page, at < 2 ? at : 2 + at - p.lo / kPage);
      row = pg < 0 || pg >= a.d.num_pages ? -1 : pg * kPage + t % kPage;
    } else {
      row = int(int64_t(p.seq) * a.d.max_ctx + t);
    }
    t += n;
    if (row < 0) {
      lost = true;
      continue;
    }
    rows += n;
    while (n > 0) {
      const int lg = min(6, 31 - __clz(n));
      if (k == lane) mine = {slot, row, lg};
      ++k;
      slot += 1 << lg;
      row += 1 << lg;
      n -= 1 << lg;
    }
  }
  return rows;
}
// What a compact tile sees from position `from` on.
__device__ inline int tile_boxes(const WindowArgs& a, const Piece& p, int from, int lane, Box& mine, bool& lost) {
  int page = -1, k = 0;
  if (a.page_table && lane < 6) {
    const int i = lane < 2 ? lane : p.lo / kPage + lane - 2;
    if (i < a.d.max_pages && i * kPage <= p.last) page = __ldg(a.page_table + int64_t(p.seq) * a.d.max_pages + i);
  }
  mine.lg = -1;
  const int rows = boxes(a, p, from, min(a.sinks - 1, p.last), page, lane, k, mine, lost);
  return rows + boxes(a, p, max(from, max(p.lo, a.sinks)), p.last, page, lane, k, mine, lost);
}

// Where P of a block's first and last 64 positions goes: over the block's rope channels, which only
// the scores need; in a compact call, whose rows stay, into a place of its own and over the queries'
// rope channels, which no other block of the tile needs.
__device__ inline uint32_t p_offset(const WindowArgs& a, int half) {
  return a.compact ? (half == 0 ? kPOff : kQOff + 8 * kQReg) : 8 * kKReg + half * kPHalf;
}

// Copies channel group g of the queries and the cache rows.  (One warp for all groups takes 650 cycles
// for the few copies of one: what it waits for is the issue, not the copies.)
__device__ inline void load_role(const WindowArgs& a, WinSmall& sm, uint8_t* base, const Span& w, int g, int lane,
                                 const WindowMaps& m) {
  Walk walk(a, lane);
  Piece p;
  uint32_t nq = 0, nk = 0;
  int was_seq = -1, was_last = 0;                    // what the places hold
  const int regions = g < 4 ? 2 : 1;
  uint64_t* q_full = g < 4 ? &sm.q_full : &sm.q8_full;
  uint64_t* q_empty = g < 4 ? &sm.q_empty : &sm.q8_empty;
  for (int u = w.first; u < w.units; u += w.step) {
    if (!walk.piece(u / w.pieces, u % w.pieces, w.pieces, p)) return;
    if (p.n == 0) continue;
    // a compact tile's boxes: what the tile before has not left there, or all of it
    Box box;
    int rows = 0;
    bool lost = false;
    if (a.compact) {
      rows = tile_boxes(a, p, p.seq == was_seq ? was_last + 1 : 0, lane, box, lost);
      was_seq = p.seq;
      was_last = p.last;
    }
    for (int j = 0; j < p.n; ++j, ++nk) {
      int row = -1;                                  // lane's half of the block (lane & 1)
      if (!a.compact) {
        const int t = place_position(a, p, j, kPage * (lane & 1));
        if (t >= 0) {
          row = row_of(a, p.seq, t);
          lost = row < 0;
        }
      }
      if (g == 0 && lost) raise_err(a.ws, CSA2_DEV_PAGE_ID);
      if (j == 0) {
        if (!wait_warp(sm, q_empty, (nq & 1) ^ 1, a.ws)) return;
        if (lane == 0) tc::mbar_expect_tx(q_full, uint32_t(regions * kQReg));
        __syncwarp();
        if (lane < regions)
          tc::tma_load_2d(&m.q, base + kQOff + (2 * g + lane) * kQReg, 64 * (2 * g + lane), p.from * a.d.heads + p.row0, q_full);
        ++nq;
      }
      if (!wait_warp(sm, &sm.k_empty[g], (nk & 1) ^ 1, a.ws)) return;
      if (a.compact) {
        // values of the tile before may have been taken out of their places
        if (g < 4 && nk > 0 && *reinterpret_cast<volatile uint32_t*>(&sm.hidden) == nk)
          rows = tile_boxes(a, p, 0, lane, box, lost);
        if (lane == 0) tc::mbar_expect_tx(&sm.k_full[g], uint32_t(regions * rows * 128));
        __syncwarp();
        if (box.lg >= 0)
          for (int r = 2 * g; r < 2 * g + regions; ++r)
            tc::tma_load_2d(&m.kv[box.lg], base + r * kKReg + box.slot * 128, 64 * r, box.row, &sm.k_full[g]);
      } else {
        const int halves = __popc(__ballot_sync(0xFFFFFFFFu, row >= 0) & 3u);
        if (lane == 0) tc::mbar_expect_tx(&sm.k_full[g], uint32_t(regions * halves * (kKReg / 2)));
        __syncwarp();
        const int r = 2 * g + (lane >> 1);
        if (lane < 2 * regions && row >= 0)
          tc::tma_load_2d(&m.kv[6], base + r * kKReg + (lane & 1) * (kKReg / 2), 64 * r, row, &sm.k_full[g]);
      }
    }
  }
}

// Issues the products.  The offsets are constants: a product takes 58 cycles, and formed at run time
// they take longer than that.
__device__ inline void mma_role(const WindowArgs& a, WinSmall& sm, uint8_t* base, const Span& w, int lane, uint32_t tmem) {
  constexpr uint32_t id_s = tc::idesc_bf16(kWinPos, kWinRows, 0, 0);
  constexpr uint32_t id_o = tc::idesc_bf16(kWinPos, kWinRows, 1, 1);
  const uint32_t at = tc::smem_u32(base);
  const uint64_t ks = tc::smem_desc(at, 16, 1024, 2), qs = tc::smem_desc(at + kQOff, 16, 1024, 2);
  const uint64_t vs = tc::smem_desc(at, kKReg, 1024, 2);
  const uint64_t p0 = tc::smem_desc(at + p_offset(a, 0), kPHalf, 1024, 2), p1 = tc::smem_desc(at + p_offset(a, 1), kPHalf, 1024, 2);
  const bool leader = elect_one();
  Walk walk(a, lane);
  Piece p;
  uint32_t nq = 0, nk = 0;
  for (int u = w.first; u < w.units; u += w.step) {
    if (!walk.piece(u / w.pieces, u % w.pieces, w.pieces, p)) return;
    if (p.n == 0) continue;
    if (!wait_warp(sm, &sm.q_full, nq & 1, a.ws)) return;
    for (int j = 0; j < p.n; ++j, ++nk) {
#pragma unroll
      for (int g = 0; g < kGroups; ++g) {
        if (!wait_warp(sm, &sm.k_full[g], nk & 1, a.ws)) return;
        if (g == 4 && j == 0 && !wait_warp(sm, &sm.q8_full, nq & 1, a.ws)) return;
        tc::tc_fence_after_sync();
        if (leader) {
#pragma unroll
          for (int i = 0; i < (g < 4 ? 8 : 4); ++i) {
            const uint32_t kb = 2 * g + (i >> 2), off = (i & 3) * 32;
            tc::mma_bf16(tmem, ks + ((kb * kKReg + off) >> 4), qs + ((kb * kQReg + off) >> 4), id_s, g + i > 0);
          }
        }
        __syncwarp();
      }
      if (leader) {
        tc::mma_commit(&sm.s_full);
        if (a.compact) tc::mma_commit(&sm.k_empty[4]);
        if (j == p.n - 1) {
          tc::mma_commit(&sm.q_empty);
          if (!a.compact) tc::mma_commit(&sm.q8_empty);
        }
      }
      __syncwarp();
      if (!wait_warp(sm, &sm.p_full, nk & 1, a.ws)) return;
      if (j == 0 && !wait_warp(sm, &sm.o_empty, (nq & 1) ^ 1, a.ws)) return;
      tc::tc_fence_after_sync();
      if (leader) {
        const bool more = j > 0;
#pragma unroll
        for (int mt = 0; mt < 4; ++mt) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            tc::mma_bf16(tmem + kOCol + 64 * mt, vs + ((2 * mt * kKReg + k * 2048) >> 4), (k < 4 ? p0 : p1) + (((k & 3) * 2048) >> 4),
                         id_o, more || k > 0);
          tc::mma_commit(&sm.k_empty[mt]);
        }
        tc::mma_commit(a.compact ? &sm.q8_empty : &sm.k_empty[4]);
        if (j == p.n - 1) tc::mma_commit(&sm.o_full);
      }
      __syncwarp();
    }
    ++nq;
  }
}

// What a row warp has to know of a piece before its scores come.
struct Ahead {
  Piece p;
  bool have;
  int mine;                                          // position of the lane's row, -1: no such row
  int t, row;                                        // position in the lane's place of the first block (-1: none), its row
};
__device__ inline void place_seen(const WindowArgs& a, const Piece& p, int j, int e, int& t, int& row) {
  t = place_position(a, p, j, e);
  row = t >= 0 ? row_of(a, p.seq, t) : -1;
}
__device__ inline void look_ahead(const WindowArgs& a, Walk& walk, const Span& w, int u, int half, int e, int lane, Ahead& n) {
  n.have = u < w.units && walk.piece(u / w.pieces, u % w.pieces, w.pieces, n.p);
  if (!n.have) return;
  const int lr = n.p.row0 + 32 * half + lane;
  n.mine = lr < n.p.len * a.d.heads ? n.p.ctx - n.p.len + lr / a.d.heads : -1;
  if (n.p.n > 0) place_seen(a, n.p, 0, e, n.t, n.row);
}

// Softmax over a block's positions (tensor-memory lanes) and the outputs.  Warp rw has the
// lanes 32 (rw % 4) .. + 31 and the rows 32 (rw / 4) .. + 31; lane i keeps the state of row i of
// these (alike in the four warps of a half, but for the sum, which is of its own lanes).
// Shared memory is the products': they take five sixths of its bandwidth, so values cross the lanes
// by shuffles.
// A wait that gives up leaves the warp in the loop, without waits or results: its hardware
// barriers have no limit, and all eight warps pass the same ones.
__device__ inline void row_role(const WindowArgs& a, WinSmall& sm, uint8_t* base, const Span& w, int rw, int lane,
                                uint32_t tmem) {
  const int quarter = rw & 3, half = rw >> 2, e = 32 * quarter + lane;
  const uint32_t lanes = tmem + (uint32_t(32 * quarter) << 16) + uint32_t(32 * half);
  const float c2 = a.scale * 1.4426950408889634f;
  uint8_t* const p_at = base + p_offset(a, quarter >> 1);
  bool dead = false;
  Walk walk(a, lane);
  Ahead now;
  look_ahead(a, walk, w, w.first, half, e, lane, now);
  uint32_t nq = 0, nk = 0;
  for (int u = w.first; now.have; u += w.step) {
    const Piece p = now.p;
    const int mine = now.mine, rows = p.len * a.d.heads;
    const int lr = p.row0 + 32 * half + lane;
    sm.pos[half][lane] = mine;
    __syncwarp();
    const int p_max = __reduce_max_sync(0xFFFFFFFFu, mine);
    const int p_min = __reduce_min_sync(0xFFFFFFFFu, lr < rows ? mine : p_max);
    float ref = -INFINITY, sum = 0.0f;
    int t = now.t, row = now.row;
    for (int j = 0; j < p.n; ++j, ++nk) {
      if (j > 0) place_seen(a, p, j, e, t, row);
      if (row < 0) t = -1;
      const bool all = t >= 0 && t <= p_min && (t > p_max - a.window || t < a.sinks);
      const bool edge = !__all_sync(0xFFFFFFFFu, all);
      if (!dead && !wait_warp(sm, &sm.s_full, nk & 1, a.ws)) dead = true;
      tc::tc_fence_after_sync();
      float x[32];
      tc::tmem_ld32(lanes, x);
#pragma unroll
      for (int i = 0; i < 32; ++i) x[i] *= c2;
      if (edge) {
        bool odd = false;                            // some score of a row that does not see the position is no number
#pragma unroll
        for (int i4 = 0; i4 < 8; ++i4) {
          const int4 pr = reinterpret_cast<const int4*>(sm.pos[half])[i4];
          const int q4[4] = {pr.x, pr.y, pr.z, pr.w};
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int i = 4 * i4 + k;
            const bool see = t >= 0 && t <= q4[k] && (t > q4[k] - a.window || t < a.sinks);
            const bool fine = fabsf(x[i]) < INFINITY;
            odd = odd || !(see || fine);
            x[i] = see ? (fine ? x[i] : NAN) : -INFINITY;
          }
        }
        if (odd) hide_values(sm, base, e, nk);
        __syncwarp();
      }
      float top = butterfly<true>(x, lane);
      sm.top[nk & 1][quarter][32 * half + lane] = top;
      bar_sync(1 + half, 128);
#pragma unroll
      for (int k = 0; k < 4; ++k) top = fmaxf(top, sm.top[nk & 1][k][32 * half + lane]);
      float alpha = 1.0f;
      if (top > ref + 8.0f) {
        const float to = ceilf(top);
        if (ref != -INFINITY) alpha = ex2(ref - to);
        ref = to;
      }
      sm.ref[half][lane] = ref == -INFINITY ? 0.0f : ref;
      const bool turn = __any_sync(0xFFFFFFFFu, alpha != 1.0f);
      if (turn) sm.alpha[half][lane] = alpha;
      __syncwarp();
      if (turn) {
        // the outputs so far to the new reference (this block's scores came after the last product: the
        // copies that they needed waited for it)
        sum *= alpha;
#pragma unroll 1
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll 1
          for (int c = 0; c < 32; c += 8) {
            float o[8];
            tc::tmem_ld8(lanes + kOCol + 64 * mt + c, o);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] *= sm.alpha[half][c + i];
            tc::tmem_st8(lanes + kOCol + 64 * mt + c, o);
          }
      }
#pragma unroll
      for (int i8 = 0; i8 < 4; ++i8) {
        uint32_t pk[4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float4 r4 = reinterpret_cast<const float4*>(sm.ref[half])[2 * i8 + k];
          const int i = 8 * i8 + 4 * k;
          x[i] = ex2(x[i] - r4.x);
          x[i + 1] = ex2(x[i + 1] - r4.y);
          x[i + 2] = ex2(x[i + 2] - r4.z);
          x[i + 3] = ex2(x[i + 3] - r4.w);
          pk[2 * k] = bf16x2_rn(x[i], x[i + 1]);
          pk[2 * k + 1] = bf16x2_rn(x[i + 2], x[i + 3]);
        }
        *reinterpret_cast<uint4*>(p_at + tc::sw128_offset(e & 63, 4 * half + i8)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
      }
      tc::fence_proxy_async_smem();
      tc::tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) arrive(&sm.p_full);
      sum += butterfly<false>(x, lane);
    }
    look_ahead(a, walk, w, u + w.step, half, e, lane, now);
    // outputs: sums of the four lane quarters, joined with the other attention's
    const bool join = a.prev_out != nullptr && w.pieces == 1;
    const int64_t row0 = int64_t(p.from) * a.d.heads + p.row0 + 32 * half;
    float prev = -INFINITY;
    if (join && lr < rows) prev = a.prev_lse[row0 + lane];
    float (&sums)[4][kWinRows] = sm.top[nk & 1];     // (the other one may still be read)
    sums[quarter][32 * half + lane] = sum;
    bar_sync(1 + half, 128);
    float total = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) total += sums[k][32 * half + lane];
    float own = total != 0.0f ? 1.0f / total : 0.0f, other = 0.0f;
    float lse = total != 0.0f ? ((ref == -INFINITY ? 0.0f : ref) + log2f(total)) * 0.6931471805599453f : -INFINITY;
    if (join && prev != -INFINITY) {
      const float most = fmaxf(lse, prev), x0 = expf(lse - most), x1 = expf(prev - most);
      own *= x0 / (x0 + x1);
      other = x1 / (x0 + x1);
      lse = most + logf(x0 + x1);
    }
    sm.ref[half][lane] = own;
    // after the transposition a lane has 8 channels of the rows 8 k + lane % 8
    const int ch = 32 * quarter + 8 * (lane >> 3);
    const int64_t at = (row0 + (lane & 7)) * kLatent + ch;
    const int left = rows - (p.row0 + 32 * half) - (lane & 7);              // row 8 k exists: 8 k < left
    uint4 old[4];
    float share[4];
    if (join) {
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        share[k] = __shfl_sync(0xFFFFFFFFu, other, 8 * k + (lane & 7));
        old[k] = make_uint4(0, 0, 0, 0);
        if (share[k] != 0.0f && 8 * k < left) old[k] = *reinterpret_cast<const uint4*>(a.prev_out + at + 8 * k * kLatent);
      }
    }
    if (p.n > 0) {
      if (!dead && !wait_warp(sm, &sm.o_full, nq & 1, a.ws)) dead = true;
      tc::tc_fence_after_sync();
    }
    __syncwarp();
    if (w.pieces > 1) {
      // a piece: its own softmax in fp32, for the merge
      if (!dead) {
        if (quarter == 0) {
          a.part_lse[u * kWinRows + 32 * half + lane] = lse;
          if (u % w.pieces == 0 && rw == 0 && lane == 0)
            a.tiles[u / w.pieces] = make_int2(int(row0), min(kWinRows, rows - p.row0));
        }
        if (p.n > 0) {
#pragma unroll 1
          for (int mt = 0; mt < 4; ++mt) {
            float o[32];
            tc::tmem_ld32(lanes + kOCol + 64 * mt, o);
            float* dst = a.part_o + (int64_t(u) * kWinRows + 32 * half) * kLatent + 128 * mt + e;
#pragma unroll
            for (int i = 0; i < 32; ++i)
              if (p.row0 + 32 * half + i < rows) dst[i * kLatent] = o[i] * sm.ref[half][i];
          }
        }
      }
    } else if (!dead) {
      if (quarter == 0 && lr < rows) a.lse[row0 + lane] = lse;
#pragma unroll 1
      for (int mt = 0; mt < 4; ++mt) {
        float o[32];
        if (p.n > 0) {
          tc::tmem_ld32(lanes + kOCol + 64 * mt, o);
#pragma unroll
          for (int i4 = 0; i4 < 8; ++i4) {
            const float4 f = reinterpret_cast<const float4*>(sm.ref[half])[i4];
            o[4 * i4] *= f.x;
            o[4 * i4 + 1] *= f.y;
            o[4 * i4 + 2] *= f.z;
            o[4 * i4 + 3] *= f.w;
          }
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0.0f;
        }
        uint32_t y[16];                              // 4 rows of 8 channels
        if (join) {
          exchange<32, 1, 0>(o, lane);
          exchange<32, 2, 1>(o, lane);
          exchange<32, 4, 2>(o, lane);
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const uint32_t x[4] = {old[k].x, old[k].y, old[k].z, old[k].w};
#pragma unroll
            for (int i = 0; i < 4; ++i)
              y[4 * k + i] = bf16x2_rn(fmaf(share[k], __uint_as_float(x[i] << 16), o[8 * k + 2 * i]),
                                       fmaf(share[k], __uint_as_float(x[i] & 0xFFFF0000u), o[8 * k + 2 * i + 1]));
            // the next channels' come while these go
            if (mt < 3 && share[k] != 0.0f && 8 * k < left)
              old[k] = *reinterpret_cast<const uint4*>(a.prev_out + at + 8 * k * kLatent + 128 * (mt + 1));
          }
        } else {
#pragma unroll
          for (int i = 0; i < 16; ++i) {
            const uint32_t z = bf16x2_rn(o[2 * i], o[2 * i + 1]);          // two rows of the lane's channel
            const uint32_t got = __shfl_xor_sync(0xFFFFFFFFu, z, 1);
            y[i] = lane & 1 ? __byte_perm(got, z, 0x7632) : __byte_perm(z, got, 0x5410);
          }
          exchange<16, 1, 1>(y, lane);
          exchange<16, 2, 2>(y, lane);
        }
#pragma unroll
        for (int k = 0; k < 4; ++k)
          if (8 * k < left)
            *reinterpret_cast<uint4*>(a.out + at + 8 * k * kLatent + 128 * mt) =
                make_uint4(y[4 * k], y[4 * k + 1], y[4 * k + 2], y[4 * k + 3]);
      }
    }
    if (p.n > 0) {
      tc::tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) arrive(&sm.o_empty);
      ++nq;
    }
    bar_sync(1 + half, 128);                         // the sums and factors have been read
  }
}

__global__ void __launch_bounds__(kWinThreads, 1)
    window_kernel(const __grid_constant__ WindowArgs a, const __grid_constant__ WindowMaps m) {
  extern __shared__ __align__(1024) uint8_t base[];  // 1024-byte aligned: checked below
  __shared__ WinSmall sm;
  const int tid = threadIdx.x, lane = tid & 31, wid = tid >> 5;
  if (tc::smem_u32(base) & 1023u) {                  // never, as laid out
    pdl_wait();
    if (tid == 0) raise_err(a.ws, CSA2_DEV_TIMEOUT);
    return;
  }
  if (wid == kMmaWarp) tc::tmem_alloc(&sm.tmem_slot, kCols);
  if (tid == 0) {
    tc::mbar_init(&sm.q_full, kGroups - 1);
    tc::mbar_init(&sm.q_empty, 1);
    tc::mbar_init(&sm.q8_full, 1);
    tc::mbar_init(&sm.q8_empty, 1);
    for (int g = 0; g < kGroups; ++g) {
      tc::mbar_init(&sm.k_full[g], 1);
      tc::mbar_init(&sm.k_empty[g], 1);
    }
    tc::mbar_init(&sm.s_full, 1);
    tc::mbar_init(&sm.p_full, kRowWarps);
    tc::mbar_init(&sm.o_full, 1);
    tc::mbar_init(&sm.o_empty, kRowWarps);
    tc::mbar_init(&sm.drain, 1);
    tc::fence_mbar_init();
    sm.abort = 0;
    sm.bad = 0;
    sm.hidden = 0;
    sm.tiles = 0;
    sm.blocks = 0;
  }
  pdl_wait();
  pdl_launch_dependents();
  __syncthreads();
  // count the tiles; starts out of order are reported and the call writes nothing
  {
    const bool paged = a.page_table != nullptr;
    const int H = a.d.heads, span = kWinRows % H == 0 ? kWinRows / H : (H + 62) / H + 1;   // most tokens of a tile
    int tiles = 0, blocks = 0;
    bool bad = false;
    for (int b = tid; b < a.batch; b += kWinThreads) {
      const int s0 = __ldg(a.q_start + b), s1 = __ldg(a.q_start + b + 1);
      if (s0 < 0 || s1 < s0 || s1 > a.total_q) {
        bad = true;
        continue;
      }
      if (blockIdx.x == 0) check_ctx(__ldg(a.ctx_len + b), a.d, paged, a.ws);
      tiles += tiles_of(a, s1 - s0);
      if (s1 > s0) {
        const int64_t see = min64(context(a, b), int64_t(a.window) + min(span, s1 - s0) - 1 + a.sinks);
        blocks = max(blocks, int((see + kWinPos - 1) / kWinPos));
      }
    }
    if (bad) atomicOr(&sm.bad, 1);
    tiles = __reduce_add_sync(0xFFFFFFFFu, tiles);
    blocks = __reduce_max_sync(0xFFFFFFFFu, blocks);
    if (lane == 0) {
      atomicAdd(&sm.tiles, tiles);
      atomicMax(&sm.blocks, blocks);
    }
  }
  tc::tc_fence_before_sync();
  __syncthreads();
  tc::tc_fence_after_sync();
  const uint32_t tmem = sm.tmem_slot;
  const int tiles = sm.bad ? 0 : sm.tiles, grid = gridDim.x;
  Span w;
  w.pieces = 1;
  if (a.may_split && tiles > 0 && 2 * tiles <= grid && sm.blocks >= kMinSplit) w.pieces = min(grid / tiles, sm.blocks);
  if (a.compact) {
    // consecutive tiles share most of their rows
    w.first = int(int64_t(tiles) * blockIdx.x / grid);
    w.units = int(int64_t(tiles) * (blockIdx.x + 1) / grid);
    w.step = 1;
  } else {
    w.first = blockIdx.x;
    w.units = tiles * w.pieces;
    w.step = grid;
  }
  if (blockIdx.x == 0 && tid == 0) {
    if (sm.bad) raise_err(a.ws, CSA2_DEV_Q_START);
    a.head[0] = tiles;
    a.head[1] = w.pieces;
  }
  if (wid < kRowWarps) row_role(a, sm, base, w, wid, lane, tmem);
  else if (wid == kMmaWarp) mma_role(a, sm, base, w, lane, tmem);
  else load_role(a, sm, base, w, wid - kLoadWarp0, lane, m);
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
  pdl_wait();
  pdl_launch_dependents();
  const int tiles = a.head[0], n = a.head[1], t = blockIdx.y;
  if (n <= 1 || t >= tiles) return;
  const int2 tile = a.tiles[t];
  const int r = blockIdx.x * kMergeRows + threadIdx.x / (kLatent / 8), c = threadIdx.x % (kLatent / 8) * 8;
  const bool have = r < tile.y;
  const int64_t row = int64_t(tile.x) + r;
  float top = -INFINITY, prev = -INFINITY;
  if (have) {
    for (int s = 0; s < n; ++s) top = fmaxf(top, a.part_lse[(t * n + s) * kWinRows + r]);
    if (a.prev_out) prev = a.prev_lse[row];
  }
  const float most = fmaxf(top, prev);
  float o[8], total = 0.0f;
#pragma unroll
  for (int k = 0; k < 8; ++k) o[k] = 0.0f;
  if (have) {
    for (int s = 0; s < n; ++s) {
      const float l = a.part_lse[(t * n + s) * kWinRows + r];
      if (l == -INFINITY) continue;                  // (that piece has written no outputs)
      const float f = expf(l - most);
      total += f;
      const float4* src = reinterpret_cast<const float4*>(a.part_o + (int64_t(t * n + s) * kWinRows + r) * kLatent + c);
      const float4 u = src[0], v = src[1];
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
      const uint4 v = *reinterpret_cast<const uint4*>(a.prev_out + row * kLatent + c);
      const uint32_t x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        o[2 * k] = fmaf(f, __uint_as_float(x[k] << 16), o[2 * k]);
        o[2 * k + 1] = fmaf(f, __uint_as_float(x[k] & 0xFFFF0000u), o[2 * k + 1]);
      }
    }
  }
  __syncthreads();                                   // every row's prev_lse has been read (lse may be the same place)
  if (!have) return;
  const float inv = total != 0.0f ? 1.0f / total : 0.0f;
  *reinterpret_cast<uint4*>(a.out + row * kLatent + c) =
      make_uint4(bf16x2_rn(o[0] * inv, o[1] * inv), bf16x2_rn(o[2] * inv, o[3] * inv), bf16x2_rn(o[4] * inv, o[5] * inv),
                 bf16x2_rn(o[6] * inv, o[7] * inv));
  if (c == 0) a.lse[row] = total != 0.0f ? most + logf(total) : -INFINITY;
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

cudaError_t launch_window(WindowArgs a, cudaStream_t st) {
  const int H = a.d.heads, span = kWinRows % H == 0 ? kWinRows / H : (H + 62) / H + 1;   // most tokens of a tile
  a.compact = int64_t(a.window) + span - 1 + a.sinks <= kWinPos;
  WindowMaps m;
  const auto enc = tensor_map_encoder();
  const uint64_t rows = a.page_table ? uint64_t(a.d.num_pages) * kPage : uint64_t(a.batch) * uint64_t(a.d.max_ctx);
  if (!encode_2d_cached(enc, &m.q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.q, kDqk, uint64_t(a.total_q) * a.d.heads, kDqk * 2,
                        64, kWinRows, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B))
    return cudaErrorUnknown;
  for (int i = a.compact ? 0 : 6; i < 7; ++i)
    if (!encode_2d_cached(enc, &m.kv[i], CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.kv, kDqk, rows, kDqk * 2, 64, 1u << i,
                          CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B))
      return cudaErrorUnknown;
  static KernelAttrs attrs;
  cudaError_t e = prepare_kernel(window_kernel, size_t(kWinSmem), false, attrs);
  if (e != cudaSuccess) return e;
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
  // fewer tiles than half of the SMs, at least: their positions may be split
  a.may_split = blocks >= kMinSplit && 2 * (int64_t(a.total_q) * H / kWinRows) <= grid;
  CSA2_PROFILED(st, "window_attn",
                (e = launch_pdl(window_kernel, dim3(unsigned(grid)), dim3(kWinThreads), size_t(kWinSmem), st, 1, a, m)));
  if (e != cudaSuccess || !a.may_split) return e;
  CSA2_PROFILED(st, "window_merge",
                (e = launch_pdl(window_merge_kernel, dim3(kWinRows / kMergeRows, unsigned(min64(tiles, grid / 2))),
                                dim3(kMergeThreads), 0, st, 1, a)));
  return e;
}

}  // namespace csa2
