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
constexpr int kMmaWarp = kRowWarps;                  // the last warp copies
constexpr int kWinThreads = (kRowWarps + 2) * 32;

constexpr int kKReg = kWinPos * 128;                 // 64 channels of a block's positions: 16 KB
constexpr int kQReg = kWinRows * 128;                // 64 channels of a tile's rows: 8 KB
constexpr int kKBytes = 9 * kKReg, kQBytes = 9 * kQReg;
constexpr int kPOff = 8 * kKReg;                     // P takes the place of the block's rope channels
constexpr int kQOff = kKBytes, kStageOff = kQOff + kQBytes;
constexpr int kStageWarp = 8 * 64;                   // 8 rows x 32 channels of outputs
constexpr int kWinSmem = kStageOff + kRowWarps * kStageWarp;
constexpr int kGroups = 5;                           // channel groups of a block: 4 x 128 latent, 64 rope
constexpr uint32_t kOCol = 64;                       // tensor memory: S^T 64 columns, O^T 4 x 64
constexpr uint32_t kCols = 512;
constexpr int kMinSplit = 3;                         // least blocks a tile's positions are split from

struct WinSmall {
  uint64_t q_full, q_empty;
  uint64_t k_full[kGroups], k_empty[kGroups];
  uint64_t s_full, p_full, o_full, o_empty, drain;
  uint32_t tmem_slot;
  int abort;
  int bad;                                           // q_start out of order
  int tiles, blocks;                                 // tiles of the call; most blocks of one
  __align__(16) float ref[kRowWarps][32];            // softmax reference of the warp's rows, for all its lanes
  __align__(16) float alpha[kRowWarps][32];
  __align__(16) int pos[kRowWarps][32];              // positions of the warp's rows (-1: no such row)
  __align__(16) float top[2][4][kWinRows];           // maxima of a block by lane quarter
  __align__(16) float sum[4][kWinRows];
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

// Four rows of a tensor map, 64 channels each (the map's box is one row high).
__device__ inline void tma_gather4(const CUtensorMap* map, uint32_t dst, int x, int4 y, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes "
      "[%0], [%1, {%2, %3, %4, %5, %6}], [%7];"
      ::"r"(dst), "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y.x), "r"(y.y), "r"(y.z), "r"(y.w), "r"(tc::smem_u32(bar))
      : "memory");
}

__device__ inline float ex2(float x) {
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}
__device__ inline float max_over_warp(float x) {
  float y;
  asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(y) : "f"(x));
  return y;
}
__device__ inline uint32_t bf16x2_rn(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// 32 values a lane summed over the warp: lane l gets the sum of value l (31 shuffles).
__device__ inline float butterfly_sum(float (&v)[32], int lane) {
#pragma unroll
  for (int half = 16; half >= 1; half >>= 1) {
    const bool up = lane & half;
#pragma unroll
    for (int i = 0; i < half; ++i) {
      const float keep = up ? v[half + i] : v[i], give = up ? v[i] : v[half + i];
      v[i] = keep + __shfl_xor_sync(0xFFFFFFFFu, give, half);
    }
  }
  return v[0];
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

// One piece of a tile's work: what its rows see, as a list of positions (first the sinks
// that the window has left behind, then the window of all its tokens), cut into blocks of 128.
struct Piece {
  int seq, from, len, ctx;      // sequence: first query token, query tokens, context
  int row0;                     // first row in the sequence
  int lo, ns, nv;               // first position of the window; sinks before it; positions of the list
  int blk, n;                   // blocks of this piece
  __device__ int pos(int v) const { return v < ns ? v : lo + v - ns; }     // of list entry v < nv
};

struct Walk {
  const WindowArgs& a;
  int b, base, nt, from, len, lane;                  // sequence, tiles before it, its tiles
  __device__ Walk(const WindowArgs& args, int l) : a(args), b(-1), base(0), nt(0), from(0), len(0), lane(l) {}
  // Goes on to the sequence of tile t (not before the present one), 32 sequences at a time.
  __device__ bool seek(int t) {
    if (t < base + nt) return true;
    int at = base + nt;
    for (int b0 = b + 1; b0 < a.batch; b0 += 32) {
      const int i = b0 + lane;
      int f = 0, l = 0, k = 0;
      if (i < a.batch) {
        f = __ldg(a.q_start + i);
        l = __ldg(a.q_start + i + 1) - f;
        k = tiles_of(a, l);
      }
      int x = k;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xFFFFFFFFu, x, o);
        if (lane >= o) x += y;
      }
      const uint32_t past = __ballot_sync(0xFFFFFFFFu, at + x > t);
      if (past) {
        const int w = __ffs(past) - 1;
        b = b0 + w;
        nt = __shfl_sync(0xFFFFFFFFu, k, w);
        base = at + __shfl_sync(0xFFFFFFFFu, x, w) - nt;
        from = __shfl_sync(0xFFFFFFFFu, f, w);
        len = __shfl_sync(0xFFFFFFFFu, l, w);
        return true;
      }
      at += __shfl_sync(0xFFFFFFFFu, x, 31);
    }
    return false;
  }
  // Piece s of n of tile t.
  __device__ bool piece(int t, int s, int n, Piece& p) {
    if (!seek(t)) return false;
    p.seq = b;
    p.from = from;
    p.len = len;
    p.ctx = context(a, b);
    p.row0 = (t - base) * kWinRows;
    const int tok0 = p.row0 / a.d.heads, tok1 = min(len - 1, (p.row0 + kWinRows - 1) / a.d.heads);
    const int last = p.ctx - len + tok1;
    p.lo = max(0, p.ctx - len + tok0 - a.window + 1);
    p.ns = min(a.sinks, p.lo);
    p.nv = last < 0 ? 0 : p.ns + last + 1 - p.lo;
    const int nb = (p.nv + kWinPos - 1) / kWinPos;
    p.blk = nb * s / n;
    p.n = nb * (s + 1) / n - p.blk;
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
__device__ __noinline__ void hide_values(uint8_t* base, int e) {
  bool whole = true;
#pragma unroll 1
  for (int c = 0; c < 64; ++c) {
    const uint4 x = *reinterpret_cast<const uint4*>(base + (c >> 3) * kKReg + tc::sw128_offset(e, c & 7));
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) whole = whole && (w[i] & 0x7F80u) != 0x7F80u && (w[i] & 0x7F800000u) != 0x7F800000u;
  }
  if (whole) return;
#pragma unroll 1
  for (int c = 0; c < 64; ++c)
    *reinterpret_cast<uint4*>(base + (c >> 3) * kKReg + tc::sw128_offset(e, c & 7)) = make_uint4(0, 0, 0, 0);
}

struct Span {
  int first, units, step, pieces;                    // the CTA's units: first, first + step, ... below units
};

// Copies queries and cache rows.  A lane has four rows of a block.
__device__ inline void load_role(const WindowArgs& a, WinSmall& sm, uint8_t* base, const Span& w, int lane,
                                 const CUtensorMap* qmap, const CUtensorMap* kmap) {
  Walk walk(a, lane);
  Piece p;
  const int none = int(a.page_table ? a.d.num_pages * kPage : int64_t(a.batch) * a.d.max_ctx);   // a row outside: zeros
  const uint32_t k0 = tc::smem_u32(base) + lane * 512;
  uint32_t nq = 0, nk = 0;
  for (int u = w.first; u < w.units; u += w.step) {
    if (!walk.piece(u / w.pieces, u % w.pieces, w.pieces, p)) return;
    for (int j = 0; j < p.n; ++j, ++nk) {
      int y[4];
      bool lost = false;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int v = (p.blk + j) * kWinPos + 4 * lane + i;
        y[i] = none;
        if (v < p.nv) {
          const int r = row_of(a, p.seq, p.pos(v));
          if (r >= 0) y[i] = r;
          else lost = true;
        }
      }
      if (lost) raise_err(a.ws, CSA2_DEV_PAGE_ID);
      if (j == 0) {
        if (!wait_warp(sm, &sm.q_empty, (nq & 1) ^ 1, a.ws)) return;
        if (lane == 0) tc::mbar_expect_tx(&sm.q_full, kQBytes);
        __syncwarp();
        if (lane < 9)
          tc::tma_load_2d(qmap, base + kQOff + lane * kQReg, 64 * lane, p.from * a.d.heads + p.row0, &sm.q_full);
        ++nq;
      }
#pragma unroll 1
      for (int g = 0; g < kGroups; ++g) {
        if (!wait_warp(sm, &sm.k_empty[g], (nk & 1) ^ 1, a.ws)) return;
        const int regions = g < 4 ? 2 : 1;
        if (lane == 0) tc::mbar_expect_tx(&sm.k_full[g], uint32_t(regions * kKReg));
        __syncwarp();
        for (int r = 2 * g; r < 2 * g + regions; ++r)
          tma_gather4(kmap, k0 + r * kKReg, 64 * r, make_int4(y[0], y[1], y[2], y[3]), &sm.k_full[g]);
      }
    }
  }
}

// Issues the products.
__device__ inline void mma_role(const WindowArgs& a, WinSmall& sm, uint8_t* base, const Span& w, int lane, uint32_t tmem) {
  constexpr uint32_t id_s = tc::idesc_bf16(kWinPos, kWinRows, 0, 0);
  constexpr uint32_t id_o = tc::idesc_bf16(kWinPos, kWinRows, 1, 1);
  const uint32_t k_at = tc::smem_u32(base);
  const uint64_t ks = tc::smem_desc(k_at, 16, 1024, 2), qs = tc::smem_desc(k_at + kQOff, 16, 1024, 2);
  const uint64_t vs = tc::smem_desc(k_at, kKReg, 1024, 2), ps = tc::smem_desc(k_at + kPOff, kKReg, 1024, 2);
  const bool leader = elect_one();
  Walk walk(a, lane);
  Piece p;
  uint32_t nq = 0, nk = 0;
  for (int u = w.first; u < w.units; u += w.step) {
    if (!walk.piece(u / w.pieces, u % w.pieces, w.pieces, p)) return;
    if (p.n == 0) continue;
    if (!wait_warp(sm, &sm.q_full, nq & 1, a.ws)) return;
    for (int j = 0; j < p.n; ++j, ++nk) {
#pragma unroll 1
      for (int g = 0; g < kGroups; ++g) {
        if (!wait_warp(sm, &sm.k_full[g], nk & 1, a.ws)) return;
        tc::tc_fence_after_sync();
        if (leader) {
          const int last = g < 4 ? 8 : 4;
          for (int i = 0; i < last; ++i) {
            const uint32_t kb = 2 * g + (i >> 2), off = (i & 3) * 32;
            tc::mma_bf16(tmem, ks + ((kb * kKReg + off) >> 4), qs + ((kb * kQReg + off) >> 4), id_s, g + i > 0);
          }
        }
        __syncwarp();
      }
      if (leader) {
        tc::mma_commit(&sm.s_full);
        if (j == p.n - 1) tc::mma_commit(&sm.q_empty);
      }
      __syncwarp();
      if (!wait_warp(sm, &sm.p_full, nk & 1, a.ws)) return;
      if (j == 0 && !wait_warp(sm, &sm.o_empty, (nq & 1) ^ 1, a.ws)) return;
      tc::tc_fence_after_sync();
      if (leader) {
#pragma unroll 1
        for (int mt = 0; mt < 4; ++mt) {
#pragma unroll
          for (int k = 0; k < 8; ++k)
            tc::mma_bf16(tmem + kOCol + 64 * mt, vs + ((2 * mt * kKReg + k * 2048) >> 4), ps + ((k * 2048) >> 4), id_o, j + k > 0);
          tc::mma_commit(&sm.k_empty[mt]);
        }
        tc::mma_commit(&sm.k_empty[4]);
        if (j == p.n - 1) tc::mma_commit(&sm.o_full);
      }
      __syncwarp();
    }
    ++nq;
  }
}

// Softmax over a block's positions (tensor-memory lanes) and the outputs.  Warp rw has the
// lanes 32 (rw % 4) .. + 31 and the rows 32 (rw / 4) .. + 31; lane i keeps the state of row i of
// these (alike in the four warps of a half, but for the sum, which is of its own lanes).
// A wait that gives up leaves the warp in the loop, without waits or results: its hardware
// barriers have no limit, and all eight warps pass the same ones.
__device__ inline void row_role(const WindowArgs& a, WinSmall& sm, uint8_t* base, const Span& w, int rw, int lane,
                                uint32_t tmem) {
  const int quarter = rw & 3, half = rw >> 2, e = 32 * quarter + lane;
  const uint32_t lanes = tmem + (uint32_t(32 * quarter) << 16) + uint32_t(32 * half);
  const float c2 = a.scale * 1.4426950408889634f;
  uint8_t* stage = base + kStageOff + rw * kStageWarp;
  bool dead = false;
  Walk walk(a, lane);
  Piece p;
  uint32_t nq = 0, nk = 0;
  for (int u = w.first; u < w.units; u += w.step) {
    if (!walk.piece(u / w.pieces, u % w.pieces, w.pieces, p)) return;
    const int lr = p.row0 + 32 * half + lane, rows = p.len * a.d.heads;
    const int mine = lr < rows ? p.ctx - p.len + lr / a.d.heads : -1;       // position of the lane's row
    __syncwarp();
    sm.pos[rw][lane] = mine;
    __syncwarp();
    const int p_max = __reduce_max_sync(0xFFFFFFFFu, mine);
    const int p_min = __reduce_min_sync(0xFFFFFFFFu, lr < rows ? mine : p_max);
    float ref = -INFINITY, sum = 0.0f;
    for (int j = 0; j < p.n; ++j, ++nk) {
      const int v = (p.blk + j) * kWinPos + e;
      int t = v < p.nv ? p.pos(v) : -1;
      if (t >= 0 && row_of(a, p.seq, t) < 0) t = -1;
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
          const int4 pr = reinterpret_cast<const int4*>(sm.pos[rw])[i4];
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
        if (odd) hide_values(base, e);
      }
      float top = -INFINITY;
#pragma unroll
      for (int i = 0; i < 32; ++i) {
        const float m = max_over_warp(x[i]);
        if (lane == i) top = m;
      }
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
      sm.ref[rw][lane] = ref == -INFINITY ? 0.0f : ref;
      const bool turn = __any_sync(0xFFFFFFFFu, alpha != 1.0f);
      if (turn) sm.alpha[rw][lane] = alpha;
      __syncwarp();
      if (turn) {
        // the outputs so far to the new reference (the block's rope channels, which the scores
        // waited for, came after the last product)
        sum *= alpha;
#pragma unroll 1
        for (int mt = 0; mt < 4; ++mt)
#pragma unroll 1
          for (int c = 0; c < 32; c += 8) {
            float o[8];
            tc::tmem_ld8(lanes + kOCol + 64 * mt + c, o);
#pragma unroll
            for (int i = 0; i < 8; ++i) o[i] *= sm.alpha[rw][c + i];
            tc::tmem_st8(lanes + kOCol + 64 * mt + c, o);
          }
      }
#pragma unroll
      for (int i8 = 0; i8 < 4; ++i8) {
        uint32_t pk[4];
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          const float4 r4 = reinterpret_cast<const float4*>(sm.ref[rw])[2 * i8 + k];
          const int i = 8 * i8 + 4 * k;
          x[i] = ex2(x[i] - r4.x);
          x[i + 1] = ex2(x[i + 1] - r4.y);
          x[i + 2] = ex2(x[i + 2] - r4.z);
          x[i + 3] = ex2(x[i + 3] - r4.w);
          pk[2 * k] = bf16x2_rn(x[i], x[i + 1]);
          pk[2 * k + 1] = bf16x2_rn(x[i + 2], x[i + 3]);
        }
        *reinterpret_cast<uint4*>(base + kPOff + tc::sw128_offset(e, 4 * half + i8)) = make_uint4(pk[0], pk[1], pk[2], pk[3]);
      }
      tc::fence_proxy_async_smem();
      tc::tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) arrive(&sm.p_full);
      sum += butterfly_sum(x, lane);
    }
    // outputs: sums of the four lane quarters, joined with the other attention's
    const bool join = a.prev_out != nullptr && w.pieces == 1;
    const int64_t row0 = int64_t(p.from) * a.d.heads + p.row0 + 32 * half;
    float prev = -INFINITY;
    if (join && lr < rows) prev = a.prev_lse[row0 + lane];
    sm.sum[quarter][32 * half + lane] = sum;
    bar_sync(1 + half, 128);
    float total = 0.0f;
#pragma unroll
    for (int k = 0; k < 4; ++k) total += sm.sum[k][32 * half + lane];
    float own = total != 0.0f ? 1.0f / total : 0.0f, other = 0.0f;
    float lse = total != 0.0f ? ((ref == -INFINITY ? 0.0f : ref) + log2f(total)) * 0.6931471805599453f : -INFINITY;
    if (join && prev != -INFINITY) {
      const float most = fmaxf(lse, prev), x0 = expf(lse - most), x1 = expf(prev - most);
      own *= x0 / (x0 + x1);
      other = x1 / (x0 + x1);
      lse = most + logf(x0 + x1);
    }
    if (p.n > 0) {
      if (!dead && !wait_warp(sm, &sm.o_full, nq & 1, a.ws)) dead = true;
      tc::tc_fence_after_sync();
    }
    sm.ref[rw][lane] = own;
    sm.alpha[rw][lane] = other;
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
              if (p.row0 + 32 * half + i < rows) dst[i * kLatent] = o[i] * sm.ref[rw][i];
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
        } else {
#pragma unroll
          for (int i = 0; i < 32; ++i) o[i] = 0.0f;
        }
        // 8 rows x 32 channels at a time through shared memory: 64 bytes of a row for four lanes
        const int ch = 128 * mt + 32 * quarter + 8 * (lane & 3);
#pragma unroll
        for (int i8 = 0; i8 < 4; ++i8) {
          const int r = 8 * i8 + (lane >> 2);
          const bool have = p.row0 + 32 * half + r < rows;
          const int64_t at = (row0 + r) * kLatent + ch;
          __syncwarp();
          if (join) {
            uint4 v = make_uint4(0, 0, 0, 0);
            if (have) v = *reinterpret_cast<const uint4*>(a.prev_out + at);
            *reinterpret_cast<uint4*>(stage + lane * 16) = v;
            __syncwarp();
          }
          uint16_t* col = reinterpret_cast<uint16_t*>(stage) + lane;
#pragma unroll
          for (int k = 0; k < 8; ++k) {
            const int i = 8 * i8 + k;
            float y = p.n > 0 ? o[i] * sm.ref[rw][i] : 0.0f;
            if (join) {
              const float f = sm.alpha[rw][i];
              if (f != 0.0f) y = fmaf(f, bf16_to_f32(col[32 * k]), y);
            }
            col[32 * k] = uint16_t(bf16x2_rn(y, 0.0f));
          }
          __syncwarp();
          if (have) *reinterpret_cast<uint4*>(a.out + at) = *reinterpret_cast<const uint4*>(stage + lane * 16);
        }
      }
    }
    if (p.n > 0) {
      tc::tc_fence_before_sync();
      __syncwarp();
      if (lane == 0) arrive(&sm.o_empty);
      ++nq;
    }
    bar_sync(1 + half, 128);                         // the sums have been read
  }
}

__global__ void __launch_bounds__(kWinThreads, 1)
    window_kernel(const __grid_constant__ WindowArgs a, const __grid_constant__ CUtensorMap qmap,
                  const __grid_constant__ CUtensorMap kmap) {
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
    tc::mbar_init(&sm.q_full, 1);
    tc::mbar_init(&sm.q_empty, 1);
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
  w.first = blockIdx.x;
  w.units = tiles * w.pieces;
  w.step = grid;
  if (blockIdx.x == 0 && tid == 0) {
    if (sm.bad) raise_err(a.ws, CSA2_DEV_Q_START);
    a.head[0] = tiles;
    a.head[1] = w.pieces;
  }
  if (wid < kRowWarps) row_role(a, sm, base, w, wid, lane, tmem);
  else if (wid == kMmaWarp) mma_role(a, sm, base, w, lane, tmem);
  else load_role(a, sm, base, w, lane, &qmap, &kmap);
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
  CUtensorMap q, kv;
  const auto enc = tensor_map_encoder();
  const uint64_t rows = a.page_table ? uint64_t(a.d.num_pages) * kPage : uint64_t(a.batch) * uint64_t(a.d.max_ctx);
  if (!encode_2d_cached(enc, &q, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.q, kDqk, uint64_t(a.total_q) * a.d.heads, kDqk * 2,
                        64, kWinRows, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B) ||
      !encode_2d_cached(enc, &kv, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, a.kv, kDqk, rows, kDqk * 2, 64, 1,
                        CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B))
    return cudaErrorUnknown;
  static KernelAttrs attrs;
  cudaError_t e = prepare_kernel(window_kernel, size_t(kWinSmem), false, attrs);
  if (e != cudaSuccess) return e;
  // bounds of what the device will find: tiles, and blocks of one
  const int H = a.d.heads, span = kWinRows % H == 0 ? kWinRows / H : (H + 62) / H + 1;
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
                (e = launch_pdl(window_kernel, dim3(unsigned(grid)), dim3(kWinThreads), size_t(kWinSmem), st, 1, a, q, kv)));
  if (e != cudaSuccess || !a.may_split) return e;
  CSA2_PROFILED(st, "window_merge",
                (e = launch_pdl(window_merge_kernel, dim3(kWinRows / kMergeRows, unsigned(min64(tiles, grid / 2))),
                                dim3(kMergeThreads), 0, st, 1, a)));
  return e;
}

}  // namespace csa2
