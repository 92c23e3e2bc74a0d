// window_tiles.cuh -- the tiles of a window attention call: what its kernels find out about the batch on
// the device.
#pragma once

#include <cuda.h>

#include "common.cuh"
#include "window.cuh"

namespace csa2 {

// Context of sequence b (bad ones are reported by the first CTA's count, and taken as 0).
__device__ inline int context(const WindowArgs& a, int b) {
  const int n = __ldg(a.ctx_len + b);
  return n < 0 || n > a.d.max_ctx || (a.page_table && n > int64_t(a.d.max_pages) * kPage) ? 0 : n;
}
// Row number over heads: a.by_heads = ceil(2^64 / heads), exact below 2^31 rows (0 for one head).
__device__ inline int over_heads(const WindowArgs& a, int row) { return a.by_heads ? int(__umul64hi(uint64_t(row), a.by_heads)) : row; }
// Tiles of a sequence of len tokens: kRows rows each.
template <int kRows>
__device__ inline int tiles_of(const WindowArgs& a, int len) { return (len * a.d.heads + kRows - 1) / kRows; }
// Most tokens of a tile.
__host__ __device__ inline int tile_tokens(int heads, int rows) { return rows % heads == 0 ? rows / heads : (heads + rows - 2) / heads + 1; }

// Cache row of position t (-1: its page id is out of range).
__device__ inline int row_of(const WindowArgs& a, int seq, int t) {
  if (!a.page_table) return int(int64_t(seq) * a.d.max_ctx + t);
  const int pg = __ldg(a.page_table + int64_t(seq) * a.d.max_pages + t / kPage);
  return pg < 0 || pg >= a.d.num_pages ? -1 : pg * kPage + t % kPage;
}

// 32 sequences, one a lane: from b0 on, with `base` tiles before them.
template <int kRows>
struct Sequences {
  int b0, base, from, len, ctx, upto;
  __device__ void load(const WindowArgs& a, int lane) {
    const int i = b0 + lane;
    from = len = ctx = upto = 0;
    if (i < a.batch) {
      from = __ldg(a.q_start + i);
      len = __ldg(a.q_start + i + 1) - from;
      ctx = context(a, i);
      upto = tiles_of<kRows>(a, len);
    }
  }
  __device__ void count(int lane) {
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xFFFFFFFFu, upto, o);
      if (lane >= o) upto += y;
    }
  }
};

// Tokens of one tile see the positions lo .. last and the sinks before lo.
struct Tile {
  int row, have;                // first row of q, rows (kRows, or what is left of the sequence)
  int seq;
  int lo, last;
  int pos, rem;                 // the first row's token position and head
};
// Tile t, not before those asked for so far; `q`: sequences up to it, counted.  For a whole warp.
template <int kRows>
__device__ inline Tile find_tile(const WindowArgs& a, Sequences<kRows>& q, int t, int lane) {
  Tile p;
  uint32_t past;
  while ((past = __ballot_sync(0xFFFFFFFFu, q.base + q.upto > t)) == 0) {
    if (q.b0 >= a.batch) return {0, 0, 0, 0, -1, 0, 0};                // the starts have changed since they were counted
    q.base += __shfl_sync(0xFFFFFFFFu, q.upto, 31);
    q.b0 += 32;
    q.load(a, lane);
    q.count(lane);
  }
  const int i = __ffs(past) - 1;
  const int tokens = __shfl_sync(0xFFFFFFFFu, q.len, i), c = __shfl_sync(0xFFFFFFFFu, q.ctx, i);
  const int before = i > 0 ? __shfl_sync(0xFFFFFFFFu, q.upto, i - 1) : 0;
  const int r0 = (t - q.base - before) * kRows, tok0 = over_heads(a, r0);
  const int tok1 = min(tokens - 1, over_heads(a, r0 + kRows - 1));
  p.row = __shfl_sync(0xFFFFFFFFu, q.from, i) * a.d.heads + r0;
  p.have = min(kRows, tokens * a.d.heads - r0);
  p.seq = q.b0 + i;
  p.pos = c - tokens + tok0;
  p.rem = r0 - tok0 * a.d.heads;
  p.last = c - tokens + tok1;
  p.lo = max(0, p.pos - a.window + 1);
  return p;
}

// Logits in base 2 per score (but for its sign; not 0, which would make NaN of a masked score).
__device__ inline float score_to_log2(const WindowArgs& a) { return fmaxf(fabsf(a.scale) * 1.4426950408889634f, 1.17549435e-38f); }

// Whether four 32-bit words hold eight finite bf16 values.
__device__ inline bool bf16x8_finite(uint4 x) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  bool finite = true;
#pragma unroll
  for (int i = 0; i < 4; ++i) finite = finite && (w[i] & 0x7F80u) != 0x7F80u && (w[i] & 0x7F800000u) != 0x7F800000u;
  return finite;
}

// Pages of 64 positions that a tile sees: `sinks` of them first, then the window's.
struct TilePages {
  int sinks, all;
};
__device__ inline TilePages pages_of(const WindowArgs& a, int lo, int last) {
  const int sp = min((a.sinks + kPage - 1) / kPage, lo / kPage);
  return {sp, last < 0 ? 0 : sp + last / kPage - lo / kPage + 1};
}

// Maps of window_long.cu: boxes of 64 channels x 32 rows (queries, keys) or 64 (values).
struct WindowLongMaps {
  CUtensorMap q, keys, values;
};
int window_long_clusters(bool join);
cudaError_t launch_window_long(const WindowArgs& a, const WindowLongMaps& m, int64_t tiles, cudaStream_t st);

}  // namespace csa2
