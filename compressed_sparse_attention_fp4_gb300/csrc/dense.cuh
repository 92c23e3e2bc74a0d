// dense.cuh -- arguments and workspace layout of the dense chunk attention.
#pragma once

#include "common.cuh"

namespace csa2 {

constexpr int kDenseTile = 128;          // rows (query token, head) of a tile
constexpr int kDenseBlk = 64;            // positions of a block: one page
constexpr int kDenseMaxClusters = 76;    // CTA pairs: one CTA on each of 152 SMs
constexpr int kDenseMinBlocks = 4;       // least blocks a run is cut to (one SM pair fills in ~1 us a block; a cut costs a merge)
static_assert(kDenseBlk == kPage, "a block never crosses a page");

struct DensePlan {
  int4* head;          // tiles, runs in use, blocks (low, high word)
  int4* runs;          // per cluster: first tile, blocks of it before the run, blocks
  int4* seqs;          // per sequence: first tile, first query, queries, context
  int4* tiles;         // two per tile (see Item)
  int64_t* before;     // per tile: blocks before it
};

struct DenseArgs {
  csa2_dims d;
  int batch, total_q, causal, window, clusters;
  int tile;            // rows of a tile: 128, or 256 on twice the SMs
  int max_tiles;       // bound of their number
  const uint16_t* q;
  const int32_t* q_start;
  const uint8_t* codes;
  const uint8_t* scales;
  const uint16_t* rope;
  const int32_t* page_table;
  const int32_t* ctx_len;
  float scale;
  uint16_t* out;
  float* lse;
  uint8_t* ws;
  DensePlan plan;
  float* part_o;       // [2 * clusters * tile / 128][512][128]
  float* part_lse;     // [2 * clusters * tile / 128][128]
};

// Byte offsets in the workspace: error word, plan, partial outputs.
struct DenseLayout {
  int64_t head, runs, seqs, tiles, before, part_lse, part_o, total;
};

inline DenseLayout make_dense_layout(const csa2_dims& d, int64_t batch, int64_t total_q) {
  DenseLayout L;
  int64_t off = 256;
  const int64_t tiles = (total_q * d.heads + kDenseTile - 1) / kDenseTile + batch;
  L.head = off;     off += 256;
  L.runs = off;     off = align256(off + kDenseMaxClusters * 16);
  L.seqs = off;     off = align256(off + batch * 16);
  L.tiles = off;    off = align256(off + tiles * 32);
  L.before = off;   off = align256(off + tiles * 8);
  L.part_lse = off; off = align256(off + int64_t(2 * kDenseMaxClusters) * kDenseTile * 4);
  L.part_o = off;   off = align256(off + int64_t(2 * kDenseMaxClusters) * kDenseTile * kLatent * 4);
  L.total = off;
  return L;
}

// Whether a call takes tiles of 256 rows on 4 SMs instead of 128 on 2: from 128 rows a
// sequence on (mean).  Measured, 64 heads, 128- against 256-row tiles: 1 token (64 rows),
// 8 contexts of 128K 311 / 349 us; 2 tokens on 8,000 positions 46.9 / 45.3; 1 to 5 tokens on
// up to 16,384 (16 sequences) 101 / 88; 8 tokens on 16,000 (8 sequences) 164 / 113;
// prompts of 301 to 2,000 tokens 546 / 426.  The larger tile widens each block once for
// twice the rows.
inline bool dense_pairs(int heads, int batch, int64_t total_q) { return total_q * heads >= int64_t(128) * batch; }

cudaError_t launch_dense(DenseArgs a, cudaStream_t st);

}  // namespace csa2
