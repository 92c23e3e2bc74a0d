// window.cuh -- arguments and workspace layout of the window attention.
#pragma once

#include "common.cuh"

namespace csa2 {

constexpr int kWinRows = 64;             // rows (query token, head) of a tile: the MMA's N
constexpr int kLongRows = 256;          // rows of a tile of window_long.cu
constexpr int kWinPos = 128;             // cache positions of a block: the MMA's M
// How far (base 2) a block's maximum may pass a row's reference before the outputs so far are rescaled.  Weights
// up to 2^16 cost no precision, only range: with 2^20 positions, values up to 2^91 stay within fp32.
constexpr float kWinSlack = 16.0f;
constexpr int kWinMaxCtas = 152;         // most pieces of a call whose tiles are split

struct WindowArgs {
  csa2_dims d;
  int batch, total_q, window, sinks;
  int may_split;       // pieces of few tiles may be split and merged
  uint64_t by_heads;   // see over_heads
  const uint16_t* q;
  const int32_t* q_start;
  const uint16_t* kv;
  const int32_t* page_table;
  const int32_t* ctx_len;
  float scale;
  const uint16_t* prev_out;
  const float* prev_lse;
  uint16_t* out;
  float* lse;
  uint8_t* ws;
  int* head;           // tiles and pieces a tile, as the attention kernel found them
  int2* tiles;         // [kWinMaxCtas] first row and rows of a tile
  float* part_lse;     // [kWinMaxCtas][64]
  float* part_o;       // [kWinMaxCtas][64][512]
};

// Byte offsets in the workspace: error word, then what a call with split tiles leaves for its merge.
struct WindowLayout {
  int64_t head, tiles, part_lse, part_o, total;
};

inline WindowLayout make_window_layout() {
  WindowLayout L;
  int64_t off = 256;
  L.head = off;     off += 256;
  L.tiles = off;    off = align256(off + kWinMaxCtas * 8);
  L.part_lse = off; off = align256(off + int64_t(kWinMaxCtas) * kWinRows * 4);
  L.part_o = off;   off = align256(off + int64_t(kWinMaxCtas) * kWinRows * kLatent * 4);
  L.total = off;
  return L;
}

cudaError_t launch_window(WindowArgs a, cudaStream_t st);

}  // namespace csa2
