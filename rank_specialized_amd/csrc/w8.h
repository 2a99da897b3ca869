// Sizes and layouts of the 8-bit base products, shared by the host side and
// the kernels (no HIP types: the argument checks compile without HIP).
#pragma once
#include <stddef.h>
#include <stdint.h>

#include "../../include/lora.h"
#include "plan.h"

namespace lora {

// Codes are laid out in tiles of 16 outputs x 64 inputs, 1 KiB each: lane l of
// a wave holds output l % 16 of the tile and, with h = l / 16, its inputs
// 16 h .. + 15, one operand of a 16 x 16 x 64 integer product.  Four tiles make
// a block of 64 outputs x 64 inputs, and a block's tiles follow one another,
// then the blocks over the inputs.  Output i of tile b of a block is
//
//   32 (b / 2) + 8 (i / 4) + 4 (b % 2) + i % 4,
//
// so that a lane, which holds four consecutive rows of a product in its
// accumulators, has eight consecutive outputs in two tiles: 16 bytes of bf16.
// Inputs past d_in and outputs past d_out hold code 0.
constexpr int kW8Block = 64;  // outputs of a block
constexpr int kW8K = 64;      // inputs of a tile
constexpr int kW8TileBytes = 1024;
constexpr int kW8BlockBytes = 4 * kW8TileBytes;
constexpr int w8_output(int b, int i) { return 32 * (b >> 1) + 8 * (i >> 2) + 4 * (b & 1) + (i & 3); }

inline int w8_blocks(int d_out) { return (d_out + kW8Block - 1) / kW8Block; }
inline int w8_k_tiles(int d_in) { return (d_in + kW8K - 1) / kW8K; }
inline int64_t w8_code_bytes(int d_in, int d_out) { return (int64_t)w8_blocks(d_out) * w8_k_tiles(d_in) * kW8BlockBytes; }
inline int64_t w8_scale_bytes(int d_out) { return (int64_t)w8_blocks(d_out) * kW8Block * 4; }

// A row of codes in a workspace.
inline int64_t w8_row_bytes(int d_in) { return ((int64_t)d_in + 15) / 16 * 16; }

// How a call is run, and the workspace it takes.
struct W8Plan {
  bool fused;   // few rows: each workgroup rounds them by itself
  bool many;    // the many-rows kernel
  int rt, nt;   // few rows: tiles of 16 outputs and of 16 rows of a workgroup
  size_t q, s;  // rounded rows and their scales
  size_t ws_bytes;
};
// Values that a workgroup of the few-rows kernel rounds by itself.
constexpr int kW8FusedRows = 4;
constexpr int kW8FusedValues = 5 * 8 * 512;  // kHold pieces of 8 per thread (w8_rows.hip)

inline W8Plan w8_plan_call(int d_in, int d_out, int T, bool quantized) {
  W8Plan p{};
  if (T <= 0) return p;
  const int64_t per_row = ((int64_t)d_in + 511) / 512 * 512;
  p.many = T > 256;
  p.nt = T <= 16 ? 1 : (T <= 32 ? 2 : 4);
  // Tiles of outputs per workgroup: more share the rows' loads, fewer give
  // every compute unit work.
  const int64_t tiles = (int64_t)w8_blocks(d_out) * 4 * ((T + 16 * p.nt - 1) / (16 * p.nt));
  p.rt = p.nt == 4 ? 4 : (tiles < 512 ? 1 : (tiles < 2048 ? 2 : 4));
  p.fused = !quantized && T <= kW8FusedRows && T * per_row <= kW8FusedValues;
  if (!quantized && !p.fused) {
    p.q = p.ws_bytes;
    p.ws_bytes += align_up((size_t)T * (size_t)w8_row_bytes(d_in), 256);
    p.s = p.ws_bytes;
    p.ws_bytes += align_up((size_t)T * 4, 256);
  }
  return p;
}

}  // namespace lora
