// Sizes and layouts of the 8-bit base products, shared by the host side and
// the kernels (no HIP types: the argument checks compile without HIP).
#pragma once
#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

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
  int tile;     // rows and outputs per workgroup of the many-rows kernel; 0: the few-rows kernel
  int rt, nt;   // few rows: tiles of 16 outputs and of 16 rows of a workgroup
  size_t q, s;  // rounded rows and their scales
  size_t ws_bytes;
};
// Rows and values that a workgroup of the few-rows kernel rounds by itself, at
// most: what its registers hold.  Rounded so, and by a kernel before, us a call:
//                            in a graph     on its own
//     1 row  3584 ->   512    4.4   6.3     9.0  13.9
//     1 row  3584 -> 18944   13.1  15.3    13.5  16.5
//     1 row  4096 -> 65536   45.2  48.5    45.6  49.1
//     4 rows 5120 -> 18944   20.1  22.4    20.5  22.7
//     5 rows 3584 ->  3584    7.9   8.1     8.7  13.0
//     5 rows 4096 ->  4096    9.4   9.9     9.8  13.3  (float32 9.3, 9.8; 10.0, 12.9)
//     5 rows 4096 -> 32768   25.0  28.2    25.3  28.4
//     8 rows  512 ->   512    4.2   5.2     8.6  13.2
//     8 rows 2048 ->  2048    6.2   6.1     8.5  13.2
//     8 rows 2048 -> 32768   12.9  15.3    13.3  15.9
//    12 rows 1280 ->  4096    6.4   5.9     8.5  13.3
//    12 rows 1280 -> 32768   12.1  12.2    12.4  13.3
//    16 rows 1024 ->  4096    6.2   6.0     8.7  13.2
//    16 rows 1024 -> 33000   15.1  12.4    15.2  13.4
// So it is slower in a graph for 12 to 16 short rows, by 0.5 us, and by 2.7 where
// they meet very many outputs.
constexpr int kW8FusedRows = 16;
constexpr int kW8FusedValues = 5 * 8 * 512;  // kHold pieces of 8 per thread (w8_rows.hip)

constexpr int kW8BigTile = 256, kW8MidTile = 128, kW8SmallTile = 64;  // small: of the few-rows kernel

// What a kernel with tiles of `tile` rows and outputs takes, in us, up to a
// constant.  Workgroups run one to a compute unit, so in rounds of 256; one's
// time goes with its tiles of inputs, and faster the emptier the round.  The
// constants are fitted to times measured at 48 to 3000 rows of ten shapes from
// 512 -> 2048 to 18944 -> 3584 (us, small, mid, big): 256 rows 3584 -> 3584 10.6,
// 16.8, 37.6; 512 rows 19.0, 17.4, 37.8; 1024 rows 34, 18.8, 38.5; 1024 rows 3584
// -> 14336 151, 72, 51; 2048 rows 286, 124, 95; 200 rows 2048 -> 8192 15.0, 12.1,
// 24.3; 3000 rows 18944 -> 3584 420, 243, 193.
inline double w8_many_us(int tile, int T, int d_out, int kt) {
  const double empty = tile == kW8BigTile ? 0.52 : (tile == kW8MidTile ? 0.17 : 0.055);
  const double load = tile == kW8BigTile ? 0.27 : (tile == kW8MidTile ? 0.09 : 0.055);
  const double start = tile == kW8BigTile ? 4.0 : 4.5;
  const int64_t groups = (int64_t)((T + tile - 1) / tile) * ((d_out + tile - 1) / tile), full = groups / 256, rest = groups % 256;
  return (double)full * (kt * (empty + load) + start) + (rest > 0 ? kt * (empty + load * (double)rest / 256.) + start : 0.);
}

inline W8Plan w8_plan_call(int d_in, int d_out, int T, bool quantized) {
  W8Plan p{};
  if (T <= 0) return p;
  const int64_t per_row = ((int64_t)d_in + 511) / 512 * 512;
  const int blocks = w8_blocks(d_out);
  if (T > 32) {
    // The smallest tiles that give every compute unit one workgroup at most; the
    // largest ones where none do, if the many-rows kernel does not take less.
    // (rows x outputs, us) 64 rows 3584 -> 512 16 x 32 4.0, 32 x 32 4.4, 32 x 64 5.6,
    // 64 x 64 7.6; 64 rows 3584 -> 3584 7.3, 6.3, 7.6, 10.6; 128 rows 11.0, 8.7, 7.8,
    // 10.5; 256 rows 17.1, 14.0, 11.9, 10.8; 48 rows 18944 -> 3584 25.6, 16.7, 22.2, 31.5.
    p.rt = p.nt = 4;
    for (const int shape : {21, 22, 42}) {
      const int rt = shape / 10, nt = shape % 10;
      if ((int64_t)blocks * (4 / rt) * ((T + 16 * nt - 1) / (16 * nt)) > 256) continue;
      p.rt = rt;
      p.nt = nt;
      break;
    }
    if (p.nt == 4) {
      const int kt = w8_k_tiles(d_in);
      const double small = w8_many_us(kW8SmallTile, T, d_out, kt), mid = w8_many_us(kW8MidTile, T, d_out, kt),
                   big = w8_many_us(kW8BigTile, T, d_out, kt);
      if (small > mid || small > big) p.tile = mid < big ? kW8MidTile : kW8BigTile;
    }
  } else {
    p.nt = T <= 16 ? 1 : 2;
    // Tiles of outputs per workgroup: more share the rows' loads, fewer give
    // every compute unit work.
    const int64_t tiles = (int64_t)blocks * 4;
    p.rt = tiles < 512 ? 1 : (tiles < 2048 ? 2 : 4);
  }
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
