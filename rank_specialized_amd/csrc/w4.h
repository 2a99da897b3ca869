// Sizes and layouts of the 4-bit base products, shared by the host side and
// the kernels (no HIP types: the argument checks compile without HIP).
#pragma once
#include <stddef.h>
#include <stdint.h>

#include "../../include/lora.h"
#include "plan.h"

namespace lora {

// Codes are laid out in tiles of 16 outputs x 128 inputs, 1 KiB each: lane l
// of a wave owns output l % 16 and, with h = l / 16, the inputs
// 32 j + 8 h .. + 7 of matrix-core step j = 0..3, one dword per step (16
// bytes per lane).  So a tile is one 16-byte load per lane of consecutive
// addresses, and a lane's dword is exactly its operand of one 16 x 16 x 32
// product.  Inside a dword, input 2 i of the eight is nibble i of the low
// half and input 2 i + 1 nibble i of the high half, and the dword is rotated
// left by 3: nibble 0 then sits on bits 3..6 of each half, where "or" with
// 16.0 (bf16, step 1/8) or 128.0 (f16, step 1/8) makes the number 16 + q or
// 128 + q.
constexpr int kW4Rows = 16;
constexpr int kW4K = 128;
constexpr int kW4TileBytes = kW4Rows * kW4K / 2;

// How a group's scale and zero point are held: bf16 scales without zero
// points in 2 bytes, with them in 4 (the zero point as the bf16 of 16 + z),
// float32 scales in 8 (scale, 16 + z).
enum W4Param { kW4Bf16 = 0, kW4Bf16Zero = 1, kW4F32 = 2 };
inline int w4_param_kind(int scale_dtype, int has_zeros) {
  return scale_dtype == LORA_DTYPE_F32 ? kW4F32 : (has_zeros ? kW4Bf16Zero : kW4Bf16);
}
constexpr int w4_param_bytes(int kind) { return kind == kW4Bf16 ? 2 : (kind == kW4Bf16Zero ? 4 : 8); }

// Scales are held per `gran` inputs, the part of a group that divides a tile:
// gcd(group, 128), 32, 64 or 128.
inline int w4_sub(int group) {  // scales per tile row
  return group % 128 == 0 ? 1 : (group % 64 == 0 ? 2 : 4);
}

inline int w4_row_tiles(int d_out) { return (d_out + kW4Rows - 1) / kW4Rows; }
inline int w4_k_tiles(int d_in) { return (d_in + kW4K - 1) / kW4K; }
inline int64_t w4_tiles(int d_in, int d_out) { return (int64_t)w4_row_tiles(d_out) * w4_k_tiles(d_in); }
inline int64_t w4_tile_param_bytes(int kind, int sub) { return (int64_t)kW4Rows * sub * w4_param_bytes(kind); }
inline int64_t w4_code_bytes(int n, int d_in, int d_out) { return n * w4_tiles(d_in, d_out) * kW4TileBytes; }
inline int64_t w4_params_bytes(int n, int d_in, int d_out, int kind, int sub) {
  return n * w4_tiles(d_in, d_out) * w4_tile_param_bytes(kind, sub);
}

// The few-rows kernel holds its rows of x in LDS: per row k_tiles * 128 values
// as bf16, of float32 rows three such planes, and 16 bytes more, so that 16
// rows' pieces of one matrix-core step lie on all banks.  64 KiB, so that two
// workgroups fit a compute unit.
constexpr int kW4FewLds = 64 * 1024;
inline int w4_few_row_bytes(int dtype, int d_in) {
  return (dtype == LORA_DTYPE_BF16 ? 1 : 3) * w4_k_tiles(d_in) * kW4K * 2 + 16;
}
inline int w4_few_rows(int dtype, int d_in) { return kW4FewLds / w4_few_row_bytes(dtype, d_in); }

// How a call is run, and the workspace it takes.
struct W4Plan {
  bool sum_in_kernel;  // weighted rows: each token's matrices run through by one workgroup, no partial rows
  int bm;              // rows per tile of the many-rows kernel; 0: a few-rows kernel
  size_t part;         // float32 rows [R][d_out] of a weighted call that keeps them
  size_t xs, up;       // many rows: x as f16, the rows' powers of two
  size_t hist, perm, tiles;  // many rows by matrix: counts and the number of tiles, the order, the tiles
  size_t ws_bytes;
};
// Rows of a weighted call up to which a token's k products are one
// workgroup's sum (if its rows fit LDS).
constexpr int kW4SumRows = 32;
// Rows per tile of the many-rows kernel.  Larger tiles unpack a code for more
// rows; 128 rows no longer fit the registers.  Measured (64, 96, 112, 128
// rows): 8192 rows, 4096 -> 14336: 1089, 936, 1015, 1180 us; 32 experts of
// 512 rows, 2048 -> 2816: 284, 264, 292, 372 us; 64 experts of 256 rows, 1408
// -> 2048: 200, 207, 211, 283 us.
constexpr int kW4BigTile = 96, kW4SmallTile = 64;
constexpr int kW4BigRows = 384;  // rows per matrix from which the big tile is taken
// Tiles of at most bm rows that R rows of n matrices (and of none) cut into.
inline int64_t w4_max_tiles(int R, int n, int bm) { return plan_max_runs(R, n + 1, bm); }

inline W4Plan w4_plan_call(const lora_w4_store& s, int dtype, int T, int k, bool weighted) {
  W4Plan p{};
  if (T <= 0) return p;
  const int64_t R = (int64_t)T * (k > 0 ? k : 1);
  p.sum_in_kernel = weighted && R <= kW4SumRows && k <= w4_few_rows(dtype, s.d_in);
  const int64_t per = (R + s.n - 1) / s.n;  // rows per matrix, on average
  const int64_t xs_bytes = R * w4_k_tiles(s.d_in) * kW4K * 2;  // 32-bit offsets
  if (dtype == LORA_DTYPE_BF16 && !p.sum_in_kernel && per > 32 && xs_bytes < ((int64_t)1 << 32)) 
    p.bm = per >= kW4BigRows ? kW4BigTile : kW4SmallTile;
  auto take = [&](size_t bytes) {
    const size_t at = p.ws_bytes;
    p.ws_bytes += align_up(bytes, 256);
    return at;
  };
  if (weighted && !p.sum_in_kernel) p.part = take((size_t)R * (size_t)s.d_out * 4);
  if (p.bm > 0) {
    p.xs = take((size_t)xs_bytes);  // R rows where each choice has its own
    p.up = take((size_t)R * 4);
    if (k > 0) {
      const int64_t chunks = (R + 8191) / 8192;
      p.hist = take(((size_t)chunks * (size_t)(s.n + 1) + 1) * 4);
      p.perm = take((size_t)R * 4);
      p.tiles = take((size_t)w4_max_tiles((int)R, s.n, p.bm) * 16);
    }
  }
  return p;
}

}  // namespace lora
