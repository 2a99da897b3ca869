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

// How a call is run, and the workspace it takes.
struct W4Plan {
  bool sum_in_kernel;  // weighted rows: each token's matrices run through by one workgroup, no partial rows
  size_t part;         // float32 rows [R][d_out] of a weighted call that keeps them
  size_t ws_bytes;
};
// Rows of a weighted call up to which a token's k products are one
// workgroup's sum.
constexpr int kW4SumRows = 32;
inline W4Plan w4_plan_call(const lora_w4_store& s, int dtype, int T, int k, bool weighted) {
  (void)dtype;
  W4Plan p{};
  if (T <= 0) return p;
  const int64_t R = (int64_t)T * (k > 0 ? k : 1);
  p.sum_in_kernel = weighted && R <= kW4SumRows;
  if (weighted && !p.sum_in_kernel) {
    p.part = p.ws_bytes;
    p.ws_bytes += align_up((size_t)R * (size_t)s.d_out * 4, 256);
  }
  return p;
}

}  // namespace lora
