// Sizes of the mixture-of-experts layer for a few tokens, shared by the host
// side and the kernels (no HIP types).
#pragma once
#include "w4.h"

namespace lora {

// An entry of the table that the first kernel leaves for the second: one
// expert's tokens, each once, with the row (t k + j) that holds its h and its
// weight (the sum of them, where a token names an expert twice).
struct MoeEntry {
  int32_t e, cnt;
  uint16_t row[LORA_W4_MOE_MAX_TOKENS];
  float w[LORA_W4_MOE_MAX_TOKENS];
};

// bf16 parts that a row is held in: x, and h = act(gate) * up.  Of bf16 rows h
// is a float32 taken to 16 bits (an error of 2^-16 of it: y, rounded to 8 bits,
// does not see it), of float32 rows both are whole.
constexpr int moe_x_parts(int dtype) { return dtype == LORA_DTYPE_BF16 ? 1 : 3; }
constexpr int moe_h_parts(int dtype) { return dtype == LORA_DTYPE_BF16 ? 2 : 3; }

// Two 16-row tiles to a product where an expert has more tokens, on average, than
// about half of what one holds (`parts` rows each).
inline bool moe_two_tiles(int T, int k, int n, int parts) { return T > 16 / parts && 2 * T * k * parts > 16 * n; }
// 16-output blocks of d_out that a workgroup of the second kernel owns.
constexpr int moe_down_blocks(bool two_tiles) { return two_tiles ? 8 : 4; }

struct MoePlan {
  int entries;       // rows of the table: the choices, or the experts
  bool by_row;
  int h_tiles;       // tiles of 128 of a row of h
  size_t h, table;   // h [T k][parts][h_tiles * 128] bf16
  bool up_wide;      // many workgroups of several tokens each, at eight blocks of 16 features
  bool up_two, down_two;  // 16-row tiles of a product
  bool down_deep;    // few workgroups of long inputs: more waves to a block
  int down_groups;   // of moe_down_blocks blocks
  size_t part;       // [down_groups][T k][16 moe_down_blocks] float32: the choices' weighted outputs
  size_t counted;    // [T k] bytes: whether a choice has such a row
  size_t arrived;    // [down_groups] workgroups that have written theirs
  size_t ws_bytes;
};

inline MoePlan moe_plan_call(int n, int ffn, int d_out, int dtype, int T, int k) {
  MoePlan p{};
  if (T <= 0) return p;
  const int R = T * k;
  p.by_row = R <= n;
  p.entries = p.by_row ? R : n;
  p.h_tiles = w4_k_tiles(ffn);
  p.up_two = moe_two_tiles(T, k, n, moe_x_parts(dtype));
  p.up_wide = p.entries * p.h_tiles >= 512 && R >= 4 * n;
  p.down_two = moe_two_tiles(T, k, n, moe_h_parts(dtype));
  const int blocks = moe_down_blocks(p.down_two);
  p.down_groups = (w4_row_tiles(d_out) + blocks - 1) / blocks;
  p.down_deep = p.entries * p.down_groups <= 256 && p.h_tiles >= 16;
  auto take = [&](size_t bytes) {
    const size_t at = p.ws_bytes;
    p.ws_bytes += align_up(bytes, 256);
    return at;
  };
  p.h = take((size_t)R * (size_t)moe_h_parts(dtype) * (size_t)p.h_tiles * kW4K * 2);
  p.table = take((size_t)p.entries * sizeof(MoeEntry));
  p.part = take((size_t)p.down_groups * (size_t)R * 16 * (size_t)blocks * 4);
  p.counted = take((size_t)R);
  p.arrived = take((size_t)p.down_groups * 4);
  return p;
}

}  // namespace lora
