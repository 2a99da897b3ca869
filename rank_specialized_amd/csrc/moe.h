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

// A form of a kernel: 16-row tiles of a product; kernel 1: 16-output blocks of a
// workgroup and waves to a block; kernel 2: blocks of a wave and waves to them
// (of moe_down_blocks blocks in all); tiles of codes in flight per wave and block.
struct MoeForm {
  int tiles, blocks, waves, ahead;
};

// Kernel 1: two waves share a block's inputs, four blocks to a workgroup.  Two
// departures where one 16-row tile holds a product:
// - float32 rows whose workgroups would not reach every compute unit: one block,
//   four waves.  A unit without work counts (3 tokens, 6 of 8 experts 4096 -> 1368:
//   kernel 1 20.3 us, and 23.3 with the four blocks).
// - wide layers of four tokens or more an expert, a group to a tile: a wave to
//   all inputs of a block, eight blocks, so that half as many workgroups bring
//   the rows (64 tokens, 8 of 64 experts 2048 -> 1408: kernel 1 40.1 us, and
//   45.1 otherwise; with one token an expert 57 otherwise, and 69 so; with
//   groups of 32, whose registers do not suffice, 53 otherwise and 74 so).
enum { kMoeUpTwo, kMoeUpOne, kMoeUpWide, kMoeUpPlain };
constexpr MoeForm kMoeUpForms[] = {{2, 2, 4, 2}, {1, 1, 4, 2}, {1, 8, 1, 3}, {1, 4, 2, 2}};
inline int moe_up_form(const MoePlan& p, int dtype, int sub) {
  if (p.up_two) return kMoeUpTwo;
  if (dtype != LORA_DTYPE_BF16) return 2 * p.entries * p.h_tiles < 256 ? kMoeUpOne : kMoeUpPlain;
  return p.up_wide && sub == 1 ? kMoeUpWide : kMoeUpPlain;
}

// Kernel 2: four blocks of their own waves, two to a block (one token, 8 of 64
// experts 1408 -> 2048: 7.4 us, and 8.9 with eight blocks, two to a wave; 7
// tokens, 4 of 32: 13.3 and 14.9).  Two 16-row tiles: eight blocks, two to a
// wave (64 tokens, 8 of 64: 36.2 us, and 42.7 with four blocks): half as many
// workgroups bring the rows.  One workgroup at most to a compute unit, and long
// inputs: eight waves to two blocks (one token, 2 of 8 experts 14336 -> 4096: 19.9
// us, and 29.4 with two waves to a block; 2 of 16 10752 -> 6144 17.9, 24.4; 2 of 8
// 4096 -> 4096 8.8, 9.6; with 6 tiles of inputs, 4 of 32 768 -> 2048, 6.3 and 5.8).
enum { kMoeDownTwo, kMoeDownDeep, kMoeDownPlain };
constexpr MoeForm kMoeDownForms[] = {{2, 2, 2, 2}, {1, 2, 8, 2}, {1, 1, 2, 2}};
inline int moe_down_form(const MoePlan& p) { return p.down_two ? kMoeDownTwo : (p.down_deep ? kMoeDownDeep : kMoeDownPlain); }

}  // namespace lora
