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
  uint16_t row[LORA_W4_MOE_MAX_TOKENS], tok[LORA_W4_MOE_MAX_TOKENS];
  float w[LORA_W4_MOE_MAX_TOKENS];
};

// bf16 parts that a row is held in: x, and h = act(gate) * up.  Of bf16 rows h
// is a float32 taken to 16 bits (an error of 2^-16 of it: y, rounded to 8 bits,
// does not see it), of float32 rows both are whole.
constexpr int moe_h_parts(int dtype) { return dtype == LORA_DTYPE_BF16 ? 2 : 3; }

struct MoePlan {
  int entries;       // rows of the table: the choices, or the experts
  bool by_row;
  int h_tiles;       // tiles of 128 of a row of h
  size_t h, table;   // h [T k][parts][h_tiles * 128] bf16
  size_t ws_bytes;
};

inline MoePlan moe_plan_call(int n, int ffn, int dtype, int T, int k) {
  MoePlan p{};
  if (T <= 0) return p;
  const int R = T * k;
  p.by_row = R <= n;
  p.entries = p.by_row ? R : n;
  p.h_tiles = w4_k_tiles(ffn);
  p.h = 0;
  p.ws_bytes = align_up((size_t)R * (size_t)moe_h_parts(dtype) * (size_t)p.h_tiles * kW4K * 2, 256);
  p.table = p.ws_bytes;
  p.ws_bytes += align_up((size_t)p.entries * sizeof(MoeEntry), 256);
  return p;
}

}  // namespace lora
