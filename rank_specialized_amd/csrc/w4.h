// Sizes and layouts of the 4-bit base products, shared by the host side and
// the kernels (no HIP types: the argument checks compile without HIP).
#pragma once
#include <stddef.h>
#include <stdint.h>

#include <initializer_list>

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
// left by 2: nibble 0 then sits on bits 2..5 of each half, where "or" with
// 32.0 in bf16 or 256.0 in f16 (both of step 1/4) makes the number 32 + q or
// 256 + q, and nibble 1 on bits 6..9, where 16.0 in f16 (step 1/64) makes 16 + q.
constexpr int kW4Rows = 16;
constexpr int kW4K = 128;
constexpr int kW4TileBytes = kW4Rows * kW4K / 2;

// How a group's scale and zero point are held: bf16 scales without zero
// points in 2 bytes, with them in 4 (the zero point as the bf16 of 32 + z),
// float32 scales in 8 (scale, 32 + z).
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

// The few-rows kernel holds its rows of x in LDS: per row and 128-input tile
// 256 bytes (float32 rows: three bf16 planes), and 16 bytes more per row, so
// that 16 rows' pieces of one matrix-core step lie on all banks.
inline int w4_lds_row_bytes(int dtype, int tiles) { return (dtype == LORA_DTYPE_BF16 ? 1 : 3) * tiles * kW4K * 2 + 16; }

// How a call is run, and the workspace it takes.
struct W4Plan {
  int bm;              // rows per tile of the many-rows kernel; 0: the few-rows kernel
  bool sum_in_kernel;  // few rows, weighted: each token's matrices run through by one workgroup
  bool keep_parts;     // float32 rows [splits][R][d_out] are kept and summed by a last kernel
  int rt, nt;          // few rows: 16-output blocks and 16-row blocks of a workgroup
  int row_cap;         // rows held in LDS at a time
  bool chunked;        // few rows: not all inputs of the rows in LDS at once
  int splits, per_split;  // splits of the inputs, tiles of one
  size_t part;
  size_t xs, up;             // many rows: x as f16, the rows' powers of two
  size_t hist, perm, tiles;  // many rows by matrix: counts and the number of tiles, the order, the tiles
  size_t ws_bytes;
};
// Rows of a weighted call up to which a token's k products are one
// workgroup's sum (if its rows fit LDS).  8 experts of 1408 -> 2048 for one
// token: 9.4 us in one kernel, 7.5 + 3.9 us as partial rows and their sum;
// the partial rows read a matrix once for all its tokens, though, so more
// than a few tokens are better off with them.
constexpr int kW4SumRows = 32;
// Rows per tile of the many-rows kernel.  Larger tiles unpack a code for more
// rows, smaller ones waste fewer rows of a matrix's last; 112 rows take every
// register there is, and were slower than 96 in each of these.  Measured (64,
// 96 rows): 8192 rows, 4096 -> 14336: 912, 871 us; 32 experts of 512 rows, 2048
// -> 2816: 224, 222 us; 64 experts of 256 rows, 1408 -> 2048: 138, 143 us.
constexpr int kW4BigTile = 96, kW4SmallTile = 64;
constexpr int kW4BigRows = 384;  // by matrix: rows each from which the big tile is taken
constexpr int kW4Chunk = 4096;  // rows sorted by one workgroup
// Tiles of at most bm rows that R rows of n matrices (and of none) cut into.
inline int64_t w4_max_tiles(int R, int n, int bm) { return plan_max_runs(R, n + 1, bm); }

// What the many-rows kernel takes, in us, up to a constant: its workgroups run
// two to a compute unit, so in rounds of 512, and a last round of at most 256
// with a compute unit each; a workgroup's time goes with its tiles of inputs;
// splits have their float32 rows written, read and added.  The constants are
// fitted to times measured at 200 to 6000 rows of 4096 -> 14336, 14336 -> 4096,
// 4096 -> 4096 and 1368 -> 4888 with groups of 128, which they give to 5%.
// Groups of 64 come 3% to 25% larger and of 32 25% to 40% (8192 rows of 4096 ->
// 14336 1091 and 1180 us, where groups of 128 took 917 in that run); the choice
// between the tiles was not fitted there.  Whole rounds matter: 1024 rows of
// 4096 -> 4096 52 us with tiles of 64 rows, 67 with 96; 2481 rows 107 and 87.
inline double w4_many_us(int rows, int64_t tiles, int per_split, int splits, double outputs) {
  const int64_t groups = tiles * splits, full = groups / 512, rest = groups % 512;
  const double pair = rows == kW4BigTile ? 2.23 : 1.72, alone = rows == kW4BigTile ? 1.66 : 1.15;
  const double rounds = (double)full * pair + (rest > 256 ? pair : (rest > 0 ? alone : 0.));
  return per_split * rounds + 2.7 * (double)(full + (rest > 0)) + (splits > 1 ? 1.1e-6 * outputs * splits : 0.);
}

// And the few-rows kernel, of one matrix and more than 64 rows, whose codes are
// read and expanded once per 64 rows: 64, 128, 256, 512 rows of 4096 -> 14336
// 30, 42, 76, 135 us (many-rows: 29, 36, 51, 71), of 14336 -> 4096 30, 46, 69,
// 122 (45, 49, 62, 88), of 4096 -> 4096 13, 21, 30, 41 (22, 29, 29, 38), of 1368
// -> 4888 9.2, 10.7, 17.9, 27.9 (18, 19, 23, 22).
inline double w4_few_us(int R, int64_t tiles) { return 9. + 5.8e-4 * (double)tiles * ((R + 63) / 64); }

// The many-rows kernel's tiles and splits, if it is taken.  It has x rewritten
// first and, by matrix, the rows sorted (5 to 20 us).  By matrix, few-rows
// against many-rows, all kernels: 32 experts of 12 rows 30 against 45 us, of 24
// rows 38 against 45, of 32 rows 90 against 64, of 64 rows 148 against 70 (2048
// -> 2816); of a few small matrices up to 48 rows each, 26 and 48 rows: 3 of 512
// -> 264 7.2, 7.6 against 15.6, 15.3; 8 of 1024 -> 1024 8.6, 10.2 against 17.6,
// 19.1; 4 of 2048 -> 2048 13.0, 16.2 against 19.8, 22.5 (with many matrices the
// rows of one that most choose would take long: 32 of 1024 -> 512, all rows of
// one, 133 against 21).  Of one matrix, what the two are expected to take.
// Offsets are 32-bit: the rewritten x and a matrix stay below 2^32 bytes.
inline void w4_plan_many(W4Plan& p, const lora_w4_store& s, int R, int per, bool by_matrix, int64_t xs_bytes) {
  const int64_t codes = w4_tiles(s.d_in, s.d_out);
  const int few = s.n <= 8 && s.n * codes <= 8192 ? 48 : 24;
  if ((by_matrix ? per <= few : R <= 64) || xs_bytes >= ((int64_t)1 << 32)) return;
  if (codes * kW4TileBytes >= ((int64_t)1 << 31)) return;
  const int kt = w4_k_tiles(s.d_in);
  double best = 0.;
  for (const int rows : {kW4SmallTile, kW4BigTile}) {
    if (by_matrix && rows != (per >= kW4BigRows ? kW4BigTile : kW4SmallTile)) continue;
    const int64_t tiles = (int64_t)s.n * ((per + rows - 1) / rows) * ((s.d_out + 255) / 256);
    // Splits of the inputs, four tiles of inputs at least to each.
    for (int want = 1; want <= 8 && (want == 1 || want <= kt / 4); ++want) {
      const int per_split = (kt + want - 1) / want, splits = (kt + per_split - 1) / per_split;
      const double us = w4_many_us(rows, tiles, per_split, splits, (double)R * s.d_out);
      if (p.bm > 0 && us >= best) continue;
      best = us;
      p.bm = rows;
      p.per_split = per_split;
      p.splits = splits;
    }
  }
  if (!by_matrix && best + 8. + 0.43e-6 * (double)xs_bytes > w4_few_us(R, codes)) p.bm = 0;
}

// The few-rows kernel's blocks and splits.
inline void w4_plan_few(W4Plan& p, const lora_w4_store& s, int dtype, int R, int per, bool by_matrix) {
  const int kt = w4_k_tiles(s.d_in), row_tiles = w4_row_tiles(s.d_out), row_bytes = w4_lds_row_bytes(dtype, kt);
  const bool bf16 = dtype == LORA_DTYPE_BF16, by_row = by_matrix && R <= s.n;
  p.splits = 1;
  p.per_split = kt;
  // A matrix's rows, with room for more than the average: what does not fit
  // takes the matrix's codes once more.  Uniform choices, and all rows of one
  // matrix: 256 rows of 64 matrices 1408 -> 2048 25.6 and 128 us with 7 rows,
  // 22.8 and 80 with 16 (256 rows 2048 -> 2816, in chunks with 16: 38 and 155,
  // 39.6 and 79; float32 in chunks is slower, 128 rows 1408 -> 2048 35
  // against 46); 64 rows of 64 2048 -> 2816 24.2 and 58 with 4, 24.2 and 36
  // with 8, 29.7 and 21 with 16.
  int rows = R;
  if (by_row) {
    const int cap = 8 * row_bytes <= 64 * 1024 ? 8 : 4;
    rows = R < cap ? R : cap;
  } else if (by_matrix) {
    rows = per < 13 && (bf16 || 16 * row_bytes <= 64 * 1024) ? 16 : per + 3;
  }
  const int64_t blocks = (int64_t)row_tiles * (by_matrix ? (R < s.n ? R : s.n) : 1);
  p.nt = rows <= 16 ? 1 : (rows <= 32 || !bf16 ? 2 : 4);
  p.row_cap = rows < 16 * p.nt ? rows : 16 * p.nt;
  const int64_t all = (int64_t)p.row_cap * row_bytes;
  // All inputs of the rows in LDS, where that leaves room for two
  // workgroups on a compute unit, or there is no more than one for it: 16
  // rows 3584 -> 3584 5.8 us so, 7.1 + 2.8 (and a sum) in chunks and
  // splits; but 3584 -> 18944 31 against 11.5 + 3.9.
  if (p.nt == 1 && (all <= 64 * 1024 || (blocks < 512 && all <= 128 * 1024))) {
    // 16-output blocks per workgroup: more share a row's LDS reads, fewer
    // give every compute unit work.  Waves and tiles in flight go with it
    // (launch_mode).  One token (blocks): 3584 -> 512 (32) 3.5, 5.4, 8.8 us
    // with 1, 2, 4; 3584 -> 18944 (1184) 9.3, 11.1, 13.4; eight experts of
    // 2048 -> 2816 (1408) 10.6, 7.8, 10.2; 40 (7040) 43, 36, 27.
    p.rt = blocks < 512 ? 0 : (blocks < 1280 ? 1 : (blocks < 2816 ? 2 : 4));
  } else {
    // In chunks, and the inputs split until there are about 768 workgroups
    // of at least eight tiles of inputs: 23 rows 18944 -> 3584 14.0 us with
    // 13 splits, 19.2 with 6.
    p.chunked = true;
    p.row_cap = 16 * p.nt;
    p.rt = p.nt == 4 ? 2 : 4;
    const int64_t groups = (blocks + p.rt - 1) / p.rt * (by_matrix ? 1 : (R + p.row_cap - 1) / p.row_cap);
    int64_t want = (768 + groups - 1) / groups;
    if (want > kt / 8) want = kt / 8;
    if (want > 1) {
      p.per_split = (int)((kt + want - 1) / want);
      p.per_split = (p.per_split + 3) / 4 * 4;
      p.splits = (kt + p.per_split - 1) / p.per_split;
    }
  }
}

inline W4Plan w4_plan_call(const lora_w4_store& s, int dtype, int T, int k, bool weighted) {
  W4Plan p{};
  if (T <= 0) return p;
  const int R = T * (k > 0 ? k : 1), kt = w4_k_tiles(s.d_in);
  const int per = (R + s.n - 1) / s.n;  // rows per matrix, on average
  const int64_t xs_bytes = (int64_t)R * kt * kW4K * 2;
  if (weighted && R <= kW4SumRows && (int64_t)k * w4_lds_row_bytes(dtype, kt) <= 64 * 1024) {
    p.sum_in_kernel = true;
    p.row_cap = k;
    p.splits = 1;
    p.per_split = kt;
  } else {
    if (dtype == LORA_DTYPE_BF16) w4_plan_many(p, s, R, per, k > 0, xs_bytes);
    if (p.bm == 0) w4_plan_few(p, s, dtype, R, per, k > 0);
  }
  auto take = [&](size_t bytes) {
    const size_t at = p.ws_bytes;
    p.ws_bytes += align_up(bytes, 256);
    return at;
  };
  p.keep_parts = (weighted && !p.sum_in_kernel) || p.splits > 1;
  if (p.keep_parts) p.part = take((size_t)p.splits * (size_t)R * (size_t)s.d_out * 4);
  if (p.bm > 0) {
    p.xs = take((size_t)xs_bytes);  // R rows where each choice has its own
    p.up = take((size_t)R * 4);
    if (k > 0) {
      const int64_t chunks = (R + kW4Chunk - 1) / kW4Chunk;
      p.hist = take(((size_t)chunks * (size_t)(s.n + 1) + 1) * 4);
      p.perm = take((size_t)R * 4);
      p.tiles = take((size_t)w4_max_tiles(R, s.n, p.bm) * 16);
    }
  }
  return p;
}

}  // namespace lora
