// 8-bit base products for many rows (prefill):
//
//   y[t, o] = s_x[t] s_w[o] sum_k q_x[t, k] q_w[o, k]
//
// bounded by the integer matrix cores and, for many rows, by the clock that their
// power leaves: 8192 rows 4096 -> 14336 back to back run at 1.73 to 1.86 GHz, with
// the matrix cores busy 65 % of the cycles (386 us on one set of inputs, 2490 TOPS;
// 401 to 418 in turn with others; a large plain product, 8192 cubed, reaches 2440).
// A workgroup takes 256 rows x 256 outputs, its eight waves 128 x 64 each; or 128 x
// 128, with two groups of waves over the inputs, where that gives more compute
// units work (1024 rows 3584 -> 3584 18.8 us, and 38.5 with the large ones; the
// choice is w8_plan_call's).
//
// Both operands go through LDS, 64 inputs at a time, in four stages that loads
// write directly; the operands of a step are read into registers during the
// products of the one before.  (Weights straight from memory to registers, which
// their layout allows, with rows staged 128 inputs at a time: 469 us, and 411.)
#include "host_util.h"
#include "w8_kernels.h"
#include "w8_ops.h"

namespace lora {
namespace {

struct W8GemmArgs {
  const char* codes;
  const float* scales;
  int k_tiles, d_in, d_out;
  const int8_t* q;
  int64_t ldq;  // below 2^23: a tile's rows stay below 2^31 bytes
  const float* s;
  char* y;
  int64_t ldy_bytes;
  int T;
  int tiles_o, tiles_t;
};

constexpr int kStep = 64;  // inputs of a stage
constexpr int kStages = 4;  // in LDS
constexpr int kOutTiles = 4;  // 16 x 16 products of a wave: RT by these
constexpr int kTileOrder = 4;  // row tiles walked together

// A workgroup's waves: WR x WO of them over rows and outputs, RT tiles of 16 rows
// by 64 outputs each, and WK groups of those over the inputs, each with stages of
// its own.
template <int WR, int WO, int WK, int RT>
struct Shape {
  static constexpr int kWR = WR, kWO = WO, kWK = WK, kRT = RT;
  static constexpr int kGroup = WR * WO, kWaves = kGroup * WK;
  static constexpr int kRows = 16 * RT * WR, kCols = kW8Block * WO;
  static constexpr int kRowBytes = kRows * kStep, kCodeBytes = kCols * kStep, kStageBytes = kRowBytes + kCodeBytes;
  static constexpr int kRowLoads = kRowBytes / 1024 / kGroup, kCodeLoads = kCodeBytes / 1024 / kGroup;  // of a wave and stage
  static constexpr int kLds = WK * kStages * kStageBytes;
  static_assert(kRowBytes % (1024 * kGroup) == 0 && kCodeBytes % (1024 * kGroup) == 0, "every wave loads the same");
  static_assert(WK == 1 || (WK == 2 && kGroup * RT * kOutTiles * 512 <= kLds), "half of the sums fits");
};
typedef Shape<2, 4, 1, 8> Big;  // 256 x 256
typedef Shape<2, 2, 2, 4> Mid;  // 128 x 128
static_assert(Big::kRows == kW8BigTile && Big::kCols == kW8BigTile && Mid::kRows == kW8MidTile && Mid::kCols == kW8MidTile, "w8_plan_call");

// Block b -> tile: each XCD (b % 8) takes a run of consecutive tiles, and the
// order walks groups of kTileOrder row tiles across all output tiles, so that
// tiles in flight on an XCD share rows and codes in its L2.
__device__ __forceinline__ void tile_of(int b, int nb, int tiles_o, int tiles_t, int& to, int& tt) {
  const int q = nb >> 3, rem = nb & 7, xcd = b & 7;
  const int g = xcd * q + (xcd < rem ? xcd : rem) + (b >> 3);
  const int width = kTileOrder * tiles_o;
  const int grp = g / width, first = grp * kTileOrder;
  const int gt = tiles_t - first < kTileOrder ? tiles_t - first : kTileOrder;
  const int in = g - grp * width;
  tt = first + in % gt;
  to = in / gt;
}

__device__ __forceinline__ void dma16(rsrc_t r, char* dst, uint32_t voff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)dst, 16, voff, 0, 0, 0);
}

// The operands of one 64-input step of a wave.
template <int RT>
struct Step {
  uint4 x[RT], b[kOutTiles];
};

// Loads of a stage: rows of x and tiles of codes, 1 KiB each.
template <typename S>
struct Loader {
  rsrc_t xr, cr;
  uint32_t row_at[S::kRowLoads], code_at[S::kCodeLoads];
  uint32_t piece, last_piece, k_tiles, place;
  __device__ __forceinline__ void fill(char* dst, int kt) const {
    const uint32_t k = min((uint32_t)kt * kStep + piece, last_piece);
    const uint32_t c = (uint32_t)kt < k_tiles ? (uint32_t)kt * kW8BlockBytes : kOutOfRange;
#pragma unroll
    for (int i = 0; i < S::kRowLoads; ++i) dma16(xr, dst + 1024 * S::kGroup * i + place, row_at[i] + k);
#pragma unroll
    for (int i = 0; i < S::kCodeLoads; ++i) dma16(cr, dst + S::kRowBytes + 1024 * S::kGroup * i + place, code_at[i] + c);
  }
};

// The products of step `now`, while the operands of the next one are read from
// `rows` and `codes` and tile `kt` is asked for into `dst`, another buffer, which
// restrict tells the compiler: no read waits for those loads.
template <typename S>
__device__ __forceinline__ void step(const Step<S::kRT>& now, Step<S::kRT>& next, const char* __restrict__ rows,
                                     const char* __restrict__ codes, char* __restrict__ dst, const Loader<S>& ld, int kt,
                                     i32x4_t (&acc)[S::kRT][kOutTiles]) {
  ld.fill(dst, kt);
#pragma unroll
  for (int a = 0; a < kOutTiles; ++a) next.b[a] = ld16(codes + a * kW8TileBytes);
#pragma unroll
  for (int t = 0; t < S::kRT; ++t) next.x[t] = ld16(rows + t * 16 * kStep);
#pragma unroll
  for (int t = 0; t < S::kRT; ++t)
#pragma unroll
    for (int a = 0; a < kOutTiles; ++a) acc[t][a] = mfma_i8(now.b[a], now.x[t], acc[t][a]);
  // Issue order: reads and loads spread between the products.
  constexpr int kReads = S::kRT + kOutTiles, kProducts = S::kRT * kOutTiles, kEach = kProducts > 2 * kReads ? 2 : 1;
  __builtin_amdgcn_sched_group_barrier(0x008, kEach, 0);
#pragma unroll
  for (int i = 0; i < kReads; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    if (i < S::kRowLoads + S::kCodeLoads) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, kEach, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x008, kProducts - kEach * (kReads + 1), 0);
}

template <typename E, typename S>
__global__ __launch_bounds__(64 * S::kWaves) __attribute__((amdgpu_waves_per_eu(2, 2)))
void w8_gemm_kernel(const W8GemmArgs p) {
  constexpr int RT = S::kRT;
  extern __shared__ __align__(16) char lds[];  // [WK][kStages]
  const int tid = (int)threadIdx.x, lane = tid & 63, col = lane & 15, h = lane >> 4;
  const int wave = __builtin_amdgcn_readfirstlane(tid >> 6), wk = wave / S::kGroup, w = wave % S::kGroup;
  const int wr = w / S::kWO, wo = w % S::kWO;
  int to, tt;
  tile_of((int)blockIdx.x, (int)gridDim.x, p.tiles_o, p.tiles_t, to, tt);
  const int64_t t0 = (int64_t)tt * S::kRows;
  const int m = min(S::kRows, (int)(p.T - t0));

  // Codes: 1 KiB loads, tile for tile as they lie in memory.  Load i of wave w is
  // tile kGroup i + w of a stage: [block][tile].  Past the last step zeros (out
  // of the buffer's range), as past the last block.
  const int blocks = (p.d_out + kW8Block - 1) / kW8Block;
  const uint32_t block_bytes = (uint32_t)p.k_tiles * kW8BlockBytes;  // at most 2^23
  const int blk0 = to * S::kWO;
  Loader<S> ld;
  ld.cr = make_rsrc(p.codes + (int64_t)blk0 * block_bytes, (uint32_t)min(S::kWO, blocks - blk0) * block_bytes);
  ld.k_tiles = (uint32_t)p.k_tiles;
  ld.place = 1024 * w;
#pragma unroll
  for (int i = 0; i < S::kCodeLoads; ++i) {
    const int tile = S::kGroup * i + w;
    ld.code_at[i] = (uint32_t)(tile >> 2) * block_bytes + (tile & 3) * kW8TileBytes + 16 * lane;
  }
  // Rows: a wave-wide load fills 1 KiB, 16 rows of 64 bytes; slot i of a row
  // holds piece i ^ (row / 4 % 4), so that the rows of one matrix-core read lie
  // on all banks.  Rows past m repeat the last, pieces past d_in the last too
  // (their weights are zeros).
  ld.xr = make_rsrc(p.q + t0 * p.ldq, (uint32_t)((m - 1) * p.ldq + ((p.d_in + 15) & ~15)));
  ld.last_piece = (uint32_t)(p.d_in - 1) & ~15u;
  ld.piece = (uint32_t)(((lane & 3) ^ (lane >> 4)) << 4);
#pragma unroll
  for (int i = 0; i < S::kRowLoads; ++i)
    ld.row_at[i] = (uint32_t)min(16 * (S::kGroup * i + w) + (lane >> 2), m - 1) * (uint32_t)p.ldq;
  // The rows' scales are asked for first: at the end, one after the other, they
  // took 3 us of the whole at 8192 rows 4096 -> 14336.
  float sx[RT];
#pragma unroll
  for (int t = 0; t < RT; ++t) sx[t] = p.s[t0 + min(16 * (RT * wr + t) + col, m - 1)];
  asm volatile("" ::: "memory");
  // Of WK groups, group wk takes tiles of inputs wk, wk + WK, ...
  char* ring = lds + wk * kStages * S::kStageBytes;
#pragma unroll
  for (int st = 0; st < kStages; ++st) ld.fill(ring + st * S::kStageBytes, S::kWK * st + wk);

  i32x4_t acc[RT][kOutTiles];
#pragma unroll
  for (int t = 0; t < RT; ++t)
#pragma unroll
    for (int a = 0; a < kOutTiles; ++a) acc[t][a] = i32x4_t{0, 0, 0, 0};
  // A lane's places in a stage.
  const uint32_t rows_at = (uint32_t)(16 * RT * wr + col) * kStep + (uint32_t)((h ^ (col >> 2)) << 4);
  const uint32_t codes_at = (uint32_t)(S::kRowBytes + wo * kW8BlockBytes + 16 * lane);
  Step<RT> s0, s1;
  // Until at most the loads of kBehind stages are in flight, and every wave's
  // reads have ended (lgkmcnt), which the barrier itself does not wait for.
  constexpr int kPer = S::kRowLoads + S::kCodeLoads, kBehind = (kStages - 2) * kPer, kFirst = (kStages - 1) * kPer;
  __builtin_amdgcn_s_waitcnt((kFirst & 15) | ((kFirst >> 4) << 14) | 0x0070);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
#pragma unroll
  for (int a = 0; a < kOutTiles; ++a) s0.b[a] = ld16(ring + codes_at + a * kW8TileBytes);
#pragma unroll
  for (int t = 0; t < RT; ++t) s0.x[t] = ld16(ring + rows_at + t * 16 * kStep);
  // Stage st: its operands are in registers, those of the next are read; its
  // buffer takes stage st + kStages.  Past the last stage the same loads are
  // asked for (the last rows again, zeros for codes), so that what is in flight
  // is always the same number.
  auto turn = [&](int st, const Step<RT>& now, Step<RT>& next) {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((kBehind & 15) | ((kBehind >> 4) << 14) | 0x0070);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    const char* from = ring + ((st + 1) % kStages) * S::kStageBytes;
    step<S>(now, next, from + rows_at, from + codes_at, ring + (st % kStages) * S::kStageBytes, ld, S::kWK * (st + kStages) + wk, acc);
  };
  const int stages = (p.k_tiles + S::kWK - 1) / S::kWK;
  for (int st = 0; st < stages; st += 2) {  // of an odd number, one step of zeros more
    turn(st, s0, s1);
    turn(st + 1, s1, s0);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load may write LDS that is another workgroup's

  // Of two groups, each hands the other half of its row tiles' sums.
  constexpr int kOwn = RT / S::kWK;
  if constexpr (S::kWK > 1) {
    __syncthreads();
    i32x4_t* half = reinterpret_cast<i32x4_t*>(lds) + (int64_t)w * kOwn * kOutTiles * 64 + lane;
    i32x4_t* mine = half + wk * S::kGroup * kOwn * kOutTiles * 64;
    const i32x4_t* theirs = half + (1 - wk) * S::kGroup * kOwn * kOutTiles * 64;
#pragma unroll
    for (int t = 0; t < kOwn; ++t)
#pragma unroll
      for (int a = 0; a < kOutTiles; ++a) mine[(t * kOutTiles + a) * 64] = wk ? acc[t][a] : acc[kOwn + t][a];
    __syncthreads();
#pragma unroll
    for (int t = 0; t < kOwn; ++t)
#pragma unroll
      for (int a = 0; a < kOutTiles; ++a) acc[t][a] = (wk ? acc[kOwn + t][a] : acc[t][a]) + theirs[(t * kOutTiles + a) * 64];
  }
  const int o0 = to * S::kCols + wo * kW8Block;
  if (o0 >= p.d_out) return;
  const float* sw = p.scales + o0 + 8 * h;
  f32x4_t ws[2][2];
#pragma unroll
  for (int g = 0; g < 2; ++g)
#pragma unroll
    for (int i = 0; i < 2; ++i) ws[g][i] = *reinterpret_cast<const f32x4_t*>(sw + 32 * g + 4 * i);
#pragma unroll
  for (int t = 0; t < kOwn; ++t) {
    const int row = 16 * (RT * wr + kOwn * wk + t) + col;
    const float s = S::kWK > 1 && wk ? sx[(S::kWK - 1) * kOwn + t] : sx[t];
    if (row >= m) continue;
    char* y = p.y + (t0 + row) * p.ldy_bytes;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int o = o0 + 32 * g + 8 * h;
      if (o < p.d_out) w8_store8<E>(y + (int64_t)o * E::kBytes, acc[t][2 * g], acc[t][2 * g + 1], s, ws[g][0], ws[g][1]);
    }
  }
}

template <typename E, typename S>
hipError_t launch_gemm(W8GemmArgs& a, hipStream_t stream) {
  a.tiles_o = (a.d_out + S::kCols - 1) / S::kCols;
  a.tiles_t = (a.T + S::kRows - 1) / S::kRows;
  static DynLdsLimit lim;
  const hipError_t e = ensure_dynamic_lds(lim, reinterpret_cast<const void*>(w8_gemm_kernel<E, S>), S::kLds);
  if (e != hipSuccess) return e;
  // at most 2^13 * 2^13 workgroups
  hipLaunchKernelGGL((w8_gemm_kernel<E, S>), dim3((unsigned)(a.tiles_o * a.tiles_t)), dim3(64 * S::kWaves), S::kLds, stream, a);
  return hipGetLastError();
}
template <typename E>
hipError_t launch_shape(W8GemmArgs& a, const W8Plan& pl, hipStream_t stream) {
  return pl.tile == kW8BigTile ? launch_gemm<E, Big>(a, stream) : launch_gemm<E, Mid>(a, stream);
}

}  // namespace

hipError_t launch_w8_gemm(const W8Call& c, hipStream_t stream) {
  W8GemmArgs a{};
  a.codes = reinterpret_cast<const char*>(c.w.codes);
  a.scales = reinterpret_cast<const float*>(c.w.scales);
  a.k_tiles = w8_k_tiles(c.w.d_in);
  a.d_in = c.w.d_in;
  a.d_out = c.w.d_out;
  a.q = c.q;
  a.ldq = c.ldq;
  a.s = c.s;
  a.y = reinterpret_cast<char*>(c.y);
  a.ldy_bytes = c.ldy * elem_bytes(c.dtype);
  a.T = c.T;
  return c.dtype == LORA_DTYPE_BF16 ? launch_shape<BF16>(a, c.plan, stream) : launch_shape<F32>(a, c.plan, stream);
}

}  // namespace lora
