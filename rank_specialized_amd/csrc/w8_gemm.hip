// 8-bit base products for many rows (prefill):
//
//   y[t, o] = s_x[t] s_w[o] sum_k q_x[t, k] q_w[o, k]
//
// bounded by the integer matrix cores and what feeds them.  A workgroup takes
// 256 rows x 256 outputs, its eight waves 128 rows x 64 outputs each (2 x 4).
// The rows' codes are staged 128 inputs at a time in LDS, two buffers, by loads
// that write LDS directly; the weights' tiles are matrix-core operands as they
// lie in memory, and go straight to registers, one stage ahead: they take no
// LDS bandwidth, of which the rows alone take most.
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

constexpr int kRows = 256, kCols = 256, kStep = 64;  // of a workgroup; inputs of a stage
constexpr int kWaves = 8;
constexpr int kRowTiles = 8, kOutTiles = 4;  // 16 x 16 products of a wave
constexpr int kRowBytes = kRows * kStep, kCodeBytes = kCols * kStep, kStageBytes = kRowBytes + kCodeBytes;
constexpr int kStages = 4;  // in LDS
constexpr int kLoads = kRowBytes / 1024 / kWaves;  // of a wave, stage and operand
constexpr int kTileOrder = 4;                      // row tiles walked together

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
struct Step {
  uint4 x[kRowTiles], b[kOutTiles];
};

// Loads of a stage: rows of x and tiles of codes, 1 KiB each.
struct Loader {
  rsrc_t xr, cr;
  uint32_t row_at[kLoads], code_at[kLoads];
  uint32_t piece, last_piece, k_tiles, place;
  __device__ __forceinline__ void fill(char* dst, int st) const {
    const uint32_t k = min((uint32_t)st * kStep + piece, last_piece);
    const uint32_t c = (uint32_t)st < k_tiles ? (uint32_t)st * kW8BlockBytes : kOutOfRange;
#pragma unroll
    for (int i = 0; i < kLoads; ++i) {
      dma16(xr, dst + 1024 * kWaves * i + place, row_at[i] + k);
      dma16(cr, dst + kRowBytes + 1024 * kWaves * i + place, code_at[i] + c);
    }
  }
};

// The products of step `now`, while the operands of the next one are read from
// `rows` and `codes` and stage `st` is asked for into `dst`, another buffer, which
// restrict tells the compiler: no read waits for those loads.
__device__ __forceinline__ void step(const Step& now, Step& next, const char* __restrict__ rows,
                                     const char* __restrict__ codes, char* __restrict__ dst, const Loader& ld, int st,
                                     i32x4_t (&acc)[kRowTiles][kOutTiles]) {
  ld.fill(dst, st);
#pragma unroll
  for (int a = 0; a < kOutTiles; ++a) next.b[a] = ld16(codes + a * kW8TileBytes);
#pragma unroll
  for (int t = 0; t < kRowTiles; ++t) next.x[t] = ld16(rows + t * 16 * kStep);
#pragma unroll
  for (int t = 0; t < kRowTiles; ++t)
#pragma unroll
    for (int a = 0; a < kOutTiles; ++a) acc[t][a] = mfma_i8(now.b[a], now.x[t], acc[t][a]);
  // Issue order: the reads spread between the products.
  __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
#pragma unroll
  for (int i = 0; i < kRowTiles + kOutTiles; ++i) {
    __builtin_amdgcn_sched_group_barrier(0x100, 1, 0);
    if (i < 2 * kLoads) __builtin_amdgcn_sched_group_barrier(0x020, 1, 0);
    __builtin_amdgcn_sched_group_barrier(0x008, 2, 0);
  }
  __builtin_amdgcn_sched_group_barrier(0x008, kRowTiles * kOutTiles - 2 * (kRowTiles + kOutTiles + 1), 0);
}

template <typename E>
__global__ __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(2, 2)))
void w8_gemm_kernel(const W8GemmArgs p) {
  extern __shared__ __align__(16) char lds[];  // kStages stages
  const int tid = (int)threadIdx.x, lane = tid & 63, col = lane & 15, h = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6), wr = w >> 2, wo = w & 3;
  int to, tt;
  tile_of((int)blockIdx.x, (int)gridDim.x, p.tiles_o, p.tiles_t, to, tt);
  const int64_t t0 = (int64_t)tt * kRows;
  const int m = min(kRows, (int)(p.T - t0));

  // Codes: 1 KiB loads, tile for tile as they lie in memory.  Load i of wave w is
  // tile 8 i + w of a stage's 16: [block][tile].  Past the last step zeros
  // (out of the buffer's range), as past the last block.
  const int blocks = (p.d_out + kW8Block - 1) / kW8Block;
  const uint32_t block_bytes = (uint32_t)p.k_tiles * kW8BlockBytes;  // at most 2^23
  const int blk0 = to * (kCols / kW8Block);
  Loader ld;
  ld.cr = make_rsrc(p.codes + (int64_t)blk0 * block_bytes, (uint32_t)min(kCols / kW8Block, blocks - blk0) * block_bytes);
  ld.k_tiles = (uint32_t)p.k_tiles;
  ld.place = 1024 * w;
#pragma unroll
  for (int i = 0; i < kLoads; ++i) ld.code_at[i] = (uint32_t)(2 * i + (w >> 2)) * block_bytes + (w & 3) * kW8TileBytes + 16 * lane;

  // Rows: a wave-wide load fills 1 KiB, 16 rows of 64 bytes; slot i of a row
  // holds piece i ^ (row / 4 % 4), so that the rows of one matrix-core read lie
  // on all banks.  Rows past m repeat the last, pieces past d_in the last too
  // (their weights are zeros).
  ld.xr = make_rsrc(p.q + t0 * p.ldq, (uint32_t)((m - 1) * p.ldq + ((p.d_in + 15) & ~15)));
  ld.last_piece = (uint32_t)(p.d_in - 1) & ~15u;
  ld.piece = (uint32_t)(((lane & 3) ^ (lane >> 4)) << 4);
#pragma unroll
  for (int i = 0; i < kLoads; ++i) ld.row_at[i] = (uint32_t)min(16 * (kWaves * i + w) + (lane >> 2), m - 1) * (uint32_t)p.ldq;
  // The rows' scales are asked for first: at the end, one after the other, they
  // took 3 us of the whole at 8192 rows 4096 -> 14336.
  float sx[kRowTiles];
#pragma unroll
  for (int t = 0; t < kRowTiles; ++t) sx[t] = p.s[t0 + min(wr * 128 + 16 * t + col, m - 1)];
  asm volatile("" ::: "memory");
#pragma unroll
  for (int st = 0; st < kStages; ++st) ld.fill(lds + st * kStageBytes, st);

  i32x4_t acc[kRowTiles][kOutTiles];
#pragma unroll
  for (int t = 0; t < kRowTiles; ++t)
#pragma unroll
    for (int a = 0; a < kOutTiles; ++a) acc[t][a] = i32x4_t{0, 0, 0, 0};
  // A lane's places in a stage.
  const uint32_t rows_at = (uint32_t)(wr * 128 + col) * kStep + (uint32_t)((h ^ (col >> 2)) << 4);
  const uint32_t codes_at = (uint32_t)(kRowBytes + wo * kW8BlockBytes + 16 * lane);
  Step s0, s1;
  // Until at most the loads of kBehind stages are in flight, and every wave's
  // reads have ended (lgkmcnt), which the barrier itself does not wait for.
  constexpr int kPer = 2 * kLoads, kBehind = (kStages - 2) * kPer, kFirst = (kStages - 1) * kPer;
  __builtin_amdgcn_s_waitcnt((kFirst & 15) | ((kFirst >> 4) << 14) | 0x0070);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
#pragma unroll
  for (int a = 0; a < kOutTiles; ++a) s0.b[a] = ld16(lds + codes_at + a * kW8TileBytes);
#pragma unroll
  for (int t = 0; t < kRowTiles; ++t) s0.x[t] = ld16(lds + rows_at + t * 16 * kStep);
  // Stage st: its operands are in registers, those of the next are read; its
  // buffer takes stage st + kStages.  Past the last stage the same loads are
  // asked for (the last rows again, zeros for codes), so that what is in flight
  // is always the same number.
  auto turn = [&](int st, const Step& now, Step& next) {
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_waitcnt((kBehind & 15) | ((kBehind >> 4) << 14) | 0x0070);
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    const char* from = lds + ((st + 1) % kStages) * kStageBytes;
    step(now, next, from + rows_at, from + codes_at, lds + (st % kStages) * kStageBytes, ld, st + kStages, acc);
  };
  for (int st = 0; st < p.k_tiles; st += 2) {  // of an odd number, one step of zeros more
    turn(st, s0, s1);
    turn(st + 1, s1, s0);
  }
  asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load may write LDS that is another workgroup's

  const int o0 = to * kCols + wo * kW8Block;
  if (o0 >= p.d_out) return;
  const float* sw = p.scales + o0 + 8 * h;
  f32x4_t ws[2][2];
#pragma unroll
  for (int g = 0; g < 2; ++g)
#pragma unroll
    for (int i = 0; i < 2; ++i) ws[g][i] = *reinterpret_cast<const f32x4_t*>(sw + 32 * g + 4 * i);
#pragma unroll
  for (int t = 0; t < kRowTiles; ++t) {
    const int row = wr * 128 + 16 * t + col;
    if (row >= m) continue;
    char* y = p.y + (t0 + row) * p.ldy_bytes;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int o = o0 + 32 * g + 8 * h;
      if (o < p.d_out) w8_store8<E>(y + (int64_t)o * E::kBytes, acc[t][2 * g], acc[t][2 * g + 1], sx[t], ws[g][0], ws[g][1]);
    }
  }
}

template <typename E>
hipError_t launch_gemm(const W8GemmArgs& a, hipStream_t stream) {
  constexpr size_t lds = kStages * kStageBytes;
  static DynLdsLimit lim;
  const hipError_t e = ensure_dynamic_lds(lim, reinterpret_cast<const void*>(w8_gemm_kernel<E>), lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((w8_gemm_kernel<E>), dim3((unsigned)(a.tiles_o * a.tiles_t)), dim3(64 * kWaves), lds, stream, a);  // at most 2^12 * 2^12
  return hipGetLastError();
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
  a.tiles_o = (c.w.d_out + kCols - 1) / kCols;
  a.tiles_t = (c.T + kRows - 1) / kRows;
  return c.dtype == LORA_DTYPE_BF16 ? launch_gemm<BF16>(a, stream) : launch_gemm<F32>(a, stream);
}

}  // namespace lora
