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

constexpr int kRows = 256, kCols = 256, kStep = 128;  // of a workgroup; inputs of a stage
constexpr int kWaves = 8;
constexpr int kRowTiles = 8, kOutTiles = 4;  // 16 x 16 products of a wave
constexpr int kStageBytes = kRows * kStep;
constexpr int kLoads = kStageBytes / 1024 / kWaves;  // of a wave and stage
constexpr int kTileOrder = 4;                        // row tiles walked together

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

// One stage: rows at `rd`, tiles of codes in registers, while the next rows go
// to `wr`, another buffer, which restrict tells the compiler: no read waits for
// the loads in flight.
__device__ __forceinline__ void stage(const char* __restrict__ rd, char* __restrict__ wr, bool more, rsrc_t xr,
                                      const uint32_t (&src)[kLoads], const uint4 (&b)[2][kOutTiles], uint32_t lane_row,
                                      int h, int sw, i32x4_t (&acc)[kRowTiles][kOutTiles]) {
  if (more)
#pragma unroll
    for (int i = 0; i < kLoads; ++i) dma16(xr, wr + i * 1024 * kWaves, src[i]);
  __builtin_amdgcn_s_setprio(1);
#pragma unroll
  for (int t = 0; t < kRowTiles; ++t)
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const uint4 x = ld16(rd + lane_row + t * 16 * kStep + (((4 * j + h) ^ sw) << 4));
#pragma unroll
      for (int a = 0; a < kOutTiles; ++a) acc[t][a] = mfma_i8(b[j][a], x, acc[t][a]);
    }
  __builtin_amdgcn_s_setprio(0);
}

template <typename E>
__global__ __launch_bounds__(64 * kWaves) __attribute__((amdgpu_waves_per_eu(2, 2)))
void w8_gemm_kernel(const W8GemmArgs p) {
  __shared__ __align__(16) char lds[2 * kStageBytes];
  const int tid = (int)threadIdx.x, lane = tid & 63, col = lane & 15, h = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6), wr = w >> 2, wo = w & 3;
  int to, tt;
  tile_of((int)blockIdx.x, (int)gridDim.x, p.tiles_o, p.tiles_t, to, tt);
  const int64_t t0 = (int64_t)tt * kRows;
  const int m = min(kRows, (int)(p.T - t0));

  // Tiles of codes of the wave's 64 outputs: two of inputs per stage, past the
  // last one zeros (out of the buffer's range).
  const int blocks = (p.d_out + kW8Block - 1) / kW8Block, blk = min(to * (kCols / kW8Block) + wo, blocks - 1);
  const uint32_t block_bytes = (uint32_t)p.k_tiles * kW8BlockBytes;  // at most 2^23
  const rsrc_t cr = make_rsrc(p.codes + (int64_t)blk * block_bytes, block_bytes);
  uint4 next[2][kOutTiles];
  auto fetch = [&](int st) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int a = 0; a < kOutTiles; ++a)
        next[j][a] = buf_ld16(cr, 16 * lane + a * kW8TileBytes, (uint32_t)(2 * st + j) * kW8BlockBytes);
  };

  // Rows: a wave-wide load fills 1 KiB, eight rows of 128 bytes; slot i of a
  // row holds piece i ^ (row % 8), so that the rows of one matrix-core read lie
  // on all banks.  Rows past m repeat the last, pieces past d_in the last too
  // (their weights are zeros).
  const rsrc_t xr = make_rsrc(p.q + t0 * p.ldq, (uint32_t)((m - 1) * p.ldq + ((p.d_in + 15) & ~15)));
  const uint32_t last_piece = (uint32_t)(p.d_in - 1) & ~15u;
  uint32_t row_at[kLoads];
  const uint32_t piece = (uint32_t)(((lane & 7) ^ (lane >> 3)) << 4);
#pragma unroll
  for (int i = 0; i < kLoads; ++i) row_at[i] = (uint32_t)min(8 * (kWaves * i + w) + (lane >> 3), m - 1) * (uint32_t)p.ldq;
  auto sources = [&](int st, uint32_t (&src)[kLoads]) {
    const uint32_t k = min((uint32_t)st * kStep + piece, last_piece);
#pragma unroll
    for (int i = 0; i < kLoads; ++i) src[i] = row_at[i] + k;
  };
  char* fill = lds + 1024 * w;
  const int stages = (p.k_tiles + 1) / 2;

  uint32_t src[kLoads];
  fetch(0);
  sources(0, src);
#pragma unroll
  for (int i = 0; i < kLoads; ++i) dma16(xr, fill + i * 1024 * kWaves, src[i]);
  i32x4_t acc[kRowTiles][kOutTiles];
#pragma unroll
  for (int t = 0; t < kRowTiles; ++t)
#pragma unroll
    for (int a = 0; a < kOutTiles; ++a) acc[t][a] = i32x4_t{0, 0, 0, 0};

  const uint32_t lane_row = (uint32_t)(wr * 128 + col) * kStep;
  for (int st = 0; st < stages; ++st) {
    const bool more = st + 1 < stages;
    // This stage's rows and codes were asked for a stage ago; every wave has
    // finished with the buffer that is filled next: its reads of it have ended
    // (lgkmcnt), which the barrier itself does not wait for.
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    uint4 b[2][kOutTiles];
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int a = 0; a < kOutTiles; ++a) b[j][a] = next[j][a];
    fetch(more ? st + 1 : st);
    sources(st + 1, src);
    const int cur = st & 1;
    stage(lds + cur * kStageBytes, fill + (cur ^ 1) * kStageBytes, more, xr, src, b, lane_row, h, col & 7, acc);
  }

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
    const float sx = p.s[t0 + row];
    char* y = p.y + (t0 + row) * p.ldy_bytes;
#pragma unroll
    for (int g = 0; g < 2; ++g) {
      const int o = o0 + 32 * g + 8 * h;
      if (o < p.d_out) w8_store8<E>(y + (int64_t)o * E::kBytes, acc[t][2 * g], acc[t][2 * g + 1], sx, ws[g][0], ws[g][1]);
    }
  }
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
  const unsigned grid = (unsigned)(a.tiles_o * a.tiles_t);  // at most 2^12 * 2^12
  if (c.dtype == LORA_DTYPE_BF16) hipLaunchKernelGGL((w8_gemm_kernel<BF16>), dim3(grid), dim3(64 * kWaves), 0, stream, a);
  else hipLaunchKernelGGL((w8_gemm_kernel<F32>), dim3(grid), dim3(64 * kWaves), 0, stream, a);
  return hipGetLastError();
}

}  // namespace lora
