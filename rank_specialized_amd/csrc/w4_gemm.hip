// 4-bit base products for many rows (prefill), bf16:
//
//   y[r, o] = sum_g s[o, g] sum_{k in g} (q[o, k] - z[o, g]) x[r, k]
//
// bounded by the matrix cores and the unpacking beside them.  A workgroup takes
// 16 NT rows x 256 outputs, each of its waves 32 or 64 outputs of all the rows,
// so that a code is unpacked once per 16 NT rows; the waves share the rows of x
// in LDS, staged 128 inputs at a time by loads that write LDS directly, two
// buffers.  Measured: 8192 rows 4096 -> 14336 775 to 800 us in long runs (1.2
// PFLOP/s; a library's bf16 product of that shape 712), 770 to 1080 by the
// clock in traces of a few, and 27 for the rows as f16; 32 experts of 512 rows
// 2048 -> 2816 207 us (0.9).
//
// By matrix the grid is that of the most tiles there can be, and each XCD has
// an eighth of it: the tiles that do not exist are all the last XCDs' (191 of
// 203 tiles in the case above, where the busiest has 7% more than the mean).  A
// tile of fewer rows costs a whole one.
//
// The codes enter the products as f16 numbers: 256 + q or 16 + q (the two
// places of a code in f16's ten fraction bits, so that one shift serves four
// codes) is one "and-or" per two codes, and one packed addition takes 256 + z
// or 16 + z off, leaving q - z itself, exactly (f16 arithmetic is packed,
// bf16's is not).  x must then be f16 too:
// a first kernel writes each row times the power of two that brings its
// largest value to [2^14, 2^15), which keeps all eight bits of every bf16
// value down to 2^-31 of the row's largest (below, the rounding is at most
// 2^-39 of that largest), and the power is put back at the end.  Products are
// exact in float32, a group's are summed by the matrix cores, and the group's
// scale multiplies its sum once per lane, in float32.
#include <hip/hip_fp16.h>

#include "host_util.h"
#include "w4_kernels.h"
#include "w4_ops.h"

namespace lora {
namespace {

typedef __attribute__((ext_vector_type(8))) _Float16 f16x8_t;
typedef __attribute__((ext_vector_type(2))) _Float16 f16x2_t;

__device__ __forceinline__ f32x4_t mfma_f16(const uint4& a, const uint4& b, f32x4_t c) {
  return __builtin_amdgcn_mfma_f32_16x16x32_f16(__builtin_bit_cast(f16x8_t, a), __builtin_bit_cast(f16x8_t, b), c, 0, 0,
                                                0);
}

struct W4GroupArgs {
  const int32_t* ids;
  int R, n, chunks, bm;
  int32_t* hist;    // [chunks][n + 1]
  int32_t* perm;    // [R]: rows, ascending matrix
  int4* tiles;      // matrix (n: none), first position, rows
  int32_t* n_tiles;
};
constexpr int kChunk = kW4Chunk;  // rows counted, and placed, by one workgroup

// Rows per matrix (n: none) of one chunk.
__device__ __forceinline__ void count_chunk(const W4GroupArgs& g, int chunk) {
  __shared__ int hist[LORA_W4_MAX_N + 1];
  const int tid = (int)threadIdx.x, threads = (int)blockDim.x, n1 = g.n + 1;
  for (int i = tid; i < n1; i += threads) hist[i] = 0;
  __syncthreads();
  const int r0 = chunk * kChunk, r1 = min(g.R, r0 + kChunk);
  constexpr int kAhead = 8;  // ids asked for together
  for (int r = r0 + tid; r < r1; r += kAhead * threads) {
    int id[kAhead];
#pragma unroll
    for (int i = 0; i < kAhead; ++i) id[i] = g.ids[min(r + i * threads, r1 - 1)];
#pragma unroll
    for (int i = 0; i < kAhead; ++i)
      if (r + i * threads < r1) atomicAdd(&hist[(unsigned)id[i] < (unsigned)g.n ? id[i] : g.n], 1);
  }
  __syncthreads();
  for (int i = tid; i < n1; i += threads) g.hist[(int64_t)chunk * n1 + i] = hist[i];
}

// ------------------------------------------------------------ x as f16
// One wave per row: xs[r] = f16(x[r] 2^-e), zeros up to the last tile's end,
// and up[r] = 2^e.  A row's infinities and NaNs stay what they are.  The
// first g.chunks workgroups count the rows per matrix instead.
__global__ __launch_bounds__(256) void w4_f16_kernel(const char* __restrict__ x, int64_t ldx_bytes, int rows, int d_in,
                                                    int kp, char* __restrict__ xs, float* __restrict__ up,
                                                    const W4GroupArgs g) {
  if ((int)blockIdx.x < g.chunks) {
    count_chunk(g, (int)blockIdx.x);
    return;
  }
  const int r = ((int)blockIdx.x - g.chunks) * 4 + ((int)threadIdx.x >> 6), lane = (int)threadIdx.x & 63;
  if (r >= rows) return;
  const char* src = x + (int64_t)r * ldx_bytes;
  uint32_t top = 0;  // the largest exponent below that of infinity
  auto look = [&](const uint4& v) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t a = (w[i] >> 7) & 255u, b = (w[i] >> 23) & 255u;
      top = a < 255u && a > top ? a : top;
      top = b < 255u && b > top ? b : top;
    }
  };
  // The first 4096 values stay in registers between the two steps; what is
  // behind them is read again (8192 rows of 4096 26.5 us, 5 TB/s; all read
  // twice 36.8).
  constexpr int kHold = 8, kStep = 512;  // 8 values per lane and step
  uint4 hold[kHold];
#pragma unroll
  for (int i = 0; i < kHold; ++i) {
    const int k = i * kStep + 8 * lane;
    hold[i] = make_uint4(0u, 0u, 0u, 0u);
    if (k < d_in) hold[i] = ld16(src + 2 * (int64_t)k);
  }
#pragma unroll
  for (int i = 0; i < kHold; ++i) look(hold[i]);
  for (int k = kHold * kStep + 8 * lane; k < d_in; k += kStep) look(ld16(src + 2 * (int64_t)k));
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const uint32_t o = (uint32_t)__shfl_xor((int)top, d);
    top = o > top ? o : top;
  }
  int e = (int)top - 127 - 14;
  e = e < -126 ? -126 : e;
  const float down = __uint_as_float((uint32_t)(127 - e) << 23);
  char* dst = xs + (int64_t)r * kp * 2;
  auto write = [&](int k, const uint4& v) {  // zeros stay zeros
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
    uint32_t out[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const f16x2_t h = {(_Float16)(bf16_lo(w[i]) * down), (_Float16)(bf16_hi(w[i]) * down)};
      out[i] = __builtin_bit_cast(uint32_t, h);
    }
    st16(dst + 2 * (int64_t)k, make_uint4(out[0], out[1], out[2], out[3]));
  };
#pragma unroll
  for (int i = 0; i < kHold; ++i) {
    const int k = i * kStep + 8 * lane;
    if (k < kp) write(k, hold[i]);
  }
  for (int k = kHold * kStep + 8 * lane; k < kp; k += kStep)
    write(k, k < d_in ? ld16(src + 2 * (int64_t)k) : make_uint4(0u, 0u, 0u, 0u));
  if (lane == 0) up[r] = __uint_as_float((uint32_t)(127 + e) << 23);
}

// ------------------------------------------------------------ rows by matrix
constexpr int kGroupThreads = 1024;

// Each workgroup places its rows: first position of a matrix, plus the rows
// of earlier workgroups, plus a counter.  (The order of a matrix's rows may
// change from call to call; a row's result does not depend on it.)  The first
// workgroup also writes the tiles: runs of at most bm rows of one matrix.
__global__ __launch_bounds__(kGroupThreads) void w4_place_kernel(const W4GroupArgs p) {
  __shared__ int pos[LORA_W4_MAX_N + 1];
  __shared__ int2 wsum[kGroupThreads / 64];
  const int tid = (int)threadIdx.x, n1 = p.n + 1, lane = tid & 63, w = tid >> 6;
  // n + 1 <= 1025 matrices: thread t scans t, and the last thread also n.
  int cnt[2] = {0, 0}, before[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int e = tid + i * kGroupThreads;
    if (e < n1)
      for (int c = 0; c < p.chunks; ++c) {
        const int v = p.hist[(int64_t)c * n1 + e];
        before[i] += c < (int)blockIdx.x ? v : 0;
        cnt[i] += v;
      }
  }
  int2 s = make_int2(cnt[0], (cnt[0] + p.bm - 1) / p.bm);
  const int2 own = s;
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) {
    const int a = __shfl_up(s.x, d), b = __shfl_up(s.y, d);
    if (lane >= d) {
      s.x += a;
      s.y += b;
    }
  }
  if (lane == 63) wsum[w] = s;
  __syncthreads();
  int2 off = make_int2(s.x - own.x, s.y - own.y), all = make_int2(0, 0);
  for (int i = 0; i < kGroupThreads / 64; ++i) {
    if (i < w) {
      off.x += wsum[i].x;
      off.y += wsum[i].y;
    }
    all.x += wsum[i].x;
    all.y += wsum[i].y;
  }
  const int extra = (cnt[1] + p.bm - 1) / p.bm;  // of matrix kGroupThreads, if there is one (thread 0)
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int e = tid + i * kGroupThreads;
    if (e >= n1) continue;
    const int first = i ? all.x : off.x, tile0 = i ? all.y : off.y;
    pos[e] = first + before[i];
    if (blockIdx.x == 0)
      for (int m = 0, t = tile0; m < cnt[i]; m += p.bm, ++t) p.tiles[t] = make_int4(e, first + m, min(p.bm, cnt[i] - m), 0);
  }
  if (blockIdx.x == 0 && tid == 0) *p.n_tiles = all.y + (n1 > kGroupThreads ? extra : 0);
  __syncthreads();
  const int r0 = (int)blockIdx.x * kChunk, r1 = min(p.R, r0 + kChunk);
  int id[kChunk / kGroupThreads];
#pragma unroll
  for (int i = 0; i < kChunk / kGroupThreads; ++i) id[i] = p.ids[min(r0 + tid + i * kGroupThreads, r1 - 1)];
#pragma unroll
  for (int i = 0; i < kChunk / kGroupThreads; ++i) {
    const int r = r0 + tid + i * kGroupThreads;
    if (r < r1) p.perm[atomicAdd(&pos[(unsigned)id[i] < (unsigned)p.n ? id[i] : p.n], 1)] = r;
  }
}

// ------------------------------------------------------------ the product
struct W4GemmArgs {
  const char* codes;
  const char* params;
  int64_t code_stride, param_stride;
  int n, k_tiles, row_tiles, d_out;
  const char* xs;   // f16 rows of k_tiles * 128
  const float* up;
  int x_div;
  char* y;          // bf16 rows, or float32 (F32OUT)
  int64_t ldy_bytes;
  int R;
  const int32_t* perm;    // nullptr: rows in order, one matrix
  const int4* tiles;
  const int32_t* n_tiles;
  int tiles_o, tiles_t;
  int per_split;  // tiles of inputs per split (blockIdx.y): float32 rows [splits][R]
};

constexpr int kCols = 256;  // outputs of a workgroup
// Its waves, each with kCols / waves of the outputs.  Eight waves of two
// 16-output blocks fit four to a SIMD, four waves of four blocks two; with
// more than one scale per tile and output eight no longer fit their
// registers.  Measured side by side (8, 4 waves): 32 experts of 512 rows 2048
// -> 2816 222, 238 us; with groups of 64 and zero points 8192 rows 4096 ->
// 14336 1019, 1007, of 32 1316, 1153.  With four waves, four float32 scales per
// tile and output spill 29 to 31 registers at 96 rows (4 at 64), every other
// form at most 2.
constexpr int gemm_waves(int sub) { return sub == 1 ? 8 : 4; }
constexpr int kTileOrder = 4;  // row tiles walked together (w4_tile_of)

// Block b -> tile, as for the bf16 base product: each XCD (b % 8) takes a run
// of consecutive tiles, and the order walks groups of kTileOrder row tiles
// across all output tiles, so that tiles in flight on an XCD share x and
// codes in its L2.
__device__ __forceinline__ void w4_tile_of(int b, int nb, int tiles_o, int tiles_t, int& to, int& tt) {
  const int q = nb >> 3, rem = nb & 7, xcd = b & 7;
  const int g = xcd * q + (xcd < rem ? xcd : rem) + (b >> 3);
  const int width = kTileOrder * tiles_o;
  const int grp = g / width, first = grp * kTileOrder;
  const int gt = tiles_t - first < kTileOrder ? tiles_t - first : kTileOrder;
  const int in = g - grp * width;
  tt = first + in % gt;
  to = in / gt;
}

// 16 bytes per lane from a buffer into LDS at dst + 16 * lane.
__device__ __forceinline__ void dma16(rsrc_t r, char* dst, uint32_t voff, uint32_t soff) {
  __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (__attribute__((address_space(3))) void*)dst, 16, voff, soff, 0, 0);
}

template <int NT, int kWaves>
constexpr int x_loads() {  // of a wave and step
  static_assert(4 * NT % kWaves == 0, "every wave loads the same number of rows");
  return 4 * NT / kWaves;
}
template <int NT>
constexpr int stage_bytes() {
  return 16 * NT * kW4K * 2;
}

// The products of one tile of 128 inputs: x rows at `rd`, codes and scales in
// registers.  `rd` and `wr` (where the next rows are being written) are
// different buffers, which restrict tells the compiler, so that no read waits
// for the loads in flight.
template <int SUB, int NT, int kWaves, int kRT>
__device__ __forceinline__ void gemm_step(const char* __restrict__ rd, char* __restrict__ wr, bool more,
                                          rsrc_t xr, const uint32_t (&src)[x_loads<NT, kWaves>()], uint32_t soff, const uint4 (&b)[kRT][4],
                                          const float (&sc)[kRT][SUB], uint32_t lane_row, int h, int row16,
                                          f32x4_t (&acc)[NT][kRT]) {
  constexpr int kSteps = 4 / SUB;
  if (more)
#pragma unroll
    for (int q = 0; q < x_loads<NT, kWaves>(); ++q) dma16(xr, wr + q * 1024 * kWaves, src[q], soff);
  __builtin_amdgcn_s_setprio(1);  // a wave with products ahead goes before one that unpacks
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    uint4 x[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) x[j] = ld16(rd + t * 16 * kW4K * 2 + lane_row + (((4 * j + h) ^ row16) << 4));
#pragma unroll
    for (int s = 0; s < SUB; ++s) {
      f32x4_t c[kRT];
#pragma unroll
      for (int j = 0; j < kSteps; ++j)
#pragma unroll
        for (int a = 0; a < kRT; ++a)
          c[a] = mfma_f16(x[s * kSteps + j], b[a][s * kSteps + j], j == 0 ? f32x4_t{0.f, 0.f, 0.f, 0.f} : c[a]);
#pragma unroll
      for (int a = 0; a < kRT; ++a)
#pragma unroll
        for (int v = 0; v < 4; ++v) acc[t][a][v] = fmaf(sc[a][s], c[a][v], acc[t][a][v]);
    }
  }
  __builtin_amdgcn_s_setprio(0);
}

template <int KIND, int SUB, int NT, bool F32OUT>
__global__ __launch_bounds__(64 * gemm_waves(SUB))
__attribute__((amdgpu_waves_per_eu(gemm_waves(SUB) / 2, gemm_waves(SUB) / 2)))
void w4_gemm_kernel(const W4GemmArgs p) {
  constexpr int kWaves = gemm_waves(SUB), kRT = kCols / 16 / kWaves;  // blocks of 16 outputs per wave
  constexpr int kRows = 16 * NT;
  __shared__ __align__(16) char lds[2 * stage_bytes<NT>()];
  __shared__ uint32_t row_of[kRows];  // rows of y
  __shared__ float row_up[kRows];     // and their powers of two
  const int tid = (int)threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int col = lane & 15, h = lane >> 4;
  int to, tt;
  w4_tile_of((int)blockIdx.x, (int)gridDim.x, p.tiles_o, p.tiles_t, to, tt);
  int e = 0, pos0 = tt * kRows, m = min(kRows, p.R - pos0);
  if (p.perm != nullptr) {
    if (tt >= *p.n_tiles) return;
    const int4 t = p.tiles[tt];
    e = t.x;
    pos0 = t.y;
    m = t.z;
  }
  const int o0 = to * kCols;
  if (e >= p.n) {  // rows without a matrix: empty sums (float32 rows are then not read)
    if (F32OUT) return;
    for (int i = tid; i < m * (kCols / 8); i += 64 * kWaves) {
      const int r = p.perm[pos0 + i / (kCols / 8)], o = o0 + 8 * (i % (kCols / 8));
      if (o >= p.d_out) continue;
      st16(p.y + (int64_t)r * p.ldy_bytes + 2 * (int64_t)o, make_uint4(0, 0, 0, 0));
    }
    return;
  }

  // ---- codes: one tile of each of the wave's output blocks, loaded a step
  // ahead; the first before the rows are looked up (64 experts of 256 rows
  // 1408 -> 2048 139 us so, 146 after).  A matrix's codes are below 2^32 bytes
  // (w4_plan_call).
  uint4 code[kRT];
  W4Params<KIND, SUB> par[kRT];
  constexpr int kParBytes = kW4Rows * W4Params<KIND, SUB>::kBytes;  // of a tile
  const rsrc_t cr = make_rsrc(p.codes + e * p.code_stride, (uint32_t)p.code_stride);
  const rsrc_t pr = make_rsrc(p.params + e * p.param_stride, (uint32_t)p.param_stride);
  uint32_t tile0[kRT];
#pragma unroll
  for (int a = 0; a < kRT; ++a)
    tile0[a] = (uint32_t)min(to * (kCols / 16) + kRT * w + a, p.row_tiles - 1) * (uint32_t)p.k_tiles;
  const uint32_t lane16 = 16 * lane, lane_par = col * W4Params<KIND, SUB>::kBytes;
  auto fetch = [&](int kt) {
#pragma unroll
    for (int a = 0; a < kRT; ++a) {
      code[a] = buf_ld16(cr, lane16, (tile0[a] + kt) * kW4TileBytes);
      par[a].load(pr, lane_par, (tile0[a] + kt) * kParBytes);
    }
  };
  const int k0 = (int)blockIdx.y * p.per_split, k1 = min(p.k_tiles, k0 + p.per_split);
  fetch(k0);

  // ---- x: a wave-wide load fills 1 KiB, four rows of 256 bytes; slot i % 16
  // of a row holds piece (i % 16) ^ (row % 16), so that the 16 rows of one
  // matrix-core read lie on all banks.  Rows past m repeat the last.
  const uint32_t x_bytes = p.k_tiles * kW4K * 2;
  const rsrc_t xr = make_rsrc(p.xs, (uint32_t)(p.R / p.x_div) * x_bytes);  // below 2^32 (w4_plan_call)
  uint32_t src[x_loads<NT, kWaves>()];
#pragma unroll
  for (int q = 0; q < x_loads<NT, kWaves>(); ++q) {
    const int row = 4 * (kWaves * q + w) + (lane >> 4);
    const int pos = pos0 + min(row, m - 1);
    const uint32_t r = p.perm != nullptr ? (uint32_t)p.perm[pos] : (uint32_t)pos;
    src[q] = (r / (uint32_t)p.x_div) * x_bytes + (((lane & 15) ^ (row & 15)) << 4);
  }
  char* fill = lds + 1024 * w;  // + q * 1024 kWaves: rows 4 (kWaves q + w) ..
  const uint32_t lane_row = col * kW4K * 2;

  const uint32_t mask_a = w4_scalar(kCodeMask), mask_b = w4_scalar(kCodeMask << 4);
  const uint32_t magic_a = w4_vector(kMagicF16A), magic_b = w4_vector(kMagicF16B);

  f32x4_t acc[NT][kRT];
#pragma unroll
  for (int t = 0; t < NT; ++t)
#pragma unroll
    for (int a = 0; a < kRT; ++a) acc[t][a] = f32x4_t{0.f, 0.f, 0.f, 0.f};

#pragma unroll
  for (int q = 0; q < x_loads<NT, kWaves>(); ++q) dma16(xr, fill + q * 1024 * kWaves, src[q], (uint32_t)k0 * kW4K * 2);
  for (int i = tid; i < kRows; i += 64 * kWaves) {  // published by a later barrier
    const int pos = pos0 + min(i, m - 1);
    const uint32_t r = p.perm != nullptr ? (uint32_t)p.perm[pos] : (uint32_t)pos;
    row_of[i] = r;
    row_up[i] = p.up[r / (uint32_t)p.x_div];
  }
  for (int kt = k0; kt < k1; ++kt) {
    const bool more = kt + 1 < k1;
    // This step's x and codes were asked for a whole step ago; every wave has
    // finished with the buffer that is filled next: its reads of it have ended
    // (lgkmcnt), which the barrier itself does not wait for.
    asm volatile("s_waitcnt vmcnt(0) lgkmcnt(0)" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    uint4 b[kRT][4];
    float sc[kRT][SUB];
#pragma unroll
    for (int a = 0; a < kRT; ++a) {
      const uint32_t cw[4] = {code[a].x, code[a].y, code[a].z, code[a].w};
#pragma unroll
      for (int s = 0; s < SUB; ++s) {
        sc[a][s] = par[a].scale(s);
        const float z32 = par[a].zero32(s);
        const _Float16 za = (_Float16)(-224.f - z32), zb = (_Float16)(16.f - z32);  // -(256 + z), -(16 + z)
        const f16x2_t zza = {za, za}, zzb = {zb, zb};
        auto sum = [](uint32_t v, f16x2_t z) { return __builtin_bit_cast(uint32_t, __builtin_bit_cast(f16x2_t, v) + z); };
#pragma unroll
        for (int j = s * (4 / SUB); j < (s + 1) * (4 / SUB); ++j) {
          const uint32_t lo = cw[j], hi = __builtin_amdgcn_alignbit(lo, lo, 8);
          b[a][j] = make_uint4(sum((lo & mask_a) | magic_a, zza), sum((lo & mask_b) | magic_b, zzb),
                               sum((hi & mask_a) | magic_a, zza), sum((hi & mask_b) | magic_b, zzb));
        }
      }
    }
    // Past the last tile its codes are read again: without a branch the loads
    // go straight into the registers that have just been read.
    fetch(more ? kt + 1 : kt);
    const int cur = (kt - k0) & 1;
    gemm_step<SUB, NT, kWaves, kRT>(lds + cur * stage_bytes<NT>(), fill + (cur ^ 1) * stage_bytes<NT>(), more, xr, src,
                             (uint32_t)(kt + 1) * kW4K * 2, b, sc, lane_row, h, col, acc);
  }

  // ---- y: times the row's power of two, through LDS, so that a row's outputs
  // of a wave leave 16 bytes per lane, as whole lines.
  constexpr int kEb = F32OUT ? 4 : 2, kPieces = kRT * kEb, kRowsAt = 64 / kPieces;  // 16-byte pieces per row
  constexpr int kLd = 16 * kPieces + 16;                                           // its bytes per row in LDS
  static_assert(kWaves * 16 * kLd <= 2 * stage_bytes<NT>(), "the output block fits the stage buffers");
  __syncthreads();  // x has been read
  char* mine = lds + w * 16 * kLd;
  char* y = p.y + (F32OUT ? (int64_t)blockIdx.y * p.R * p.ldy_bytes : 0);
#pragma unroll
  for (int t = 0; t < NT; ++t) {
#pragma unroll
    for (int v = 0; v < 4; ++v) {
      const float u = row_up[16 * t + 4 * h + v];
#pragma unroll
      for (int a = 0; a < kRT; ++a) {
        char* at = mine + (4 * h + v) * kLd + kEb * (16 * a + col);
        if constexpr (F32OUT) *reinterpret_cast<float*>(at) = acc[t][a][v] * u;
        else *reinterpret_cast<uint16_t*>(at) = (uint16_t)f32_to_bf16(acc[t][a][v] * u);
      }
    }
    asm volatile("" ::: "memory");  // a wave's LDS operations are in order
#pragma unroll
    for (int i = 0; i < 16 / kRowsAt; ++i) {
      const int row = kRowsAt * i + lane / kPieces, piece = lane % kPieces;
      const int o = o0 + 16 * kRT * w + (16 / kEb) * piece;
      if (16 * t + row < m && o < p.d_out)
        st16(y + (int64_t)row_of[16 * t + row] * p.ldy_bytes + kEb * (int64_t)o, ld16(mine + row * kLd + 16 * piece));
    }
    asm volatile("" ::: "memory");
  }
}

template <int KIND, int SUB, int NT>
hipError_t launch_nt(const W4GemmArgs& a, bool f32_out, hipStream_t stream) {
  const int64_t grid = (int64_t)a.tiles_o * a.tiles_t;
  if (grid > 0x7fffffff) return hipErrorInvalidValue;
  const unsigned splits = (unsigned)((a.k_tiles + a.per_split - 1) / a.per_split);
  if (f32_out) hipLaunchKernelGGL((w4_gemm_kernel<KIND, SUB, NT, true>), dim3((unsigned)grid, splits), dim3(64 * gemm_waves(SUB)), 0, stream, a);
  else hipLaunchKernelGGL((w4_gemm_kernel<KIND, SUB, NT, false>), dim3((unsigned)grid, splits), dim3(64 * gemm_waves(SUB)), 0, stream, a);
  return hipGetLastError();
}
template <int KIND, int SUB>
hipError_t launch_rows(const W4GemmArgs& a, int bm, bool f32_out, hipStream_t stream) {
  return bm == kW4BigTile ? launch_nt<KIND, SUB, kW4BigTile / 16>(a, f32_out, stream)
                          : launch_nt<KIND, SUB, kW4SmallTile / 16>(a, f32_out, stream);
}

}  // namespace

hipError_t launch_w4_gemm(const W4Call& c, hipStream_t stream) {
  const lora_w4_store& s = c.s;
  const W4Plan& pl = c.plan;
  const int kind = w4_param_kind(s.scale_dtype, s.has_zeros), sub = w4_sub(s.group);
  W4GemmArgs a{};
  a.codes = reinterpret_cast<const char*>(s.codes);
  a.params = reinterpret_cast<const char*>(s.params);
  a.code_stride = w4_code_bytes(1, s.d_in, s.d_out);
  a.param_stride = w4_params_bytes(1, s.d_in, s.d_out, kind, sub);
  a.n = s.n;
  a.k_tiles = w4_k_tiles(s.d_in);
  a.row_tiles = w4_row_tiles(s.d_out);
  a.d_out = s.d_out;
  a.x_div = c.x_div;
  a.R = c.R;
  a.per_split = pl.per_split;
  a.xs = c.ws + pl.xs;
  a.up = reinterpret_cast<const float*>(c.ws + pl.up);
  const int x_rows = c.R / c.x_div;
  W4GroupArgs g{};
  if (c.ids != nullptr) {
    g.ids = c.ids;
    g.R = c.R;
    g.n = s.n;
    g.chunks = (c.R + kChunk - 1) / kChunk;
    g.bm = pl.bm;
    g.hist = reinterpret_cast<int32_t*>(c.ws + pl.hist);
    g.perm = reinterpret_cast<int32_t*>(c.ws + pl.perm);
    g.tiles = reinterpret_cast<int4*>(c.ws + pl.tiles);
    g.n_tiles = g.hist + (int64_t)g.chunks * (s.n + 1);
  }
  hipLaunchKernelGGL(w4_f16_kernel, dim3((unsigned)(g.chunks + (x_rows + 3) / 4)), dim3(256), 0, stream,
                     reinterpret_cast<const char*>(c.x), c.ldx * 2, x_rows, s.d_in, a.k_tiles * kW4K, c.ws + pl.xs,
                     reinterpret_cast<float*>(c.ws + pl.up), g);
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  a.tiles_o = (s.d_out + kCols - 1) / kCols;
  a.tiles_t = (c.R + pl.bm - 1) / pl.bm;
  if (c.ids != nullptr) {
    hipLaunchKernelGGL(w4_place_kernel, dim3((unsigned)g.chunks), dim3(kGroupThreads), 0, stream, g);
    if ((e = hipGetLastError()) != hipSuccess) return e;
    a.perm = g.perm;
    a.tiles = g.tiles;
    a.n_tiles = g.n_tiles;
    a.tiles_t = (int)w4_max_tiles(c.R, s.n, pl.bm);
  }
  const bool f32_out = pl.keep_parts;
  a.y = f32_out ? c.ws + pl.part : reinterpret_cast<char*>(c.y);
  a.ldy_bytes = f32_out ? (int64_t)s.d_out * 4 : c.ldy * 2;
  switch (kind * 8 + sub) {
    case kW4Bf16 * 8 + 1: return launch_rows<kW4Bf16, 1>(a, pl.bm, f32_out, stream);
    case kW4Bf16 * 8 + 2: return launch_rows<kW4Bf16, 2>(a, pl.bm, f32_out, stream);
    case kW4Bf16 * 8 + 4: return launch_rows<kW4Bf16, 4>(a, pl.bm, f32_out, stream);
    case kW4Bf16Zero * 8 + 1: return launch_rows<kW4Bf16Zero, 1>(a, pl.bm, f32_out, stream);
    case kW4Bf16Zero * 8 + 2: return launch_rows<kW4Bf16Zero, 2>(a, pl.bm, f32_out, stream);
    case kW4Bf16Zero * 8 + 4: return launch_rows<kW4Bf16Zero, 4>(a, pl.bm, f32_out, stream);
    case kW4F32 * 8 + 1: return launch_rows<kW4F32, 1>(a, pl.bm, f32_out, stream);
    case kW4F32 * 8 + 2: return launch_rows<kW4F32, 2>(a, pl.bm, f32_out, stream);
    default: return launch_rows<kW4F32, 4>(a, pl.bm, f32_out, stream);
  }
}

}  // namespace lora
