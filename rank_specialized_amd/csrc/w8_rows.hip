// 8-bit base products for few rows (the decode step, and batches of some):
//
//   y[t, o] = s_x[t] s_w[o] sum_k q_x[t, k] q_w[o, k]
//
// What bounds it is the stream of codes.  A workgroup owns 16 RT outputs of 16
// NT rows, and its waves take the 64-input tiles in turn, U of them ahead, each
// adding its own sums in 32-bit integers; they meet in LDS, where integer
// additions give the same sum in any order.  Codes of weights are matrix-core
// operands as they lie in memory.  Rows go through LDS, a piece of it for each
// wave, by loads that write it directly: a wave waits for its own loads, no
// barrier is needed.  (Read from memory as operands, 16 bytes of 16 rows per
// load, they took four times as long as rows of 64 bytes do: 64 rows 3584 -> 512
// 11.7 us, and 7.5 so.)  Or, for the few rows of a decode step, every workgroup
// rounds them itself into LDS: one launch less, while its first codes are on
// their way.
#include "host_util.h"
#include "w8_kernels.h"
#include "w8_ops.h"

namespace lora {
namespace {

struct W8RowsArgs {
  const char* codes;
  const float* scales;
  int k_tiles, d_in, d_out;
  const int8_t* q;
  int64_t ldq;
  const float* s;
  const char* x;  // FUSED
  int64_t ldx_bytes;
  char* y;
  int64_t ldy_bytes;
  int T;
};

// 1 KiB of a tile of 16 rows x 64 inputs into LDS: slot i of a row holds piece
// i ^ (row / 4 % 4), so that the rows of one matrix-core read lie on all banks.
__device__ __forceinline__ void dma_rows(const int8_t* src, char* dst) {
  __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)src,
                                   (__attribute__((address_space(3))) void*)dst, 16, 0, 0);
}
// The products of a tile: its rows at `rd`, while those of a later one go to
// `wr`, another buffer, which restrict tells the compiler: no read waits for the
// loads in flight.  Then the later one's codes.
template <int RT, int NT>
__device__ __forceinline__ void ring_step(const char* __restrict__ rd, char* __restrict__ wr, const int8_t* const (&src)[NT],
                                          const char* next_code, uint4 (&code)[RT], i32x4_t (&acc)[RT][NT]) {
#pragma unroll
  for (int t = 0; t < NT; ++t) dma_rows(src[t], wr + t * kW8TileBytes);
#pragma unroll
  for (int t = 0; t < NT; ++t) {
    const uint4 x = ld16(rd + t * kW8TileBytes);
#pragma unroll
    for (int a = 0; a < RT; ++a) acc[a][t] = mfma_i8(code[a], x, acc[a][t]);
  }
#pragma unroll
  for (int a = 0; a < RT; ++a) code[a] = ld16(next_code + a * kW8TileBytes);
}
// Wait until at most N of the wave's loads are in flight, and its LDS reads have
// ended.
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0070);
  asm volatile("" ::: "memory");
}

template <typename E, int RT, int NT, int U, int W, bool FUSED>
__global__ __launch_bounds__(64 * W) __attribute__((amdgpu_waves_per_eu(2)))
void w8_rows_kernel(const W8RowsArgs p) {
  constexpr int kHold = 5 * 512 / (64 * W);  // pieces of 8 values per thread (FUSED): kW8FusedValues in all
  static_assert(!FUSED || NT == 1, "few rows");
  extern __shared__ __align__(16) char lds[];  // FUSED: rows of codes; else the waves' rings [W][U + 1][NT] KiB
  __shared__ __align__(16) int sums[RT * NT * 256];
  __shared__ uint32_t tops[kW8FusedRows];
  const int tid = (int)threadIdx.x, lane = tid & 63, col = lane & 15, h = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);
  const int blk = (int)blockIdx.x / (4 / RT), b0 = (int)blockIdx.x % (4 / RT) * RT;
  const int t0 = (int)blockIdx.y * 16 * NT, m = min(p.T - t0, 16 * NT);
  const char* code0 = p.codes + (int64_t)blk * p.k_tiles * kW8BlockBytes + b0 * kW8TileBytes + 16 * lane;

  // ---- FUSED: the rows' values are asked for first.  A wave-wide load takes
  // 512 values of one row.
  const int per_row = (p.d_in + 511) / 512, loads = FUSED ? m * per_row : 0;
  W8Piece<E> hold[FUSED ? kHold : 1];
  if constexpr (FUSED) {
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      const int f = min(w + i * W, loads - 1), row = f / per_row, k = 512 * (f - row * per_row) + 8 * lane;
      hold[i].load(p.x + (int64_t)row * p.ldx_bytes + (int64_t)min(k, p.d_in - 8) * E::kBytes);
    }
  }
  i32x4_t acc[RT][NT];
#pragma unroll
  for (int a = 0; a < RT; ++a)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[a][t] = i32x4_t{0, 0, 0, 0};
  uint4 code[U][RT];
  const auto code_of = [&](int i) { return code0 + (int64_t)min(i, p.k_tiles - 1) * kW8BlockBytes; };

  if constexpr (FUSED) {
#pragma unroll
    for (int u = 0; u < U; ++u)
#pragma unroll
      for (int a = 0; a < RT; ++a) code[u][a] = ld16(code_of(w + u * W) + a * kW8TileBytes);
    for (int i = tid; i < RT * NT * 256; i += 64 * W) sums[i] = 0;
    if (tid < kW8FusedRows) tops[tid] = 0u;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kHold; ++i)
      if (w + i * W < loads) {
        const uint32_t top = wave_max_u32(hold[i].top(0u));
        if (lane == 0) atomicMax(&tops[(w + i * W) / per_row], top);
      }
    __syncthreads();
    const int stride = p.k_tiles * kW8K + 16;
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      const int f = w + i * W, row = f / per_row, k = 512 * (f - row * per_row) + 8 * lane;
      if (f < loads && k < p.k_tiles * kW8K) {
        const W8Round r(tops[row]);
        *reinterpret_cast<uint2*>(lds + row * stride + k) = hold[i].codes(r);
      }
    }
    __syncthreads();
    const char* xl = lds + min(col, m - 1) * stride + 16 * h;
    for (int i0 = w; i0 < p.k_tiles; i0 += U * W) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * W;
        if (i < p.k_tiles) {
          const uint4 x = ld16(xl + i * kW8K);
#pragma unroll
          for (int a = 0; a < RT; ++a) acc[a][0] = mfma_i8(code[u][a], x, acc[a][0]);
        }
#pragma unroll
        for (int a = 0; a < RT; ++a) code[u][a] = ld16(code_of(i + U * W) + a * kW8TileBytes);
      }
    }
  } else {
    // ---- rows: lane l of a load takes piece l % 4 ^ (l / 16) of row l / 4 of 16.
    // Rows past m repeat the last; pieces past d_in the last one (their weights
    // are zeros).
    const int last_piece = (p.d_in - 1) & ~15, piece = ((lane & 3) ^ (lane >> 4)) << 4;
    const int8_t* row[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) row[t] = p.q + (int64_t)(t0 + min(16 * t + (lane >> 2), m - 1)) * p.ldq;
    constexpr int kSlot = NT * kW8TileBytes, kPer = RT + NT;  // loads of a tile
    char* ring = lds + w * (U + 1) * kSlot;
    const int rd = col * kW8K + ((h ^ (col >> 2)) << 4);
    const auto sources = [&](int i, const int8_t* (&src)[NT]) {
      const int k = min(min(i, p.k_tiles - 1) * kW8K + piece, last_piece);
#pragma unroll
      for (int t = 0; t < NT; ++t) src[t] = row[t] + k;
    };
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int8_t* src[NT];
      sources(w + u * W, src);
#pragma unroll
      for (int t = 0; t < NT; ++t) dma_rows(src[t], ring + u * kSlot + t * kW8TileBytes);
#pragma unroll
      for (int a = 0; a < RT; ++a) code[u][a] = ld16(code_of(w + u * W) + a * kW8TileBytes);
      asm volatile("" ::: "memory");
    }
    for (int i = tid; i < RT * NT * 256; i += 64 * W) sums[i] = 0;
    wait_loads<0>();  // the compiler then knows of no load into what the loop reads first
    int at = 0, i = w;  // the slot of tile i; the one before it takes tile i + U W
    const auto turn = [&](int u) {
      const int8_t* src[NT];
      sources(i + U * W, src);
      wait_loads<kPer*(U - 1)>();
      ring_step<RT, NT>(ring + at * kSlot + rd, ring + (at == 0 ? U : at - 1) * kSlot, src, code_of(i + U * W), code[u], acc);
      at = at == U ? 0 : at + 1;
      i += W;
    };
    while (i + (U - 1) * W < p.k_tiles) {
#pragma unroll
      for (int u = 0; u < U; ++u) turn(u);
    }
#pragma unroll
    for (int u = 0; u < U - 1; ++u)
      if (i < p.k_tiles) turn(u);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // no load may write LDS that is another workgroup's
    __syncthreads();                                  // the sums are zeros
  }
#pragma unroll
  for (int a = 0; a < RT; ++a)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int v = 0; v < 4; ++v) atomicAdd(&sums[(a * NT + t) * 256 + 64 * v + lane], acc[a][t][v]);
  __syncthreads();

  // ---- y: four outputs of a row per thread
  for (int i = tid; i < RT * NT * 64; i += 64 * W) {
    const int l = i & 63, t = (i >> 6) % NT, a = (i >> 6) / NT, row = 16 * t + (l & 15);
    const int o = blk * kW8Block + w8_output(b0 + a, 4 * (l >> 4));
    if (row >= m || o >= p.d_out) continue;
    float sx;
    if constexpr (FUSED) sx = W8Round(tops[row]).scale;
    else sx = p.s[t0 + row];
    const f32x4_t sw = *reinterpret_cast<const f32x4_t*>(p.scales + o);
    float f[4];
#pragma unroll
    for (int v = 0; v < 4; ++v) f[v] = (float)sums[(a * NT + t) * 256 + 64 * v + l] * sx * sw[v];
    char* dst = p.y + (int64_t)(t0 + row) * p.ldy_bytes + (int64_t)o * E::kBytes;
    if constexpr (E::kBytes == 2) *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]));
    else *reinterpret_cast<f32x4_t*>(dst) = f32x4_t{f[0], f[1], f[2], f[3]};
  }
}

template <typename E, int RT, int NT, int U, int W, bool FUSED>
hipError_t launch_one(const W8RowsArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)(w8_blocks(a.d_out) * (4 / RT)), (unsigned)((a.T + 16 * NT - 1) / (16 * NT)));
  const size_t lds = FUSED ? (size_t)a.T * (a.k_tiles * kW8K + 16) : (size_t)W * (U + 1) * NT * kW8TileBytes;
  static DynLdsLimit lim;
  const hipError_t e = ensure_dynamic_lds(lim, reinterpret_cast<const void*>(w8_rows_kernel<E, RT, NT, U, W, FUSED>), lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((w8_rows_kernel<E, RT, NT, U, W, FUSED>), grid, dim3(64 * W), lds, stream, a);
  return hipGetLastError();
}

template <typename E>
hipError_t launch_rows(const W8RowsArgs& a, const W8Plan& pl, hipStream_t stream) {
  if (pl.fused) {
    switch (pl.rt) {
      case 1: return launch_one<E, 1, 1, 4, 8, true>(a, stream);
      case 2: return launch_one<E, 2, 1, 2, 8, true>(a, stream);
      default: return launch_one<E, 4, 1, 2, 8, true>(a, stream);
    }
  }
  switch (10 * pl.rt + pl.nt) {
    case 11: return launch_one<E, 1, 1, 4, 8, false>(a, stream);
    case 21: return launch_one<E, 2, 1, 4, 8, false>(a, stream);
    case 41: return launch_one<E, 4, 1, 2, 8, false>(a, stream);
    case 12: return launch_one<E, 1, 2, 4, 8, false>(a, stream);
    case 22: return launch_one<E, 2, 2, 2, 8, false>(a, stream);
    case 42: return launch_one<E, 4, 2, 2, 8, false>(a, stream);
    default: return launch_one<E, 4, 4, 2, 8, false>(a, stream);
  }
}

}  // namespace

hipError_t launch_w8_rows(const W8Call& c, hipStream_t stream) {
  const int eb = elem_bytes(c.dtype);
  W8RowsArgs a{};
  a.codes = reinterpret_cast<const char*>(c.w.codes);
  a.scales = reinterpret_cast<const float*>(c.w.scales);
  a.k_tiles = w8_k_tiles(c.w.d_in);
  a.d_in = c.w.d_in;
  a.d_out = c.w.d_out;
  a.q = c.q;
  a.ldq = c.ldq;
  a.s = c.s;
  a.x = reinterpret_cast<const char*>(c.x);
  a.ldx_bytes = c.ldx * eb;
  a.y = reinterpret_cast<char*>(c.y);
  a.ldy_bytes = c.ldy * eb;
  a.T = c.T;
  return c.dtype == LORA_DTYPE_BF16 ? launch_rows<BF16>(a, c.plan, stream) : launch_rows<F32>(a, c.plan, stream);
}

}  // namespace lora
