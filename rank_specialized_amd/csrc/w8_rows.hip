// 8-bit base products for few rows (the decode step, and batches of some):
//
//   y[t, o] = s_x[t] s_w[o] sum_k q_x[t, k] q_w[o, k]
//
// What bounds it is the stream of codes.  A workgroup owns 16 RT outputs of 16
// NT rows, and its waves take the 64-input tiles in turn, U of them ahead, each
// adding its own sums in 32-bit integers; they meet in LDS, where integer
// additions give the same sum in any order.  The rows' codes come from memory
// (the L2, mostly) as matrix-core operands, or, for the few rows of a decode
// step, every workgroup rounds them itself into LDS: one launch less, while its
// first codes are on their way.
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

template <typename E, int RT, int NT, int U, int W, bool FUSED>
__global__ __launch_bounds__(64 * W) __attribute__((amdgpu_waves_per_eu(2)))
void w8_rows_kernel(const W8RowsArgs p) {
  constexpr int kHold = 5 * 512 / (64 * W);  // pieces of 8 values per thread (FUSED): kW8FusedValues in all
  static_assert(!FUSED || NT == 1, "few rows");
  extern __shared__ __align__(16) char lds[];  // FUSED: rows of codes
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
  const int last_piece = (p.d_in - 1) & ~15;
  const int8_t* xrow[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) xrow[t] = FUSED ? nullptr : p.q + (int64_t)(t0 + min(16 * t + col, m - 1)) * p.ldq;
  const int stride = p.k_tiles * kW8K + 16;
  uint4 code[U][RT], xq[U][FUSED ? 1 : NT];
  auto fetch = [&](int u, int kt) {
#pragma unroll
    for (int a = 0; a < RT; ++a) code[u][a] = ld16(code0 + (int64_t)kt * kW8BlockBytes + a * kW8TileBytes);
    if constexpr (!FUSED)
#pragma unroll
      for (int t = 0; t < NT; ++t) xq[u][t] = ld16(xrow[t] + min(kt * kW8K + 16 * h, last_piece));
  };
#pragma unroll
  for (int u = 0; u < U; ++u) fetch(u, min(w + u * W, p.k_tiles - 1));

  for (int i = tid; i < RT * NT * 256; i += 64 * W) sums[i] = 0;
  if constexpr (FUSED) {
    if (tid < kW8FusedRows) tops[tid] = 0u;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kHold; ++i)
      if (w + i * W < loads) {
        const uint32_t top = wave_max_u32(hold[i].top(0u));
        if (lane == 0) atomicMax(&tops[(w + i * W) / per_row], top);
      }
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kHold; ++i) {
      const int f = w + i * W, row = f / per_row, k = 512 * (f - row * per_row) + 8 * lane;
      if (f < loads && k < p.k_tiles * kW8K) {
        const W8Round r(tops[row]);
        *reinterpret_cast<uint2*>(lds + row * stride + k) = hold[i].codes(r);
      }
    }
  }
  __syncthreads();

  i32x4_t acc[RT][NT];
#pragma unroll
  for (int a = 0; a < RT; ++a)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[a][t] = i32x4_t{0, 0, 0, 0};
  const char* xl = lds + (FUSED ? min(col, m - 1) * stride : 0) + 16 * h;
  for (int i0 = w; i0 < p.k_tiles; i0 += U * W) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int i = i0 + u * W;
      if (i < p.k_tiles) {
        if constexpr (FUSED) xq[u][0] = ld16(xl + i * kW8K);
#pragma unroll
        for (int a = 0; a < RT; ++a)
#pragma unroll
          for (int t = 0; t < NT; ++t) acc[a][t] = mfma_i8(code[u][a], xq[u][t], acc[a][t]);
      }
      fetch(u, min(i + U * W, p.k_tiles - 1));
    }
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
  const size_t lds = FUSED ? (size_t)a.T * (a.k_tiles * kW8K + 16) : 0;
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
  if (pl.nt == 4) return launch_one<E, 4, 4, 1, 8, false>(a, stream);
  if (pl.nt == 2) {
    switch (pl.rt) {
      case 1: return launch_one<E, 1, 2, 4, 8, false>(a, stream);
      case 2: return launch_one<E, 2, 2, 2, 8, false>(a, stream);
      default: return launch_one<E, 4, 2, 2, 8, false>(a, stream);
    }
  }
  switch (pl.rt) {
    case 1: return launch_one<E, 1, 1, 4, 8, false>(a, stream);
    case 2: return launch_one<E, 2, 1, 4, 8, false>(a, stream);
    default: return launch_one<E, 4, 1, 2, 8, false>(a, stream);
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
