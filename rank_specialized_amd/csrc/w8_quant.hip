// Rows rounded to 8-bit integers (lora_w8_quantize), and the layout of an
// 8-bit store (lora_w8_pack).
#include "w8_kernels.h"
#include "w8_ops.h"

namespace lora {
namespace {

// W waves per row: its largest |value|, then its codes.  The first 8 pieces of
// a thread stay in registers between the two; what is behind them is read
// again.
template <typename E, int W>
__global__ __launch_bounds__(W == 1 ? 256 : 64 * W) void w8_quantize_kernel(const char* __restrict__ x, int64_t ldx_bytes, int T, int d_in,
                                                          int8_t* __restrict__ q, int64_t ldq, float* __restrict__ scales) {
  constexpr int kHold = 8 / (E::kBytes / 2), kStep = 64 * W * 8;
  __shared__ uint32_t tops[W];
  const int tid = (int)threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int64_t t = W == 1 ? (int64_t)blockIdx.x * 4 + w : (int64_t)blockIdx.x;
  if (W == 1 && t >= T) return;
  const char* src = x + t * ldx_bytes;
  const int k0 = 8 * (W == 1 ? lane : tid);
  W8Piece<E> hold[kHold];
#pragma unroll
  for (int i = 0; i < kHold; ++i)  // past the end: the last piece again
    hold[i].load(src + (int64_t)min(k0 + i * kStep, d_in - 8) * E::kBytes);
  uint32_t top = 0;
#pragma unroll
  for (int i = 0; i < kHold; ++i) top = hold[i].top(top);
  for (int k = k0 + kHold * kStep; k < d_in; k += kStep) {
    W8Piece<E> v;
    v.load(src + (int64_t)k * E::kBytes);
    top = v.top(top);
  }
  top = wave_max_u32(top);
  if constexpr (W > 1) {
    if (lane == 0) tops[w] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < W; ++i) top = max(top, tops[i]);
  }
  const W8Round r(top);
  int8_t* dst = q + t * ldq;
#pragma unroll
  for (int i = 0; i < kHold; ++i) {
    const int k = k0 + i * kStep;
    if (k < d_in) *reinterpret_cast<uint2*>(dst + k) = hold[i].codes(r);
  }
  for (int k = k0 + kHold * kStep; k < d_in; k += kStep) {
    W8Piece<E> v;
    v.load(src + (int64_t)k * E::kBytes);
    *reinterpret_cast<uint2*>(dst + k) = v.codes(r);
  }
  if (k0 == 0) scales[t] = r.scale;
}

template <typename E>
hipError_t launch_quantize(const void* x, int64_t ldx, int T, int d_in, int8_t* q, int64_t ldq, float* scales,
                           hipStream_t stream) {
  const char* src = reinterpret_cast<const char*>(x);
  // Waves per row: 23 rows of 18944 and their product 17.7 us with 8, 18.5 with 4
  // or 16; 5 rows of 4096 and theirs 9.9, 9.7, 10.4.
  const int64_t ldx_bytes = ldx * E::kBytes;
  if (d_in > 8192 && T < 512) hipLaunchKernelGGL((w8_quantize_kernel<E, 8>), dim3((unsigned)T), dim3(512), 0, stream, src, ldx_bytes, T, d_in, q, ldq, scales);
  else if (d_in > 4096 || (T < 1024 && d_in > 512)) hipLaunchKernelGGL((w8_quantize_kernel<E, 4>), dim3((unsigned)T), dim3(256), 0, stream, src, ldx_bytes, T, d_in, q, ldq, scales);
  else hipLaunchKernelGGL((w8_quantize_kernel<E, 1>), dim3((unsigned)((T + 3) / 4)), dim3(256), 0, stream, src, ldx_bytes, T, d_in, q, ldq, scales);
  return hipGetLastError();
}

// One wave per tile of 16 outputs x 64 inputs, a lane's 16 codes from two
// 8-byte loads (a row of codes is 8-byte aligned); the first tile of a block
// also writes its 64 scales.
__global__ __launch_bounds__(256) void w8_pack_kernel(int d_in, int d_out, int k_tiles, const int8_t* __restrict__ q,
                                                      const void* __restrict__ scales, int scale_dtype,
                                                      char* __restrict__ codes, float* __restrict__ out_scales) {
  const int lane = (int)threadIdx.x & 63, b = (int)threadIdx.x >> 6;
  const int kt = (int)blockIdx.x;
  const int64_t blk = blockIdx.y;
  const int64_t o = blk * kW8Block + w8_output(b, lane & 15);
  const int k = kt * kW8K + 16 * (lane >> 4);
  uint4 v = make_uint4(0u, 0u, 0u, 0u);
  if (o < d_out) {
    const int8_t* src = q + o * d_in + k;
    if (k < d_in) {
      const uint2 a = *reinterpret_cast<const uint2*>(src);
      v.x = a.x; v.y = a.y;
    }
    if (k + 8 < d_in) {
      const uint2 a = *reinterpret_cast<const uint2*>(src + 8);
      v.z = a.x; v.w = a.y;
    }
  }
  st16(codes + (blk * k_tiles + kt) * kW8BlockBytes + b * kW8TileBytes + 16 * lane, v);
  if (kt == 0 && b == 0) {
    const int64_t c = blk * kW8Block + lane;
    float s = 0.f;
    if (c < d_out)
      s = scale_dtype == LORA_DTYPE_F32 ? reinterpret_cast<const float*>(scales)[c]
                                        : bf16_lo(reinterpret_cast<const uint16_t*>(scales)[c]);
    out_scales[c] = s;
  }
}

}  // namespace

hipError_t launch_w8_quantize(int dtype, const void* x, int64_t ldx, int T, int d_in, int8_t* q, int64_t ldq,
                              float* scales, hipStream_t stream) {
  return dtype == LORA_DTYPE_BF16 ? launch_quantize<BF16>(x, ldx, T, d_in, q, ldq, scales, stream)
                                  : launch_quantize<F32>(x, ldx, T, d_in, q, ldq, scales, stream);
}

hipError_t launch_w8_pack(int d_in, int d_out, const int8_t* q, const void* scales, int scale_dtype, void* codes,
                          float* out_scales, hipStream_t stream) {
  const dim3 grid((unsigned)w8_k_tiles(d_in), (unsigned)w8_blocks(d_out));  // at most 2^11 by 2^14
  hipLaunchKernelGGL(w8_pack_kernel, grid, dim3(256), 0, stream, d_in, d_out, w8_k_tiles(d_in), q, scales,
                     scale_dtype, reinterpret_cast<char*>(codes), out_scales);
  return hipGetLastError();
}

}  // namespace lora
