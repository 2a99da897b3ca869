// A call of the 4-bit base products: the kernel its plan names, then, where
// rows were kept in float32 (weights, or splits of the inputs), their sums.
#include "host_util.h"
#include "w4_kernels.h"
#include "w4_ops.h"

namespace lora {
namespace {

// y[t] = sum_j w[t, j] (part[0][t k + j] + part[1][t k + j] + ...), in order of
// j and of the splits; ids without a matrix add nothing.  Without weights k
// is 1.  One thread per 4 outputs.
struct W4SumArgs {
  const float* part;  // [splits][R][d_out]
  int splits, R, k, n, d_out;
  const int32_t* ids;
  const float* weights;
  char* y;
  int64_t ldy_bytes;
};
template <typename E>
__global__ __launch_bounds__(256) void w4_sum_kernel(const W4SumArgs p) {
  const int o = 4 * (int)(blockIdx.y * 256 + threadIdx.x);
  const int t = (int)blockIdx.x;
  if (o >= p.d_out) return;
  f32x4_t s = {0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < p.k; ++j) {
    const int64_t r = (int64_t)t * p.k + j;
    if (p.ids != nullptr && (unsigned)p.ids[r] >= (unsigned)p.n) continue;
    const float* src = p.part + r * p.d_out + o;
    f32x4_t v = *reinterpret_cast<const f32x4_t*>(src);
#pragma unroll 8
    for (int z = 1; z < p.splits; ++z) v += *reinterpret_cast<const f32x4_t*>(src + (int64_t)z * p.R * p.d_out);
    if (p.weights == nullptr) {
      s = v;
    } else {
      const float wt = p.weights[r];
#pragma unroll
      for (int i = 0; i < 4; ++i) s[i] = fmaf(wt, v[i], s[i]);
    }
  }
  char* dst = p.y + (int64_t)t * p.ldy_bytes + (int64_t)o * E::kBytes;
  if constexpr (E::kBytes == 2)
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
  else
    *reinterpret_cast<f32x4_t*>(dst) = s;
}

}  // namespace

hipError_t launch_w4(const W4Call& c, hipStream_t stream) {
  const W4Plan& pl = c.plan;
  hipError_t e = pl.bm > 0 ? launch_w4_gemm(c, stream)
                           : (c.dtype == LORA_DTYPE_BF16 ? launch_w4_rows_bf16(c, stream) : launch_w4_rows_f32(c, stream));
  if (e != hipSuccess || !pl.keep_parts) return e;
  W4SumArgs a{};
  a.part = reinterpret_cast<const float*>(c.ws + pl.part);
  a.splits = pl.splits;
  a.R = c.R;
  a.k = c.weights ? c.k : 1;
  a.n = c.s.n;
  a.d_out = c.s.d_out;
  a.ids = c.ids;
  a.weights = c.weights;
  a.y = reinterpret_cast<char*>(c.y);
  a.ldy_bytes = c.ldy * elem_bytes(c.dtype);
  const dim3 grid((unsigned)(c.R / a.k), (unsigned)((a.d_out / 4 + 255) / 256));
  if (c.dtype == LORA_DTYPE_BF16) hipLaunchKernelGGL((w4_sum_kernel<BF16>), grid, dim3(256), 0, stream, a);
  else hipLaunchKernelGGL((w4_sum_kernel<F32>), grid, dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace lora
