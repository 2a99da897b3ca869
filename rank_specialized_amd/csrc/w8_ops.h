// Device-side pieces of the 8-bit base products.
#pragma once
#include "device_common.h"
#include "w8.h"

namespace lora {

typedef __attribute__((ext_vector_type(4))) int i32x4_t;

// 16 x 16 outputs of 64 inputs, exact sums in 32-bit integers.  Lane l supplies
// row l % 16 of each operand and inputs 16 (l / 16) .. + 15; it holds column
// l % 16, rows 4 (l / 16) .. + 3 of the result.
__device__ __forceinline__ i32x4_t mfma_i8(const uint4& a, const uint4& b, i32x4_t c) {
  return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4_t, a), __builtin_bit_cast(i32x4_t, b), c, 0, 0, 0);
}

// The largest |value| of a row as the bits of a float32, in which order is
// that of the numbers, infinities above every number and NaNs above those.
__device__ __forceinline__ uint32_t w8_top(const BF16&, const uint4& v, uint32_t top) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const uint32_t a = (w[i] << 16) & 0x7fffffffu, b = w[i] & 0x7fff0000u;
    top = max(top, max(a, b));
  }
  return top;
}
__device__ __forceinline__ uint32_t w8_top(const F32&, const uint4& v, uint32_t top) {
  return max(max(max(top, v.x & 0x7fffffffu), max(v.y & 0x7fffffffu, v.z & 0x7fffffffu)), v.w & 0x7fffffffu);
}
__device__ __forceinline__ uint32_t wave_max_u32(uint32_t v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v = max(v, (uint32_t)__shfl_xor((int)v, d));
  return v;
}

// A row's rounding, from its largest |value| a: codes round(127 x / a), the
// even one of two as near, and the scale a / 127; a = 0 gives zeros, an
// infinity or a NaN the scale NaN.
//
// The choice between two codes is that of the exact quotient, in three float64
// operations.  p = x (127 / a) is off by less than 2^-45.  Adding 1.5 2^14
// rounds it to a multiple of 2^-38: a border k + 1/2 is one, so a p that
// belongs on it lands there; one that does not is 2^-33 away or more
// (|254 x - (2 k + 1) a| is a multiple of the last place of x, and a float32
// has 24 bits).  Adding 1.5 2^52 - 1.5 2^14 then rounds to an integer, half to
// even, which the last bits of the sum hold.
struct W8Round {
  double r;
  float scale;
  __device__ explicit W8Round(uint32_t top) {
    const double a = (double)__uint_as_float(top);
    const bool ok = top < 0x7f800000u && top != 0u;
    r = ok ? 127.0 / a : 0.0;
    scale = top < 0x7f800000u ? (float)(a / 127.0) : __uint_as_float(0x7fc00000u);
  }
  __device__ __forceinline__ uint32_t code(float x) const {  // in the low byte
    const double u = fma((double)x, r, 24576.0);
    return (uint32_t)__double_as_longlong(u + (6755399441055744.0 - 24576.0));
  }
  __device__ __forceinline__ uint32_t four(float a, float b, float c, float d) const {
    const uint32_t lo = __builtin_amdgcn_perm(code(b), code(a), 0x0c0c0400u);
    const uint32_t hi = __builtin_amdgcn_perm(code(d), code(c), 0x04000c0cu);
    return lo | hi;
  }
};

// 8 values of x of either type, and their codes.
template <typename E>
struct W8Piece {
  static constexpr int kWords = E::kBytes / 2;  // of 16 bytes
  uint4 v[kWords];
  __device__ __forceinline__ void load(const char* p) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) v[i] = ld16(p + 16 * i);
  }
  __device__ __forceinline__ uint32_t top(uint32_t t) const {
#pragma unroll
    for (int i = 0; i < kWords; ++i) t = w8_top(E{}, v[i], t);
    return t;
  }
  __device__ __forceinline__ uint2 codes(const W8Round& r) const {
    float f[8];
#pragma unroll
    for (int i = 0; i < kWords; ++i) E::widen(v[i], f + i * E::kVec);
    return make_uint2(r.four(f[0], f[1], f[2], f[3]), r.four(f[4], f[5], f[6], f[7]));
  }
};

// Eight consecutive outputs of a row: sums times the row's and the outputs'
// scales.
template <typename E>
__device__ __forceinline__ void w8_store8(char* dst, const i32x4_t& a, const i32x4_t& b, float sx, const f32x4_t& wa,
                                          const f32x4_t& wb) {
  float f[8];
#pragma unroll
  for (int v = 0; v < 4; ++v) {
    f[v] = (float)a[v] * sx * wa[v];
    f[4 + v] = (float)b[v] * sx * wb[v];
  }
#pragma unroll
  for (int i = 0; i < E::kBytes / 2; ++i) st16(dst + 16 * i, E::narrow(f + i * E::kVec));
}

}  // namespace lora
