// Device-side pieces of the 4-bit base products.
#pragma once
#include "device_common.h"
#include "w4.h"

namespace lora {

// Four operand dwords (two numbers each) of a lane's eight codes: each half
// of `magic` is 16.0 in bf16 (0x4180) or 128.0 in f16 (0x5800), whose last
// bits the code takes: 16 + q, 128 + q, exact.  `mask` and `magic` come from
// w4_constant, so that each step is one v_and_or_b32.
__device__ __forceinline__ uint4 w4_expand(uint32_t w, uint32_t mask, uint32_t magic) {
  return make_uint4((w & mask) | magic, ((w >> 4) & mask) | magic, ((w >> 8) & mask) | magic,
                    (__builtin_amdgcn_alignbit(w, w, 12) & mask) | magic);
}
// A constant the compiler takes for a value: two literals would not fit one
// v_and_or_b32, and it would use two instructions.  (The and-or itself stays
// out of inline assembly: a matrix instruction must not read a register
// within two wait states of its write, and the compiler cannot see one there.)
__device__ __forceinline__ uint32_t w4_constant(uint32_t v) {
  uint32_t r;
  asm("s_mov_b32 %0, %1" : "=s"(r) : "i"(v));
  return r;
}
constexpr uint32_t kCodeMask = 0x00780078u;
constexpr uint32_t kMagicBf16 = 0x41804180u;
constexpr uint32_t kMagicF16 = 0x58005800u;

// A lane's scales and zero points of one tile: SUB groups of its output row.
template <int KIND, int SUB>
struct W4Params {
  static constexpr int kBytes = SUB * w4_param_bytes(KIND);
  static constexpr int kWords = kBytes < 4 ? 1 : kBytes / 4;
  uint32_t w[kWords];
  __device__ __forceinline__ void load(const char* p) {
    if constexpr (kBytes == 2) {
      w[0] = *reinterpret_cast<const uint16_t*>(p);
    } else if constexpr (kBytes == 4) {
      w[0] = *reinterpret_cast<const uint32_t*>(p);
    } else if constexpr (kBytes == 8) {
      const uint2 v = *reinterpret_cast<const uint2*>(p);
      w[0] = v.x; w[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) {
        const uint4 v = ld16(p + 16 * i);
        w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
      }
    }
  }
  __device__ __forceinline__ float scale(int s) const {
    if constexpr (KIND == kW4Bf16) return (s & 1) ? bf16_hi(w[s >> 1]) : bf16_lo(w[s >> 1]);
    else if constexpr (KIND == kW4Bf16Zero) return bf16_lo(w[s]);
    else return __uint_as_float(w[2 * s]);
  }
  // 16 + z
  __device__ __forceinline__ float zero16(int s) const {
    if constexpr (KIND == kW4Bf16) return 24.f;
    else if constexpr (KIND == kW4Bf16Zero) return bf16_hi(w[s]);
    else return __uint_as_float(w[2 * s + 1]);
  }
};

// Eight activations as matrix-core operands: one bf16 operand, or a float32
// value as the exact sum of three (its top 8 bits, the next 8, the rest).
template <typename E>
struct XFrag;
template <>
struct XFrag<BF16> {
  static constexpr int kParts = 1;
  uint4 v;
  __device__ __forceinline__ void load(const char* p) { v = ld16(p); }
  __device__ __forceinline__ void parts(uint4 (&o)[1]) const { o[0] = v; }
};
template <>
struct XFrag<F32> {
  static constexpr int kParts = 3;
  uint4 v[2];
  __device__ __forceinline__ void load(const char* p) {
    v[0] = ld16(p);
    v[1] = ld16(p + 16);
  }
  __device__ __forceinline__ void parts(uint4 (&o)[3]) const {
    const uint32_t in[8] = {v[0].x, v[0].y, v[0].z, v[0].w, v[1].x, v[1].y, v[1].z, v[1].w};
    uint32_t out[3][4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      float a = __uint_as_float(in[2 * i]), b = __uint_as_float(in[2 * i + 1]);
#pragma unroll
      for (int q = 0; q < 3; ++q) {
        const uint32_t ha = __float_as_uint(a) & 0xffff0000u, hb = __float_as_uint(b) & 0xffff0000u;
        out[q][i] = (ha >> 16) | hb;
        a -= __uint_as_float(ha);  // exact: what is left of 24 bits
        b -= __uint_as_float(hb);
      }
    }
#pragma unroll
    for (int q = 0; q < 3; ++q) o[q] = make_uint4(out[q][0], out[q][1], out[q][2], out[q][3]);
  }
};

}  // namespace lora
