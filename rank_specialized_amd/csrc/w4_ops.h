// Device-side pieces of the 4-bit base products.
#pragma once
#include "device_common.h"
#include "w4.h"

namespace lora {

// Four operand dwords (two numbers each) of a lane's eight codes: each half
// of `magic` is 32.0 in bf16 (0x4200), whose last bits the code takes: 32 + q,
// exact.  `mask` and `magic` come from w4_scalar and w4_vector, so that each
// step is one v_and_or_b32.
__device__ __forceinline__ uint4 w4_expand(uint32_t w, uint32_t mask, uint32_t magic) {
  return make_uint4((w & mask) | magic, ((w >> 4) & mask) | magic, ((w >> 8) & mask) | magic,
                    (__builtin_amdgcn_alignbit(w, w, 12) & mask) | magic);
}
// Constants the compiler takes for values, one in a scalar and one in a vector
// register: v_and_or_b32 takes no literals and one scalar operand, and would
// be two instructions otherwise.  (The and-or itself stays out of inline
// assembly: a matrix instruction must not read a register within two wait
// states of its write, and the compiler cannot see one there.)
__device__ __forceinline__ uint32_t w4_scalar(uint32_t v) {
  uint32_t r;
  asm("s_mov_b32 %0, %1" : "=s"(r) : "i"(v));
  return r;
}
__device__ __forceinline__ uint32_t w4_vector(uint32_t v) {
  uint32_t r;
  asm("v_mov_b32 %0, %1" : "=v"(r) : "s"(w4_scalar(v)));
  return r;
}
constexpr uint32_t kCodeMask = 0x003c003cu;
// q - z itself, exact in bf16 (at most five bits): the eight numbers widened,
// 32 + z taken off, the halves put together again (27 instructions for eight
// codes against 7).
__device__ __forceinline__ uint4 w4_expand_exact(uint32_t w, uint32_t mask, uint32_t magic, float zero32) {
  const uint4 v = w4_expand(w, mask, magic);
  const uint32_t in[4] = {v.x, v.y, v.z, v.w};
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float lo = bf16_lo(in[i]) - zero32, hi = bf16_hi(in[i]) - zero32;
    out[i] = __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}
constexpr uint32_t kMagicBf16 = 0x42004200u;
// f16: a code on bits 2..5 of 256 (step 1/4), on bits 6..9 of 16 (step 1/64)
constexpr uint32_t kMagicF16A = 0x5c005c00u, kMagicF16B = 0x4c004c00u;

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
  __device__ __forceinline__ void load(rsrc_t r, uint32_t voff, uint32_t soff) {
    if constexpr (kBytes == 2) {
      w[0] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b16(r, voff, soff, 0);
    } else if constexpr (kBytes == 4) {
      w[0] = (uint32_t)__builtin_amdgcn_raw_buffer_load_b32(r, voff, soff, 0);
    } else if constexpr (kBytes == 8) {
      const uint2 v = __builtin_bit_cast(uint2, __builtin_amdgcn_raw_buffer_load_b64(r, voff, soff, 0));
      w[0] = v.x; w[1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < kBytes / 16; ++i) {
        const uint4 v = buf_ld16(r, voff + 16 * i, soff);
        w[4 * i] = v.x; w[4 * i + 1] = v.y; w[4 * i + 2] = v.z; w[4 * i + 3] = v.w;
      }
    }
  }
  __device__ __forceinline__ float scale(int s) const {
    if constexpr (KIND == kW4Bf16) return (s & 1) ? bf16_hi(w[s >> 1]) : bf16_lo(w[s >> 1]);
    else if constexpr (KIND == kW4Bf16Zero) return bf16_lo(w[s]);
    else return __uint_as_float(w[2 * s]);
  }
  // 32 + z
  __device__ __forceinline__ float zero32(int s) const {
    if constexpr (KIND == kW4Bf16) return 40.f;
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
