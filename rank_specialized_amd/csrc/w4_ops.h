// Device-side pieces of the 4-bit base products.
#pragma once
#include "device_common.h"
#include "w4.h"

namespace lora {

// Four operand dwords (two numbers each) of a lane's eight codes: each half
// of `magic` is 16.0 in bf16 (0x4180) or 128.0 in f16 (0x5800), whose last
// bits the code takes: 16 + q, 128 + q, exact.  `mask` and `magic` come from
// w4_scalar and w4_vector, so that each step is one v_and_or_b32.
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
constexpr uint32_t kCodeMask = 0x00780078u;
// q - z itself, exact in bf16 (at most five bits): the eight numbers widened,
// 16 + z taken off, the halves put together again (27 instructions for eight
// codes against 7).
__device__ __forceinline__ uint4 w4_expand_exact(uint32_t w, uint32_t mask, uint32_t magic, float zero16) {
  const uint4 v = w4_expand(w, mask, magic);
  const uint32_t in[4] = {v.x, v.y, v.z, v.w};
  uint32_t out[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float lo = bf16_lo(in[i]) - zero16, hi = bf16_hi(in[i]) - zero16;
    out[i] = __builtin_amdgcn_perm(__float_as_uint(hi), __float_as_uint(lo), 0x07060302u);
  }
  return make_uint4(out[0], out[1], out[2], out[3]);
}
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

// What the row kernels are called with.
struct W4RowsArgs {
  const char* codes;
  const char* params;
  int64_t code_stride, param_stride;  // bytes per matrix
  int n, k_tiles, row_tiles, d_in, d_out;
  const char* x;
  int64_t ldx_bytes;
  int x_div;
  char* y;  // rows of the output type, or of float32 (f32_out)
  int64_t ldy_bytes;
  int R, k;
  const int32_t* ids;    // nullptr: matrix 0
  const float* weights;  // a token's rows summed by one workgroup
  int by_row;            // routed: blockIdx.y is a row (the first row of its matrix works), else a matrix
  int f32_out;
  int row_cap;           // rows that the kernel holds in LDS at a time
};

constexpr int kListMax = 4096;  // rows of a routed call that are listed at a time

template <typename E>
__device__ __forceinline__ void w4_store(char* row, int o, float v, int f32_out) {
  if (E::kBytes == 4 || f32_out) reinterpret_cast<float*>(row)[o] = v;
  else reinterpret_cast<uint16_t*>(row)[o] = (uint16_t)f32_to_bf16(v);
}

// The rows of [win, win + kListMax) whose id is e (or, `none`, outside
// [0, n)), ascending, into `list`; returns their number.  Per chunk of 64 W
// rows, each wave counts its 64 by ballot and the waves' counts are added up
// in order.
template <int W>
__device__ __forceinline__ int w4_rows_of(const W4RowsArgs& p, int e, bool none, int win, uint16_t* list, int* s_cnt) {
  const int tid = (int)threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int end = min(p.R, win + kListMax);
  int cnt = 0;
  for (int r0 = win; r0 < end; r0 += 64 * W) {
    const int r = r0 + tid;
    const int id = r < end ? p.ids[r] : 0;
    const bool hit = r < end && (none ? (unsigned)id >= (unsigned)p.n : id == e);
    const uint64_t mask = __ballot(hit);
    if (lane == 0) s_cnt[w] = __popcll(mask);
    __syncthreads();
    int before = cnt, total = cnt;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      before += i < w ? s_cnt[i] : 0;
      total += s_cnt[i];
    }
    if (hit) list[before + __popcll(mask & lanemask_lt())] = (uint16_t)(r - win);
    cnt = total;
    __syncthreads();
  }
  return cnt;
}

// Empty sums: outputs [o0, o0 + width) of `cnt` listed rows.
template <typename E>
__device__ __forceinline__ void w4_zero_rows(const W4RowsArgs& p, int win, const uint16_t* list, int cnt, int o0, int width) {
  for (int i = (int)threadIdx.x; i < cnt * width; i += (int)blockDim.x) {
    const int o = o0 + i % width;
    if (o < p.d_out) w4_store<E>(p.y + (int64_t)(win + list[i / width]) * p.ldy_bytes, o, 0.f, p.f32_out);
  }
}

}  // namespace lora
