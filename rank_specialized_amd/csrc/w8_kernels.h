// Launchers of the 8-bit base products (called by w8_api.hip); every launcher
// only enqueues work on `stream`.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "w8.h"

namespace lora {

hipError_t launch_w8_pack(int d_in, int d_out, const int8_t* q, const void* scales, int scale_dtype, void* codes,
                          float* out_scales, hipStream_t stream);
hipError_t launch_w8_quantize(int dtype, const void* x, int64_t ldx, int T, int d_in, int8_t* q, int64_t ldq,
                              float* scales, hipStream_t stream);

// One product call: rows of codes q with scales s, or (fused) rows of x.
struct W8Call {
  lora_w8_store w;
  int dtype;  // of y (and x)
  const int8_t* q;
  int64_t ldq;
  const float* s;
  const void* x;
  int64_t ldx;
  void* y;
  int64_t ldy;
  int T;
  W8Plan plan;
};
hipError_t launch_w8_rows(const W8Call& c, hipStream_t stream);
hipError_t launch_w8_gemm(const W8Call& c, hipStream_t stream);

}  // namespace lora
