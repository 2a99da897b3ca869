// Launchers of the 4-bit base products and of the router (called by
// w4_api.hip); every launcher only enqueues work on `stream`.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "w4.h"

namespace lora {

hipError_t launch_w4_pack(const lora_w4_store& s, const uint8_t* q, const void* scales, const uint8_t* zeros,
                          void* codes, void* params, hipStream_t stream);

// One product call: rows r = 0 .. R - 1, row r from x row r / x_div, with the
// matrix ids[r] (ids == nullptr: matrix 0).
struct W4Call {
  lora_w4_store s;
  int dtype;
  const void* x;
  int64_t ldx;
  int x_div;
  void* y;
  int64_t ldy;
  int R;
  const int32_t* ids;
  const float* weights;  // per row; with them y row t is the weighted sum of rows t k .. t k + k - 1
  int k;
  W4Plan plan;
  char* ws;
};
hipError_t launch_w4(const W4Call& c, hipStream_t stream);
hipError_t launch_w4_rows_bf16(const W4Call& c, hipStream_t stream);
hipError_t launch_w4_rows_f32(const W4Call& c, hipStream_t stream);
hipError_t launch_w4_gemm(const W4Call& c, hipStream_t stream);

struct RouteArgs {
  const void* logits;
  int64_t ldl;
  int T, E, k, score;
  const float* bias;
  int groups, top_groups, renormalize;
  float scale;
  int32_t* ids;
  float* weights;
};
hipError_t launch_route(const RouteArgs& a, int dtype, hipStream_t stream);

}  // namespace lora
