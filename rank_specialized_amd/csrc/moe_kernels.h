// Launcher of the mixture-of-experts layer for a few tokens (called by
// moe_api.hip); it only enqueues work on `stream`.
#pragma once
#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe.h"

namespace lora {

struct MoeCall {
  lora_w4_store gate, up, down;
  int dtype, act;
  const void* x;
  int64_t ldx;
  void* y;
  int64_t ldy;
  int T, k;
  const int32_t* ids;
  const float* weights;
  MoePlan plan;
  char* ws;
};
hipError_t launch_moe_bf16(const MoeCall& c, hipStream_t stream);
hipError_t launch_moe_f32(const MoeCall& c, hipStream_t stream);

}  // namespace lora
