// Argument checks that the entry points with 4-bit stores share (host only).
#pragma once
#include "w4.h"

namespace lora {

inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

inline int check_w4_shape(int n, int d_in, int d_out, int group, int scale_dtype, int has_zeros) {
  if (n < 1 || d_in < 1 || d_out < 1 || group < 1 || (has_zeros != 0 && has_zeros != 1)) return LORA_ERR_INVALID_ARG;
  if (scale_dtype != LORA_DTYPE_BF16 && scale_dtype != LORA_DTYPE_F32) return LORA_ERR_UNSUPPORTED;
  if (n > LORA_W4_MAX_N || d_in > LORA_W4_MAX_DIM || d_out > LORA_W4_MAX_DIM) return LORA_ERR_UNSUPPORTED;
  if (d_in % 8 != 0 || d_out % 8 != 0 || group % 32 != 0) return LORA_ERR_UNSUPPORTED;
  return LORA_OK;
}

inline int check_w4_store(const lora_w4_store* s) {
  if (s == nullptr) return LORA_ERR_INVALID_ARG;
  const int st = check_w4_shape(s->n, s->d_in, s->d_out, s->group, s->scale_dtype, s->has_zeros);
  if (st != LORA_OK) return st;
  if (s->codes == nullptr || s->params == nullptr) return LORA_ERR_INVALID_ARG;
  return aligned(s->codes, 16) && aligned(s->params, 16) ? LORA_OK : LORA_ERR_UNSUPPORTED;
}

inline int check_w4_ws(const void* ws, size_t ws_bytes, size_t need) {
  if (need == 0) return LORA_OK;
  if (ws == nullptr || ws_bytes < need) return LORA_ERR_INVALID_ARG;
  return aligned(ws, 16) ? LORA_OK : LORA_ERR_UNSUPPORTED;
}

}  // namespace lora
