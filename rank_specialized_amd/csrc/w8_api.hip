// C ABI of the 8-bit base layers (include/lora.h): argument checks, then
// launches on the caller's stream.
#include <hip/hip_runtime.h>

#include <cstring>

#include "host_util.h"
#include "validate.h"
#include "w8_kernels.h"

using namespace lora;

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

int check_w8_shape(int d_in, int d_out) {
  if (d_in < 1 || d_out < 1) return LORA_ERR_INVALID_ARG;
  if (d_in > LORA_W8_MAX_IN || d_out > LORA_W8_MAX_OUT || d_in % 8 != 0 || d_out % 8 != 0) return LORA_ERR_UNSUPPORTED;
  return LORA_OK;
}

int check_w8_store(const lora_w8_store* s) {
  if (s == nullptr) return LORA_ERR_INVALID_ARG;
  const int st = check_w8_shape(s->d_in, s->d_out);
  if (st != LORA_OK) return st;
  if (s->codes == nullptr || s->scales == nullptr) return LORA_ERR_INVALID_ARG;
  return aligned(s->codes, 16) && aligned(s->scales, 16) ? LORA_OK : LORA_ERR_UNSUPPORTED;
}

int check_w8_dtype(int dtype) {
  return dtype == LORA_DTYPE_BF16 || dtype == LORA_DTYPE_F32 ? LORA_OK : LORA_ERR_UNSUPPORTED;
}

// Rows of codes and their scales.
int check_w8_codes(const int8_t* q, int64_t ldq, int d_in, const float* scales, int T) {
  if (T > 0 && (q == nullptr || scales == nullptr)) return LORA_ERR_INVALID_ARG;
  if (ldq < d_in) return LORA_ERR_INVALID_ARG;
  if (ldq % 16 != 0 || ldq > LORA_W8_MAX_LDQ || !aligned(q, 16) || !aligned(scales, 4)) return LORA_ERR_UNSUPPORTED;
  return LORA_OK;
}

int run_w8(W8Call& c, hipStream_t stream) {
  const hipError_t e = c.plan.tile > 0 ? launch_w8_gemm(c, stream) : launch_w8_rows(c, stream);
  return e == hipSuccess ? LORA_OK : hip_fail(e);
}

}  // namespace

extern "C" {

int lora_w8_bytes(int d_in, int d_out, size_t* code_bytes_host, size_t* scale_bytes_host) {
  if (!code_bytes_host || !scale_bytes_host) return LORA_ERR_INVALID_ARG;
  const int st = check_w8_shape(d_in, d_out);
  if (st != LORA_OK) return st;
  *code_bytes_host = (size_t)w8_code_bytes(d_in, d_out);
  *scale_bytes_host = (size_t)w8_scale_bytes(d_out);
  return LORA_OK;
}

int lora_w8_pack(lora_w8_store* out_host, int d_in, int d_out, const int8_t* q, const void* scales, int scale_dtype,
                 void* codes, float* out_scales, void* stream) {
  if (!out_host) return LORA_ERR_INVALID_ARG;
  int st = check_w8_shape(d_in, d_out);
  if (st != LORA_OK) return st;
  if (!q || !scales || !codes || !out_scales) return LORA_ERR_INVALID_ARG;
  if ((st = check_w8_dtype(scale_dtype)) != LORA_OK) return st;
  if (!aligned(q, 8) || !aligned(scales, (size_t)elem_bytes(scale_dtype)) || !aligned(codes, 16) || !aligned(out_scales, 16))
    return LORA_ERR_UNSUPPORTED;
  const hipError_t e =
      launch_w8_pack(d_in, d_out, q, scales, scale_dtype, codes, out_scales, reinterpret_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e);
  lora_w8_store s;
  std::memset(&s, 0, sizeof(s));
  s.d_in = d_in;
  s.d_out = d_out;
  s.codes = codes;
  s.scales = out_scales;
  *out_host = s;
  return LORA_OK;
}

int lora_w8_quantize(int dtype, const void* x, int64_t ldx, int T, int d_in, int8_t* q, int64_t ldq, float* scales,
                     void* stream) {
  if (T < 0) return LORA_ERR_INVALID_ARG;
  int st = check_w8_shape(d_in, 8);
  if (st != LORA_OK) return st;
  if ((st = check_w8_dtype(dtype)) != LORA_OK) return st;
  if ((st = check_rows(x, ldx, d_in, dtype, T)) != LORA_OK) return st;
  if ((st = check_w8_codes(q, ldq, d_in, scales, T)) != LORA_OK) return st;
  if (T > LORA_W8_MAX_ROWS) return LORA_ERR_UNSUPPORTED;
  if (T == 0) return LORA_OK;
  const hipError_t e = launch_w8_quantize(dtype, x, ldx, T, d_in, q, ldq, scales, reinterpret_cast<hipStream_t>(stream));
  return e == hipSuccess ? LORA_OK : hip_fail(e);
}

size_t lora_w8_workspace_bytes(const lora_w8_store* store_host, int T, int quantized) {
  if (check_w8_store(store_host) != LORA_OK || T < 0 || T > LORA_W8_MAX_ROWS) return 0;
  return w8_plan_call(store_host->d_in, store_host->d_out, T, quantized != 0).ws_bytes;
}

int lora_w8_apply(const lora_w8_store* store_host, int dtype, const void* x, int64_t ldx, void* y, int64_t ldy, int T,
                  void* ws, size_t ws_bytes, void* stream) {
  int st = check_w8_store(store_host);
  if (st != LORA_OK) return st;
  if (T < 0) return LORA_ERR_INVALID_ARG;
  if ((st = check_w8_dtype(dtype)) != LORA_OK) return st;
  const int d_in = store_host->d_in;
  if ((st = check_rows(x, ldx, d_in, dtype, T)) != LORA_OK) return st;
  if ((st = check_rows(y, ldy, store_host->d_out, dtype, T)) != LORA_OK) return st;
  if (T > LORA_W8_MAX_ROWS) return LORA_ERR_UNSUPPORTED;
  W8Call c{};
  c.w = *store_host;
  c.dtype = dtype;
  c.x = x;
  c.ldx = ldx;
  c.y = y;
  c.ldy = ldy;
  c.T = T;
  c.plan = w8_plan_call(d_in, c.w.d_out, T, false);
  if (c.plan.ws_bytes > 0) {
    if (ws == nullptr || ws_bytes < c.plan.ws_bytes) return LORA_ERR_INVALID_ARG;
    if (!aligned(ws, 16)) return LORA_ERR_UNSUPPORTED;
  }
  if (T == 0) return LORA_OK;
  const hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
  if (!c.plan.fused) {
    int8_t* q = reinterpret_cast<int8_t*>(ws) + c.plan.q;
    float* s = reinterpret_cast<float*>(reinterpret_cast<char*>(ws) + c.plan.s);
    c.q = q;
    c.s = s;
    c.ldq = w8_row_bytes(d_in);
    const hipError_t e = launch_w8_quantize(dtype, x, ldx, T, d_in, q, c.ldq, s, hs);
    if (e != hipSuccess) return hip_fail(e);
  }
  return run_w8(c, hs);
}

int lora_w8_apply_quantized(const lora_w8_store* store_host, const int8_t* q, int64_t ldq, const float* scales, int dtype,
                            void* y, int64_t ldy, int T, void* ws, size_t ws_bytes, void* stream) {
  int st = check_w8_store(store_host);
  if (st != LORA_OK) return st;
  if (T < 0) return LORA_ERR_INVALID_ARG;
  if ((st = check_w8_dtype(dtype)) != LORA_OK) return st;
  if ((st = check_w8_codes(q, ldq, store_host->d_in, scales, T)) != LORA_OK) return st;
  if ((st = check_rows(y, ldy, store_host->d_out, dtype, T)) != LORA_OK) return st;
  if (T > LORA_W8_MAX_ROWS) return LORA_ERR_UNSUPPORTED;
  W8Call c{};
  c.w = *store_host;
  c.dtype = dtype;
  c.q = q;
  c.ldq = ldq;
  c.s = scales;
  c.y = y;
  c.ldy = ldy;
  c.T = T;
  c.plan = w8_plan_call(c.w.d_in, c.w.d_out, T, true);
  if (c.plan.ws_bytes > 0) {
    if (ws == nullptr || ws_bytes < c.plan.ws_bytes) return LORA_ERR_INVALID_ARG;
    if (!aligned(ws, 16)) return LORA_ERR_UNSUPPORTED;
  }
  if (T == 0) return LORA_OK;
  return run_w8(c, reinterpret_cast<hipStream_t>(stream));
}

}  // extern "C"
