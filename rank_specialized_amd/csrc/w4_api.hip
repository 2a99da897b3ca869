// C ABI of the 4-bit base layers and the router (include/lora.h): argument
// checks, then launches on the caller's stream.
#include <hip/hip_runtime.h>

#include <cstring>

#include "host_util.h"
#include "validate.h"
#include "w4_kernels.h"

using namespace lora;

namespace {

bool aligned(const void* p, size_t a) { return ((uintptr_t)p & (a - 1)) == 0; }

int check_w4_shape(int n, int d_in, int d_out, int group, int scale_dtype, int has_zeros) {
  if (n < 1 || d_in < 1 || d_out < 1 || group < 1 || (has_zeros != 0 && has_zeros != 1)) return LORA_ERR_INVALID_ARG;
  if (scale_dtype != LORA_DTYPE_BF16 && scale_dtype != LORA_DTYPE_F32) return LORA_ERR_UNSUPPORTED;
  if (n > LORA_W4_MAX_N || d_in > LORA_W4_MAX_DIM || d_out > LORA_W4_MAX_DIM) return LORA_ERR_UNSUPPORTED;
  if (d_in % 8 != 0 || d_out % 8 != 0 || group % 32 != 0) return LORA_ERR_UNSUPPORTED;
  return LORA_OK;
}

int check_w4_store(const lora_w4_store* s) {
  if (s == nullptr) return LORA_ERR_INVALID_ARG;
  const int st = check_w4_shape(s->n, s->d_in, s->d_out, s->group, s->scale_dtype, s->has_zeros);
  if (st != LORA_OK) return st;
  if (s->codes == nullptr || s->params == nullptr) return LORA_ERR_INVALID_ARG;
  return aligned(s->codes, 16) && aligned(s->params, 16) ? LORA_OK : LORA_ERR_UNSUPPORTED;
}

int check_w4_call(const W4Call& c, int x_rows, int y_rows, int64_t rows) {
  if (c.dtype != LORA_DTYPE_BF16 && c.dtype != LORA_DTYPE_F32) return LORA_ERR_UNSUPPORTED;
  int st;
  if ((st = check_rows(c.x, c.ldx, c.s.d_in, c.dtype, x_rows)) != LORA_OK) return st;
  if ((st = check_rows(c.y, c.ldy, c.s.d_out, c.dtype, y_rows)) != LORA_OK) return st;
  return rows > LORA_W4_MAX_ROWS ? LORA_ERR_UNSUPPORTED : LORA_OK;
}

int check_w4_ws(const void* ws, size_t ws_bytes, size_t need) {
  if (need == 0) return LORA_OK;
  if (ws == nullptr || ws_bytes < need) return LORA_ERR_INVALID_ARG;
  return aligned(ws, 16) ? LORA_OK : LORA_ERR_UNSUPPORTED;
}

}  // namespace

extern "C" {

int lora_w4_bytes(int n, int d_in, int d_out, int group, int scale_dtype, int has_zeros, size_t* code_bytes_host,
                  size_t* param_bytes_host) {
  if (!code_bytes_host || !param_bytes_host) return LORA_ERR_INVALID_ARG;
  const int st = check_w4_shape(n, d_in, d_out, group, scale_dtype, has_zeros);
  if (st != LORA_OK) return st;
  *code_bytes_host = (size_t)w4_code_bytes(n, d_in, d_out);
  *param_bytes_host = (size_t)w4_params_bytes(n, d_in, d_out, w4_param_kind(scale_dtype, has_zeros), w4_sub(group));
  return LORA_OK;
}

int lora_w4_pack(lora_w4_store* out_host, int n, int d_in, int d_out, int group, const uint8_t* q, const void* scales,
                 int scale_dtype, const uint8_t* zeros, void* codes, void* params, void* stream) {
  if (!out_host) return LORA_ERR_INVALID_ARG;
  const int st = check_w4_shape(n, d_in, d_out, group, scale_dtype, zeros != nullptr);
  if (st != LORA_OK) return st;
  if (!q || !scales || !codes || !params) return LORA_ERR_INVALID_ARG;
  if (!aligned(q, 4) || !aligned(scales, scale_dtype == LORA_DTYPE_F32 ? 4 : 2) || !aligned(codes, 16) ||
      !aligned(params, 16))
    return LORA_ERR_UNSUPPORTED;
  lora_w4_store s;
  std::memset(&s, 0, sizeof(s));
  s.n = n;
  s.d_in = d_in;
  s.d_out = d_out;
  s.group = group;
  s.scale_dtype = scale_dtype;
  s.has_zeros = zeros != nullptr;
  s.codes = codes;
  s.params = params;
  const hipError_t e = launch_w4_pack(s, q, scales, zeros, codes, params, reinterpret_cast<hipStream_t>(stream));
  if (e != hipSuccess) return hip_fail(e);
  *out_host = s;
  return LORA_OK;
}

size_t lora_w4_workspace_bytes(const lora_w4_store* store_host, int dtype, int T, int k, int weighted) {
  if (check_w4_store(store_host) != LORA_OK || T < 0 || k < 0) return 0;
  if (dtype != LORA_DTYPE_BF16 && dtype != LORA_DTYPE_F32) return 0;
  if ((int64_t)T * (k > 0 ? k : 1) > LORA_W4_MAX_ROWS) return 0;
  return w4_plan_call(*store_host, dtype, T, k, weighted != 0).ws_bytes;
}

int lora_w4_apply(const lora_w4_store* store_host, int dtype, const void* x, int64_t ldx, void* y, int64_t ldy, int T,
                  void* ws, size_t ws_bytes, void* stream) {
  int st = check_w4_store(store_host);
  if (st != LORA_OK) return st;
  if (T < 0 || store_host->n != 1) return LORA_ERR_INVALID_ARG;
  W4Call c{};
  c.s = *store_host;
  c.dtype = dtype;
  c.x = x;
  c.ldx = ldx;
  c.x_div = 1;
  c.y = y;
  c.ldy = ldy;
  c.R = T;
  c.k = 1;
  if ((st = check_w4_call(c, T, T, T)) != LORA_OK) return st;
  c.plan = w4_plan_call(c.s, dtype, T, 0, false);
  if ((st = check_w4_ws(ws, ws_bytes, c.plan.ws_bytes)) != LORA_OK) return st;
  if (T == 0) return LORA_OK;
  c.ws = reinterpret_cast<char*>(ws);
  const hipError_t e = launch_w4(c, reinterpret_cast<hipStream_t>(stream));
  return e == hipSuccess ? LORA_OK : hip_fail(e);
}

int lora_w4_apply_experts(const lora_w4_store* store_host, int dtype, const void* x, int64_t ldx, int x_per_choice,
                          void* y, int64_t ldy, int T, int k, const int32_t* ids, const float* weights, void* ws,
                          size_t ws_bytes, void* stream) {
  int st = check_w4_store(store_host);
  if (st != LORA_OK) return st;
  if (T < 0 || k < 1 || (x_per_choice != 0 && x_per_choice != 1)) return LORA_ERR_INVALID_ARG;
  if (T > 0 && ids == nullptr) return LORA_ERR_INVALID_ARG;
  const int64_t rows = (int64_t)T * k;
  if (rows > LORA_W4_MAX_ROWS) return LORA_ERR_UNSUPPORTED;
  W4Call c{};
  c.s = *store_host;
  c.dtype = dtype;
  c.x = x;
  c.ldx = ldx;
  c.x_div = x_per_choice ? 1 : k;
  c.y = y;
  c.ldy = ldy;
  c.R = (int)rows;
  c.ids = ids;
  c.weights = weights;
  c.k = k;
  if ((st = check_w4_call(c, x_per_choice ? (int)rows : T, weights ? T : (int)rows, rows)) != LORA_OK) return st;
  if ((ids && !aligned(ids, 4)) || (weights && !aligned(weights, 4))) return LORA_ERR_UNSUPPORTED;
  c.plan = w4_plan_call(c.s, dtype, T, k, weights != nullptr);
  if ((st = check_w4_ws(ws, ws_bytes, c.plan.ws_bytes)) != LORA_OK) return st;
  if (T == 0) return LORA_OK;
  c.ws = reinterpret_cast<char*>(ws);
  const hipError_t e = launch_w4(c, reinterpret_cast<hipStream_t>(stream));
  return e == hipSuccess ? LORA_OK : hip_fail(e);
}

int lora_route(const void* logits, int64_t ldl, int dtype, int T, int E, int k, int score, const float* bias,
               int groups, int top_groups, int renormalize, float scale, int32_t* ids, float* weights, void* stream) {
  if (T < 0 || E < 1 || k < 1 || groups < 1 || E % groups != 0 || top_groups < 1 || top_groups > groups ||
      k > E / groups * top_groups || ldl < E || (score != LORA_ROUTE_SOFTMAX && score != LORA_ROUTE_SIGMOID))
    return LORA_ERR_INVALID_ARG;
  if (T > 0 && (!logits || !ids || !weights)) return LORA_ERR_INVALID_ARG;
  if (dtype != LORA_DTYPE_BF16 && dtype != LORA_DTYPE_F32) return LORA_ERR_UNSUPPORTED;
  if (E > LORA_ROUTE_MAX_EXPERTS || k > LORA_ROUTE_MAX_K || groups > LORA_ROUTE_MAX_GROUPS ||
      T > LORA_ROUTE_MAX_TOKENS)
    return LORA_ERR_UNSUPPORTED;
  if (!aligned(logits, (size_t)elem_bytes(dtype)) || !aligned(bias, 4) || !aligned(ids, 4) || !aligned(weights, 4))
    return LORA_ERR_UNSUPPORTED;
  if (T == 0) return LORA_OK;
  RouteArgs a{};
  a.logits = logits;
  a.ldl = ldl;
  a.T = T;
  a.E = E;
  a.k = k;
  a.score = score;
  a.bias = bias;
  a.groups = groups;
  a.top_groups = top_groups;
  a.renormalize = renormalize != 0;
  a.scale = scale;
  a.ids = ids;
  a.weights = weights;
  const hipError_t e = launch_route(a, dtype, reinterpret_cast<hipStream_t>(stream));
  return e == hipSuccess ? LORA_OK : hip_fail(e);
}

}  // extern "C"
