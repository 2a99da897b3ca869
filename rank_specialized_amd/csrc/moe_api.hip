// C ABI of the mixture-of-experts layer (include/lora.h): argument checks, then
// launches on the caller's stream.
#include <hip/hip_runtime.h>

#include "host_util.h"
#include "moe_kernels.h"
#include "validate.h"
#include "w4_check.h"

using namespace lora;

namespace {

int check_moe_stores(const lora_w4_store* g, const lora_w4_store* u, const lora_w4_store* d) {
  int st;
  if ((st = check_w4_store(g)) != LORA_OK || (st = check_w4_store(u)) != LORA_OK || (st = check_w4_store(d)) != LORA_OK)
    return st;
  if (u->n != g->n || u->d_in != g->d_in || u->d_out != g->d_out || u->group != g->group ||
      u->scale_dtype != g->scale_dtype || u->has_zeros != g->has_zeros || d->n != g->n || d->d_in != g->d_out)
    return LORA_ERR_INVALID_ARG;
  return LORA_OK;
}

int check_moe_sizes(int dtype, int T, int k) {
  if (T < 0 || k < 1) return LORA_ERR_INVALID_ARG;
  if (dtype != LORA_DTYPE_BF16 && dtype != LORA_DTYPE_F32) return LORA_ERR_UNSUPPORTED;
  return T > LORA_W4_MOE_MAX_TOKENS || k > LORA_W4_MOE_MAX_K ? LORA_ERR_UNSUPPORTED : LORA_OK;
}

}  // namespace

extern "C" {

size_t lora_w4_moe_workspace_bytes(const lora_w4_store* gate_host, const lora_w4_store* up_host,
                                   const lora_w4_store* down_host, int dtype, int T, int k) {
  if (check_moe_stores(gate_host, up_host, down_host) != LORA_OK || check_moe_sizes(dtype, T, k) != LORA_OK) return 0;
  return moe_plan_call(gate_host->n, gate_host->d_out, down_host->d_out, dtype, T, k).ws_bytes;
}

int lora_w4_moe(const lora_w4_store* gate_host, const lora_w4_store* up_host, const lora_w4_store* down_host, int dtype,
                int act, const void* x, int64_t ldx, void* y, int64_t ldy, int T, int k, const int32_t* ids,
                const float* weights, void* ws, size_t ws_bytes, void* stream) {
  int st = check_moe_stores(gate_host, up_host, down_host);
  if (st != LORA_OK) return st;
  if ((st = check_moe_sizes(dtype, T, k)) != LORA_OK) return st;
  if (act != LORA_MOE_SILU && act != LORA_MOE_GELU_TANH) return LORA_ERR_INVALID_ARG;
  if (T > 0 && (ids == nullptr || weights == nullptr)) return LORA_ERR_INVALID_ARG;
  if ((st = check_rows(x, ldx, gate_host->d_in, dtype, T)) != LORA_OK) return st;
  if ((st = check_rows(y, ldy, down_host->d_out, dtype, T)) != LORA_OK) return st;
  if (((uintptr_t)ids & 3u) || ((uintptr_t)weights & 3u)) return LORA_ERR_UNSUPPORTED;
  MoeCall c{};
  c.gate = *gate_host;
  c.up = *up_host;
  c.down = *down_host;
  c.dtype = dtype;
  c.act = act;
  c.x = x;
  c.ldx = ldx;
  c.y = y;
  c.ldy = ldy;
  c.T = T;
  c.k = k;
  c.ids = ids;
  c.weights = weights;
  c.plan = moe_plan_call(c.gate.n, c.gate.d_out, c.down.d_out, dtype, T, k);
  if ((st = check_w4_ws(ws, ws_bytes, c.plan.ws_bytes)) != LORA_OK) return st;
  if (T == 0) return LORA_OK;
  c.ws = reinterpret_cast<char*>(ws);
  const hipStream_t hs = reinterpret_cast<hipStream_t>(stream);
  const hipError_t e = dtype == LORA_DTYPE_BF16 ? launch_moe_bf16(c, hs) : launch_moe_f32(c, hs);
  return e == hipSuccess ? LORA_OK : hip_fail(e);
}

}  // extern "C"
