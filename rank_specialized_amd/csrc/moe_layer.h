// A mixture-of-experts layer for a few tokens, in two kernels:
//
//   h[t, e] = act(G_e x[t]) * (U_e x[t])          e = ids[t, j]
//   y[t]    = sum_j w[t, j] D_e h[t, e]
//
// with 4-bit matrices (w4.h).  What bounds both is the stream of codes.  In
// both, codes enter the bf16 matrix cores as in the few-rows products
// (w4_rows.h): 32 + q with (32 + z) times the rows' sum taken off, or, for
// float32 rows, q - z itself.
//
// Kernel 1: a workgroup owns 16 WB features of one expert, gate and up, for
// the tokens that chose it (found by every wave alone, a token per lane); WK
// waves share the inputs of 16 features, and their sums meet in LDS.  h leaves
// as bf16 parts, the operands of the second kernel, and the expert's tokens as
// an entry of a table.
// Kernel 2: a workgroup owns 16 WB outputs of all tokens and walks the table;
// WE waves share the tiles of 16 outputs.  Each wave adds its weighted sums to
// rows of its own in LDS, which are added in wave order at the end: sums have
// one order, whatever the schedule.
#pragma once
#include "host_util.h"
#include "moe_kernels.h"
#include "w4_ops.h"

namespace lora {
namespace {

constexpr int kMoePad = 17;  // LDS row stride of a 16 x 16 block of sums
constexpr int kMoeRows = 16;

// The products of one tile of 128 inputs: rows at `x` (this lane's row and
// piece) in PARTS planes, codes and scales of NB blocks of 16 outputs.
template <int PARTS, bool EXACT, int SUB, int NB, typename Par>
__device__ __forceinline__ void moe_tile(const char* x, int plane, const uint4 (&code)[NB], const Par (&par)[NB],
                                         uint32_t mask, uint32_t magic, f32x4_t (&acc)[NB]) {
  constexpr int kSteps = 4 / SUB;
  const uint4 ones = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
#pragma unroll
  for (int s = 0; s < SUB; ++s) {
    uint4 xp[kSteps][PARTS];
    f32x4_t xsum = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int j = 0; j < kSteps; ++j)
#pragma unroll
      for (int q = 0; q < PARTS; ++q) {
        xp[j][q] = ld16(x + q * plane + 64 * (s * kSteps + j));
        if constexpr (!EXACT) xsum = mfma_bf16_16x16x32(xp[j][q], ones, xsum);
      }
#pragma unroll
    for (int a = 0; a < NB; ++a) {
      const uint32_t cw[4] = {code[a].x, code[a].y, code[a].z, code[a].w};
      const float sc = par[a].scale(s), z32 = par[a].zero32(s);
      f32x4_t c;
#pragma unroll
      for (int v = 0; v < 4; ++v) c[v] = EXACT ? 0.f : -z32 * xsum[v];
#pragma unroll
      for (int j = 0; j < kSteps; ++j) {
        const uint4 b = EXACT ? w4_expand_exact(cw[s * kSteps + j], mask, magic, z32) : w4_expand(cw[s * kSteps + j], mask, magic);
#pragma unroll
        for (int q = 0; q < PARTS; ++q) c = mfma_bf16_16x16x32(xp[j][q], b, c);
      }
#pragma unroll
      for (int v = 0; v < 4; ++v) acc[a][v] = fmaf(sc, c[v], acc[a][v]);
    }
  }
}

// ------------------------------------------------------------ gate and up
struct MoeUpArgs {
  const char *gate, *gate_par, *up, *up_par;
  int64_t code_stride, param_stride;  // bytes per matrix
  int n, d, ffn, k_tiles, row_tiles, h_tiles;
  const char* x;
  int64_t ldx_bytes;
  int T, k, act, by_row, lds_bytes;
  const int32_t* ids;
  const float* weights;
  uint16_t* h;
  MoeEntry* table;
};

// act(g) u, each a few float32 roundings from the formula: silu(g) = g / (1 +
// exp(-g)); the tanh form of gelu, g / 2 (1 + tanh(v)) = g / (1 + exp(-2 v)).
__device__ __forceinline__ float moe_act(int act, float g, float u) {
  float v = g;
  if (act == LORA_MOE_GELU_TANH) v = 1.5957691216057308f * (g + 0.044715f * g * g * g);
  return g / (1.f + expf(-v)) * u;
}

// h in bf16 parts.
template <int PARTS>
__device__ __forceinline__ void moe_parts(float v, uint16_t (&o)[PARTS]) {
#pragma unroll
  for (int q = 0; q < PARTS; ++q) {
    // The last of two rounds; the others cut, and leave an exact rest.
    const uint32_t b = PARTS == 2 && q == 1 ? f32_to_bf16(v) : __float_as_uint(v) >> 16;
    o[q] = (uint16_t)b;
    v -= __uint_as_float(b << 16);
  }
}

template <typename E, int KIND, int SUB, int WB, int WK, int U>
__global__ __launch_bounds__(64 * WB * WK) __attribute__((amdgpu_waves_per_eu(2)))
void moe_up_kernel(const MoeUpArgs p) {
  constexpr int kParts = XFrag<E>::kParts, kHParts = kParts == 1 ? 2 : 3, W = WB * WK;
  typedef W4Params<KIND, SUB> Par;
  extern __shared__ __align__(16) char lds[];  // x; then the waves' sums
  __shared__ uint16_t s_row[LORA_W4_MOE_MAX_TOKENS], s_tok[LORA_W4_MOE_MAX_TOKENS];
  const int tid = (int)threadIdx.x, lane = tid & 63, col = lane & 15, h = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6), wb = w / WK, wk = w % WK;

  // ---- the expert's tokens, a token per lane, its weights added up; every
  // wave finds the same
  const int e = p.by_row ? p.ids[blockIdx.y] : (int)blockIdx.y;
  int first = -1;
  float wsum = 0.f;
  if (lane < p.T) {
#pragma unroll 8
    for (int j = 0; j < p.k; ++j) {
      const int r = lane * p.k + j;
      if (p.ids[r] == e) {
        wsum = first < 0 ? p.weights[r] : wsum + p.weights[r];
        first = first < 0 ? r : first;
      }
    }
  }
  const uint64_t hits = (unsigned)e < (unsigned)p.n ? __ballot(first >= 0) : 0ull;
  int cnt = __popcll(hits);
  // By choice: the first row of an expert works for all of its rows.
  if (cnt > 0 && p.by_row && __builtin_amdgcn_readlane(first, __ffsll((unsigned long long)hits) - 1) != (int)blockIdx.y) cnt = 0;
  if (blockIdx.x == 0 && w == 0) {
    MoeEntry& t = p.table[blockIdx.y];
    if (lane == 0) {
      t.e = e;
      t.cnt = cnt;
    }
    if (cnt > 0 && first >= 0) {
      const int at = __popcll(hits & lanemask_lt());
      t.row[at] = (uint16_t)first;
      t.tok[at] = (uint16_t)lane;
      t.w[at] = wsum;
    }
  }
  if (cnt == 0) return;
  if (first >= 0) {  // all waves write the same
    const int at = __popcll(hits & lanemask_lt());
    s_row[at] = (uint16_t)first;
    s_tok[at] = (uint16_t)lane;
  }
  __syncthreads();

  const int fb = (int)blockIdx.x * WB + wb;  // block of 16 features; from row_tiles on: pads of h
  const uint32_t mask = w4_scalar(kCodeMask), magic = w4_vector(kMagicBf16);
  const int64_t tile0 = (int64_t)min(fb, p.row_tiles - 1) * p.k_tiles;
  const int64_t code_at = e * p.code_stride + tile0 * kW4TileBytes + 16 * lane;
  const int64_t par_at = e * p.param_stride + tile0 * kW4Rows * Par::kBytes + col * Par::kBytes;
  const char* code0[2] = {p.gate + code_at, p.up + code_at};
  const char* par0[2] = {p.gate_par + par_at, p.up_par + par_at};

  for (int m0 = 0; m0 < cnt; m0 += kMoeRows) {
    const int m = min(kMoeRows, cnt - m0);
    // All inputs of the rows in LDS, or as many tiles as fit.
    const int chunk = min(p.k_tiles, (p.lds_bytes / m - 16) / (kParts * kW4K * 2));
    const int plane = chunk * kW4K * 2, xrow = kParts * plane + 16;
    const char* xl = lds + min(col, m - 1) * xrow + 16 * h;
    f32x4_t acc[2] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
    for (int c0 = 0; c0 < p.k_tiles; c0 += chunk) {
      const int c1 = min(p.k_tiles, c0 + chunk);
      uint4 code[U][2];
      Par par[U][2];
      auto fetch = [&](int u, int kt) {
#pragma unroll
        for (int a = 0; a < 2; ++a) {
          code[u][a] = ld16(code0[a] + (int64_t)kt * kW4TileBytes);
          par[u][a].load(par0[a] + (int64_t)kt * (kW4Rows * Par::kBytes));
        }
      };
#pragma unroll
      for (int u = 0; u < U; ++u) fetch(u, min(c0 + wk + u * WK, c1 - 1));
      __syncthreads();  // the chunk (or the sums) before has been read
      const int pieces = (c1 - c0) * (kW4K / 8);
      for (int i = tid; i < m * pieces; i += 64 * W) {
        const int row = i / pieces, at = i - row * pieces, kk = c0 * kW4K + 8 * at;
        uint4 parts[kParts];
        if (kk < p.d) {
          XFrag<E> f;
          f.load(p.x + (int64_t)s_tok[m0 + row] * p.ldx_bytes + (int64_t)kk * E::kBytes);
          f.parts(parts);
        } else {
#pragma unroll
          for (int q = 0; q < kParts; ++q) parts[q] = make_uint4(0u, 0u, 0u, 0u);
        }
#pragma unroll
        for (int q = 0; q < kParts; ++q) st16(lds + row * xrow + q * plane + 16 * at, parts[q]);
      }
      __syncthreads();
      for (int i0 = c0 + wk; i0 < c1; i0 += U * WK) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = i0 + u * WK;
          if (i < c1) moe_tile<kParts, (kParts > 1), SUB, 2, Par>(xl + (i - c0) * kW4K * 2, plane, code[u], par[u], mask, magic, acc);
          if (i0 + U * WK < c1) fetch(u, min(i + U * WK, c1 - 1));
        }
      }
    }
    // ---- the waves' sums, in wave order; then h
    __syncthreads();
    float* red = reinterpret_cast<float*>(lds);
#pragma unroll
    for (int a = 0; a < 2; ++a)
#pragma unroll
      for (int v = 0; v < 4; ++v) red[(w * 2 + a) * 16 * kMoePad + (4 * h + v) * kMoePad + col] = acc[a][v];
    __syncthreads();
    for (int i = tid; i < WB * 16 * m; i += 64 * W) {
      const int c = i & 15, b = (i >> 4) % WB, row = (i >> 4) / WB;
      float g = 0.f, u = 0.f;
#pragma unroll
      for (int ww = 0; ww < WK; ++ww) {
        g += red[((b * WK + ww) * 2) * 16 * kMoePad + row * kMoePad + c];
        u += red[((b * WK + ww) * 2 + 1) * 16 * kMoePad + row * kMoePad + c];
      }
      const int f = 16 * ((int)blockIdx.x * WB + b) + c, fp = p.h_tiles * kW4K;
      if (f >= fp) continue;
      uint16_t o[kHParts];
      moe_parts<kHParts>(f < p.ffn ? moe_act(p.act, g, u) : 0.f, o);
#pragma unroll
      for (int q = 0; q < kHParts; ++q) p.h[((int64_t)s_row[m0 + row] * kHParts + q) * fp + f] = o[q];
    }
  }
}

// ------------------------------------------------------------ down
struct MoeDownArgs {
  const char *codes, *params;
  int64_t code_stride, param_stride;
  int d_out, k_tiles, row_tiles;
  int T, entries, cap;  // rows of h held in LDS at a time
  const uint16_t* h;
  const MoeEntry* table;
  char* y;
  int64_t ldy_bytes;
};

constexpr int kMoeItems = 16;  // chunks of an expert's rows that are taken together

template <typename E, int KIND, int SUB, int WB, int WE, int U>
__global__ __launch_bounds__(64 * WB * WE) __attribute__((amdgpu_waves_per_eu(2)))
void moe_down_kernel(const MoeDownArgs p) {
  constexpr int kParts = E::kBytes == 2 ? 2 : 3, W = WB * WE;
  typedef W4Params<KIND, SUB> Par;
  // The waves' sums [W][T][16], then rows of h.
  extern __shared__ __align__(16) char lds[];
  struct Item {
    int e, entry, first, m, at;  // expert; its rows first .. + m - 1 of the entry; the first one's place in LDS
  };
  __shared__ Item items[kMoeItems];
  const int tid = (int)threadIdx.x, lane = tid & 63, col = lane & 15, h = lane >> 4;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6), wb = w / WE, we = w % WE;
  float* sums = reinterpret_cast<float*>(lds);
  char* rows = lds + W * p.T * 64;
  const int plane = p.k_tiles * kW4K * 2, hrow = kParts * plane + 16;
  for (int i = tid; i < W * p.T * 16; i += 64 * W) sums[i] = 0.f;
  float* mine = sums + w * p.T * 16;
  const int ob = (int)blockIdx.x * WB + wb;
  const uint32_t mask = w4_scalar(kCodeMask), magic = w4_vector(kMagicBf16);
  const int64_t tile0 = (int64_t)min(ob, p.row_tiles - 1) * p.k_tiles;
  const char* code0 = p.codes + tile0 * kW4TileBytes + 16 * lane;
  const char* par0 = p.params + tile0 * kW4Rows * Par::kBytes + col * Par::kBytes;

  int at_entry = 0, at_row = 0;  // uniform: the walk through the table
  while (at_entry < p.entries) {
    __syncthreads();  // the rows and items before have been read
    int n_items = 0, used = 0;
    while (at_entry < p.entries && n_items < kMoeItems && used < p.cap) {
      const int cnt = p.table[at_entry].cnt, left = cnt - at_row;
      if (left <= 0) {
        ++at_entry;
        at_row = 0;
        continue;
      }
      const int m = min(min(left, kMoeRows), p.cap - used);
      if (tid == 0) items[n_items] = Item{p.table[at_entry].e, at_entry, at_row, m, used};
      ++n_items;
      used += m;
      at_row += m;
    }
    __syncthreads();
    const int pieces = hrow / 16 - 1;
    for (int i = tid; i < used * pieces; i += 64 * W) {
      const int row = i / pieces, at = i - row * pieces;
      int it = 0;
      while (it + 1 < n_items && items[it + 1].at <= row) ++it;
      const int r = p.table[items[it].entry].row[items[it].first + row - items[it].at];
      st16(rows + row * hrow + 16 * at, ld16(reinterpret_cast<const char*>(p.h) + (int64_t)r * kParts * plane + 16 * at));
    }
    __syncthreads();
    f32x4_t acc[1] = {{0.f, 0.f, 0.f, 0.f}};
    int cur = -1;
    auto flush = [&]() {
      const Item t = items[cur];
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (4 * h + v < t.m) {
          const int i = t.first + 4 * h + v;
          float* s = mine + p.table[t.entry].tok[i] * 16 + col;
          *s = fmaf(p.table[t.entry].w[i], acc[0][v], *s);
        }
      acc[0] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    };
    const int tiles = n_items * p.k_tiles;
    for (int i = we; i < tiles; i += WE) {
      const int it = i / p.k_tiles, kt = i - it * p.k_tiles;
      if (it != cur) {
        if (cur >= 0) flush();
        cur = it;
      }
      const Item t = items[it];
      uint4 code[1] = {ld16(code0 + t.e * p.code_stride + (int64_t)kt * kW4TileBytes)};
      Par par[1];
      par[0].load(par0 + t.e * p.param_stride + (int64_t)kt * (kW4Rows * Par::kBytes));
      const char* x = rows + (t.at + min(col, t.m - 1)) * hrow + 16 * h + kt * kW4K * 2;
      moe_tile<kParts, (kParts > 2), SUB, 1, Par>(x, plane, code, par, mask, magic, acc);
    }
    if (cur >= 0) flush();
  }
  __syncthreads();
  for (int i = tid; i < WB * 16 * p.T; i += 64 * W) {
    const int c = i & 15, b = (i >> 4) % WB, t = (i >> 4) / WB;
    const int o = 16 * ((int)blockIdx.x * WB + b) + c;
    if (o >= p.d_out) continue;
    float s = 0.f;
#pragma unroll
    for (int ww = 0; ww < WE; ++ww) s += sums[((b * WE + ww) * p.T + t) * 16 + c];
    char* dst = p.y + (int64_t)t * p.ldy_bytes;
    if constexpr (E::kBytes == 2) reinterpret_cast<uint16_t*>(dst)[o] = (uint16_t)f32_to_bf16(s);
    else reinterpret_cast<float*>(dst)[o] = s;
  }
}

constexpr int kMoeLds = 64 * 1024;  // of rows

template <typename E, int KIND, int SUB>
hipError_t launch_up(const MoeCall& c, hipStream_t stream) {
  constexpr int WB = 2, WK = 4, U = 2;
  constexpr int kParts = XFrag<E>::kParts;
  MoeUpArgs a{};
  a.gate = reinterpret_cast<const char*>(c.gate.codes);
  a.gate_par = reinterpret_cast<const char*>(c.gate.params);
  a.up = reinterpret_cast<const char*>(c.up.codes);
  a.up_par = reinterpret_cast<const char*>(c.up.params);
  a.n = c.gate.n;
  a.d = c.gate.d_in;
  a.ffn = c.gate.d_out;
  a.code_stride = w4_code_bytes(1, a.d, a.ffn);
  a.param_stride = w4_params_bytes(1, a.d, a.ffn, KIND, SUB);
  a.k_tiles = w4_k_tiles(a.d);
  a.row_tiles = w4_row_tiles(a.ffn);
  a.h_tiles = c.plan.h_tiles;
  a.x = reinterpret_cast<const char*>(c.x);
  a.ldx_bytes = c.ldx * E::kBytes;
  a.T = c.T;
  a.k = c.k;
  a.act = c.act;
  a.by_row = c.plan.by_row;
  a.ids = c.ids;
  a.weights = c.weights;
  a.h = reinterpret_cast<uint16_t*>(c.ws + c.plan.h);
  a.table = reinterpret_cast<MoeEntry*>(c.ws + c.plan.table);
  const int64_t row = (int64_t)kParts * a.k_tiles * kW4K * 2 + 16;
  const int64_t all = (c.T < kMoeRows ? c.T : kMoeRows) * row;
  const int64_t sums = (int64_t)WB * WK * 2 * 16 * kMoePad * 4;
  a.lds_bytes = (int)(all < kMoeLds ? (all > sums ? all : sums) : kMoeLds);
  static DynLdsLimit lim;
  const hipError_t e = ensure_dynamic_lds(lim, reinterpret_cast<const void*>(moe_up_kernel<E, KIND, SUB, WB, WK, U>), (size_t)a.lds_bytes);
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)((a.h_tiles * 8 + WB - 1) / WB), (unsigned)c.plan.entries);
  hipLaunchKernelGGL((moe_up_kernel<E, KIND, SUB, WB, WK, U>), grid, dim3(64 * WB * WK), (size_t)a.lds_bytes, stream, a);
  return hipGetLastError();
}

template <typename E, int KIND, int SUB>
hipError_t launch_down(const MoeCall& c, hipStream_t stream) {
  constexpr int WB = 1, WE = 8, U = 2;
  constexpr int kParts = E::kBytes == 2 ? 2 : 3;
  MoeDownArgs a{};
  a.codes = reinterpret_cast<const char*>(c.down.codes);
  a.params = reinterpret_cast<const char*>(c.down.params);
  a.d_out = c.down.d_out;
  a.code_stride = w4_code_bytes(1, c.down.d_in, a.d_out);
  a.param_stride = w4_params_bytes(1, c.down.d_in, a.d_out, KIND, SUB);
  a.k_tiles = c.plan.h_tiles;
  a.row_tiles = w4_row_tiles(a.d_out);
  a.T = c.T;
  a.entries = c.plan.entries;
  a.h = reinterpret_cast<const uint16_t*>(c.ws + c.plan.h);
  a.table = reinterpret_cast<const MoeEntry*>(c.ws + c.plan.table);
  a.y = reinterpret_cast<char*>(c.y);
  a.ldy_bytes = c.ldy * E::kBytes;
  const int64_t row = (int64_t)kParts * a.k_tiles * kW4K * 2 + 16;
  const int64_t sums = (int64_t)WB * WE * c.T * 64;
  int64_t cap = kMoeLds / row;
  cap = cap < 1 ? 1 : (cap > (int64_t)c.T * c.k ? (int64_t)c.T * c.k : cap);
  a.cap = (int)cap;
  const int64_t lds = sums + cap * row;
  if (lds > 150 * 1024) return hipErrorInvalidValue;
  static DynLdsLimit lim;
  const hipError_t e = ensure_dynamic_lds(lim, reinterpret_cast<const void*>(moe_down_kernel<E, KIND, SUB, WB, WE, U>), (size_t)lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((moe_down_kernel<E, KIND, SUB, WB, WE, U>), dim3((unsigned)((a.row_tiles + WB - 1) / WB)), dim3(64 * WB * WE),
                     (size_t)lds, stream, a);
  return hipGetLastError();
}

template <typename E, bool UP>
hipError_t launch_kind(const MoeCall& c, hipStream_t st) {
  const lora_w4_store& s = UP ? c.gate : c.down;
#define LORA_MOE_CASE(K, S) \
  case K * 8 + S: if constexpr (UP) return launch_up<E, K, S>(c, st); else return launch_down<E, K, S>(c, st)
  switch (w4_param_kind(s.scale_dtype, s.has_zeros) * 8 + w4_sub(s.group)) {
    LORA_MOE_CASE(kW4Bf16, 1);
    LORA_MOE_CASE(kW4Bf16, 2);
    LORA_MOE_CASE(kW4Bf16, 4);
    LORA_MOE_CASE(kW4Bf16Zero, 1);
    LORA_MOE_CASE(kW4Bf16Zero, 2);
    LORA_MOE_CASE(kW4Bf16Zero, 4);
    LORA_MOE_CASE(kW4F32, 1);
    LORA_MOE_CASE(kW4F32, 2);
    LORA_MOE_CASE(kW4F32, 4);
  }
#undef LORA_MOE_CASE
  return hipErrorInvalidValue;
}

template <typename E>
hipError_t launch_moe(const MoeCall& c, hipStream_t stream) {
  const hipError_t e = launch_kind<E, true>(c, stream);
  return e != hipSuccess ? e : launch_kind<E, false>(c, stream);
}

}  // namespace
}  // namespace lora
