// 4-bit base products for few rows (the decode step):
//
//   y[r, o] = sum_g s[o, g] sum_{k in g} (q[o, k] - z[o, g]) x[r, k]
//
// with one matrix, or with the matrix that ids[r] names.
//
// A workgroup owns 16 RT outputs; its waves take the 128-input tiles of the
// codes in turn and their float32 sums meet in LDS, added in wave order (the
// same order at every call).  The tiles of an output row are consecutive in
// memory, so the workgroup streams them in order, 1 KiB per wave and load.
// What bounds it is that stream.
//
// Products run on the matrix cores with x on the row side and the codes on
// the column side, 16 rows x 16 outputs.  A code enters as the bf16 number
// 16 + q, which costs one "and-or" per two codes; the excess is taken out
// with the sum of x over the group,
//
//   sum (q - z) x = sum (16 + q) x - (16 + z) sum x,
//
// where sum x comes from one more product against ones, in the same lane
// layout, and its multiple is the accumulator that the group's products
// start from.  All products are exact in float32 and only the sums round;
// 16 is the smallest base that bf16 can hold with a step of one code, which
// keeps the cancelled part small (about three times the result).  Float32
// rows, which take three products per step anyway, are multiplied with q - z
// itself: more work per code, no cancellation.
#include "host_util.h"
#include "w4_kernels.h"
#include "w4_ops.h"

namespace lora {
namespace {

template <typename E, int KIND, int SUB, int RT, int NT>
struct Slot {
  uint4 code[RT];
  W4Params<KIND, SUB> par[RT];
  XFrag<E> x[NT][4];
};

template <typename E, int KIND, int SUB, int RT, int NT, int U, int W>
__global__ __launch_bounds__(64 * W) __attribute__((amdgpu_waves_per_eu(2)))
void w4_rows_kernel(const W4RowsArgs p) {
  constexpr int kTok = 16 * NT;
  constexpr int kStepsPerSub = 4 / SUB;
  constexpr bool kExact = XFrag<E>::kParts > 1;
  constexpr int kPad = 17;  // LDS row stride of a 16 x 16 block
  __shared__ float red[W][RT][NT][16 * kPad];
  __shared__ uint16_t list[kListMax];
  __shared__ int s_cnt[W + 1];
  const int tid = (int)threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);  // uniform: addresses of codes stay scalar
  const int col = lane & 15, h = lane >> 4;
  const int rt0 = (int)blockIdx.x * RT;

  const bool listed = p.ids != nullptr;
  const int self = listed && p.by_row ? (int)blockIdx.y : -1;
  int e = 0;
  bool none = false;
  if (listed) {
    e = p.by_row ? p.ids[self] : (int)blockIdx.y;
    none = (unsigned)e >= (unsigned)p.n;  // rows without a matrix (by matrix: one workgroup row for them)
  }
  const int tiles = p.k_tiles;
  const int last_chunk = p.d_in - 8, k_full = p.d_in / kW4K;
  const uint32_t lane16 = 16 * lane, lane_par = col * W4Params<KIND, SUB>::kBytes;
  const uint4 ones = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
  const uint32_t mask = w4_scalar(kCodeMask), magic = w4_vector(kMagicBf16);
  int rt_of[RT];
#pragma unroll
  for (int a = 0; a < RT; ++a) rt_of[a] = min(rt0 + a, p.row_tiles - 1);

  // ---- the rows: a run of rows (one matrix), or the rows whose id is e,
  // found in windows of kListMax rows.
  for (int win = 0; win < (listed ? p.R : 1); win += kListMax) {
  int base = 0, m_all = 0;
  if (!listed) {
    base = (int)blockIdx.y * kTok;
    m_all = min(kTok, p.R - base);
  } else {
    int cnt = w4_rows_of<W>(p, e, none, win, list, s_cnt);
    // By row (one window): an earlier row's workgroup has this matrix.
    if (p.by_row && (int)list[0] != self) return;
    base = win;
    if (none) {
      w4_zero_rows<E>(p, win, list, cnt, 16 * rt0, 16 * RT);
      cnt = 0;
    }
    m_all = cnt;
  }

  for (int m0 = 0; m0 < m_all; m0 += kTok) {
    const int m = min(kTok, m_all - m0);
    // Lanes of rows past m read the last row again: their columns are not used.
    const char* xrow[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) {
      const int i = m0 + min(16 * t + col, m - 1);
      const int r = base + (listed ? (int)list[i] : i);
      xrow[t] = p.x + (int64_t)(r / p.x_div) * p.ldx_bytes + 8 * h * E::kBytes;
    }
    f32x4_t acc[RT][NT];
#pragma unroll
    for (int a = 0; a < RT; ++a)
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[a][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};

    Slot<E, KIND, SUB, RT, NT> slot[U];
    const char* cb = p.codes + e * p.code_stride;
    const char* pb = p.params + e * p.param_stride;
    auto fetch = [&](int u, int kt) {
#pragma unroll
      for (int a = 0; a < RT; ++a) {
        const int64_t at = (int64_t)rt_of[a] * p.k_tiles + kt;
        slot[u].code[a] = ld16_stream(cb + at * kW4TileBytes + lane16);
        slot[u].par[a].load(pb + at * kW4Rows * W4Params<KIND, SUB>::kBytes + lane_par);
      }
      if (kt < k_full) {
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          const char* xk = xrow[t] + (int64_t)kt * (kW4K * E::kBytes);
#pragma unroll
          for (int j = 0; j < 4; ++j) slot[u].x[t][j].load(xk + 32 * j * E::kBytes);
        }
      } else {  // the tile that d_in ends in: chunks past the end meet codes equal to their zero point
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const int k = min(kW4K * kt + 32 * j + 8 * h, last_chunk) - 8 * h;
            slot[u].x[t][j].load(xrow[t] + (int64_t)k * E::kBytes);
          }
      }
    };
    auto compute = [&](int u) {
#pragma unroll
      for (int s = 0; s < SUB; ++s) {
        uint4 xp[NT][kStepsPerSub][XFrag<E>::kParts];
        f32x4_t xs[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          xs[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < kStepsPerSub; ++j) {
            slot[u].x[t][s * kStepsPerSub + j].parts(xp[t][j]);
            if constexpr (!kExact) xs[t] = mfma_bf16_16x16x32(xp[t][j][0], ones, xs[t]);
          }
        }
#pragma unroll
        for (int a = 0; a < RT; ++a) {
          const uint32_t cw[4] = {slot[u].code[a].x, slot[u].code[a].y, slot[u].code[a].z, slot[u].code[a].w};
          uint4 b[kStepsPerSub];
#pragma unroll
          for (int j = 0; j < kStepsPerSub; ++j)
            b[j] = kExact ? w4_expand_exact(cw[s * kStepsPerSub + j], mask, magic, slot[u].par[a].zero16(s))
                          : w4_expand(cw[s * kStepsPerSub + j], mask, magic);
          const float sc = slot[u].par[a].scale(s);
          const float zz = -slot[u].par[a].zero16(s);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            f32x4_t c;
#pragma unroll
            for (int v = 0; v < 4; ++v) c[v] = kExact ? 0.f : zz * xs[t][v];
#pragma unroll
            for (int j = 0; j < kStepsPerSub; ++j)
#pragma unroll
              for (int q = 0; q < XFrag<E>::kParts; ++q) c = mfma_bf16_16x16x32(xp[t][j][q], b[j], c);
#pragma unroll
            for (int v = 0; v < 4; ++v) acc[a][t][v] = fmaf(sc, c[v], acc[a][t][v]);
          }
        }
      }
    };
    // U tiles in flight per wave.  Loads past the last tile read it again
    // (an unconditional load keeps the waits of the earlier ones exact).
#pragma unroll
    for (int u = 0; u < U; ++u) fetch(u, min(w + u * W, tiles - 1));
    for (int i0 = w; i0 < tiles; i0 += U * W) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (i0 + u * W < tiles) compute(u);
        if (i0 + U * W < tiles) fetch(u, min(i0 + (u + U) * W, tiles - 1));
      }
    }

    // ---- the waves' sums, in wave order
#pragma unroll
    for (int a = 0; a < RT; ++a)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int v = 0; v < 4; ++v) red[w][a][t][(4 * h + v) * kPad + col] = acc[a][t][v];
    __syncthreads();
    for (int i = tid; i < 16 * m * RT; i += 64 * W) {
      const int o16 = i & 15, a = (i >> 4) % RT, row = (i >> 4) / RT;
      const int o = 16 * (rt0 + a) + o16;
      if (o >= p.d_out) continue;
      float v = 0.f;
#pragma unroll
      for (int ww = 0; ww < W; ++ww) v += red[ww][a][row >> 4][(row & 15) * kPad + o16];
      const int r = base + (listed ? (int)list[m0 + row] : row);
      char* yrow = p.y + (int64_t)r * p.ldy_bytes;
      w4_store<E>(yrow, o, v, p.f32_out);
    }
    __syncthreads();  // the sums (and, in a further window, the list) are written again
  }
  }
}

// y[t] = sum_j w[t, j] part[t k + j], in order of j; ids without a matrix add
// nothing.  One thread per 4 outputs.
template <typename E>
__global__ __launch_bounds__(256) void w4_combine_kernel(const float* __restrict__ part, const int32_t* __restrict__ ids,
                                                         const float* __restrict__ weights, int T, int k, int n, int d_out,
                                                         char* __restrict__ y, int64_t ldy_bytes) {
  const int o = 4 * (int)(blockIdx.y * 256 + threadIdx.x);
  const int t = (int)blockIdx.x;
  if (o >= d_out) return;
  f32x4_t s = {0.f, 0.f, 0.f, 0.f};
  for (int j = 0; j < k; ++j) {
    const int64_t r = (int64_t)t * k + j;
    if ((unsigned)ids[r] >= (unsigned)n) continue;
    const float wt = weights[r];
    const f32x4_t v = *reinterpret_cast<const f32x4_t*>(part + r * d_out + o);
#pragma unroll
    for (int i = 0; i < 4; ++i) s[i] = fmaf(wt, v[i], s[i]);
  }
  char* dst = y + (int64_t)t * ldy_bytes + (int64_t)o * E::kBytes;
  if constexpr (E::kBytes == 2)
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
  else
    *reinterpret_cast<f32x4_t*>(dst) = s;
}

template <typename E, int KIND, int SUB, int RT, int NT, int U, int W>
hipError_t launch_one(const W4RowsArgs& a, unsigned gy, hipStream_t stream) {
  const dim3 grid((unsigned)((a.row_tiles + RT - 1) / RT), gy);
  hipLaunchKernelGGL((w4_rows_kernel<E, KIND, SUB, RT, NT, U, W>), grid, dim3(64 * W), 0, stream, a);
  return hipGetLastError();
}

template <typename E, int KIND, int SUB>
hipError_t launch_rows(const W4RowsArgs& a, int rows_per, unsigned gy, hipStream_t stream) {
  constexpr int kU = E::kBytes == 2 ? 4 : 2;
  if (rows_per <= 16) return launch_one<E, KIND, SUB, 1, 1, kU, 8>(a, gy, stream);
  return launch_one<E, KIND, SUB, 2, 2, 1, 4>(a, gy, stream);
}

template <typename E>
hipError_t launch_kind(const W4RowsArgs& a, int kind, int sub, int rows_per, unsigned gy, hipStream_t st) {
  switch (kind * 8 + sub) {
    case kW4Bf16 * 8 + 1: return launch_rows<E, kW4Bf16, 1>(a, rows_per, gy, st);
    case kW4Bf16 * 8 + 2: return launch_rows<E, kW4Bf16, 2>(a, rows_per, gy, st);
    case kW4Bf16 * 8 + 4: return launch_rows<E, kW4Bf16, 4>(a, rows_per, gy, st);
    case kW4Bf16Zero * 8 + 1: return launch_rows<E, kW4Bf16Zero, 1>(a, rows_per, gy, st);
    case kW4Bf16Zero * 8 + 2: return launch_rows<E, kW4Bf16Zero, 2>(a, rows_per, gy, st);
    case kW4Bf16Zero * 8 + 4: return launch_rows<E, kW4Bf16Zero, 4>(a, rows_per, gy, st);
    case kW4F32 * 8 + 1: return launch_rows<E, kW4F32, 1>(a, rows_per, gy, st);
    case kW4F32 * 8 + 2: return launch_rows<E, kW4F32, 2>(a, rows_per, gy, st);
    default: return launch_rows<E, kW4F32, 4>(a, rows_per, gy, st);
  }
}

}  // namespace

hipError_t launch_w4_rows(const W4Call& c, hipStream_t stream) {
  if (c.R <= 0) return hipSuccess;
  const lora_w4_store& s = c.s;
  const int kind = w4_param_kind(s.scale_dtype, s.has_zeros), sub = w4_sub(s.group), eb = elem_bytes(c.dtype);
  W4RowsArgs a{};
  a.codes = reinterpret_cast<const char*>(s.codes);
  a.params = reinterpret_cast<const char*>(s.params);
  a.code_stride = w4_code_bytes(1, s.d_in, s.d_out);
  a.param_stride = w4_params_bytes(1, s.d_in, s.d_out, kind, sub);
  a.n = s.n;
  a.k_tiles = w4_k_tiles(s.d_in);
  a.row_tiles = w4_row_tiles(s.d_out);
  a.d_in = s.d_in;
  a.d_out = s.d_out;
  a.x = reinterpret_cast<const char*>(c.x);
  a.ldx_bytes = c.ldx * eb;
  a.x_div = c.x_div;
  a.y = reinterpret_cast<char*>(c.y);
  a.ldy_bytes = c.ldy * eb;
  a.R = c.R;
  a.k = c.k;
  a.ids = c.ids;
  int rows_per = c.R;
  unsigned gy;
  const bool combine = c.plan.sum_in_kernel;
  a.weights = combine ? c.weights : nullptr;
  const int cap = w4_few_rows(c.dtype, s.d_in);
  a.row_cap = cap < 16 ? cap : 16;
  if (combine) {
    gy = (unsigned)(c.R / c.k);
    a.row_cap = c.x_div == 1 ? c.k : 1;
    return launch_w4_few(a, c.dtype, kind, sub, gy, stream);
  } else if (c.ids != nullptr) {
    if (c.weights != nullptr) {
      a.y = c.ws + c.plan.part;
      a.ldy_bytes = (int64_t)s.d_out * 4;
      a.f32_out = 1;
    }
    a.by_row = c.R <= s.n && c.R <= kListMax;
    gy = a.by_row ? (unsigned)c.R : (unsigned)s.n + 1;
    rows_per = a.by_row ? 1 : (c.R + s.n - 1) / s.n;
  } else {
    gy = (unsigned)((c.R + (c.R <= 16 ? 15 : 31)) / (c.R <= 16 ? 16 : 32));
  }
  if (rows_per <= 16 && a.row_cap >= (rows_per < 16 ? rows_per : 16)) {
    const int want = rows_per + 3 < c.R ? rows_per + 3 : c.R;
    a.row_cap = a.row_cap < want ? a.row_cap : want;
    return launch_w4_few(a, c.dtype, kind, sub, c.ids ? gy : (unsigned)((c.R + a.row_cap - 1) / a.row_cap), stream);
  }
  return c.dtype == LORA_DTYPE_BF16 ? launch_kind<BF16>(a, kind, sub, rows_per, gy, stream)
                                    : launch_kind<F32>(a, kind, sub, rows_per, gy, stream);
}

hipError_t launch_w4_combine(const W4Call& c, const float* part, hipStream_t stream) {
  const int T = c.R / c.k, eb = elem_bytes(c.dtype), d_out = c.s.d_out;
  const dim3 grid((unsigned)T, (unsigned)((d_out / 4 + 255) / 256));
  char* y = reinterpret_cast<char*>(c.y);
  if (c.dtype == LORA_DTYPE_BF16)
    hipLaunchKernelGGL((w4_combine_kernel<BF16>), grid, dim3(256), 0, stream, part, c.ids, c.weights, T, c.k, c.s.n,
                       d_out, y, c.ldy * eb);
  else
    hipLaunchKernelGGL((w4_combine_kernel<F32>), grid, dim3(256), 0, stream, part, c.ids, c.weights, T, c.k, c.s.n,
                       d_out, y, c.ldy * eb);
  return hipGetLastError();
}

hipError_t launch_w4(const W4Call& c, hipStream_t stream) {
  hipError_t e = c.plan.bm > 0 ? launch_w4_gemm(c, stream) : launch_w4_rows(c, stream);
  if (e == hipSuccess && c.weights != nullptr && !c.plan.sum_in_kernel)
    e = launch_w4_combine(c, reinterpret_cast<const float*>(c.ws + c.plan.part), stream);
  return e;
}

}  // namespace lora
