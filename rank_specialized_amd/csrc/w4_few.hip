// 4-bit base products for at most 16 rows at a time, held in LDS (the decode
// step's own form):
//
//   y[r, o] = sum_g s[o, g] sum_{k in g} (q[o, k] - z[o, g]) x[r, k]
//
// The arithmetic is that of w4_rows.hip.  The difference is where x is: the
// workgroup copies its rows into LDS once, so that a wave's loads in flight
// are codes alone, U x RT KiB of them, and the time is that of the stream of
// codes.  (With x loaded beside the codes, a lane's four 16-byte pieces of x
// per tile take four times the registers of the codes and as many passes
// through the load path.)
#include "host_util.h"
#include "w4_kernels.h"
#include "w4_ops.h"

namespace lora {
namespace {

constexpr int kPad = 17;  // LDS row stride of a 16 x 16 block of sums

// An LDS barrier that leaves loads from memory in flight (__syncthreads()
// waits for them: its fence).
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}

// What the rows of a workgroup are: a run of rows (one matrix); the rows whose
// id is its matrix; or one token's k rows, each with its own matrix, summed.
enum Mode { kRun, kListed, kSum };

// At least two waves per SIMD: with up to 256 registers per lane the matrix
// instructions keep their results in ordinary registers, which the vector
// instructions around them read without a move.
template <typename E, int KIND, int SUB, int RT, int U, int W, int MODE>
__global__ __launch_bounds__(64 * W) __attribute__((amdgpu_waves_per_eu(2)))
void w4_few_kernel(const W4RowsArgs p) {
  constexpr int kParts = XFrag<E>::kParts;
  constexpr int kSteps = 4 / SUB;  // matrix-core steps per scale
  constexpr bool kExact = kParts > 1;
  constexpr int kBatch = 4;  // 16-byte pieces of x per thread and pass
  constexpr bool kSumUp = MODE == kSum, kList = MODE == kListed;
  extern __shared__ __align__(16) char xs[];
  __shared__ float red[W][RT][16 * kPad];
  __shared__ uint16_t list[kList ? kListMax : 1];
  __shared__ int s_cnt[W];
  const int tid = (int)threadIdx.x, lane = tid & 63;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6);  // uniform: the codes' addresses stay scalar
  const int col = lane & 15, h = lane >> 4;
  const int rt0 = (int)blockIdx.x * RT;
  const int plane = p.k_tiles * kW4K * 2, xrow_bytes = kParts * plane + 16;  // w4_few_row_bytes
  const int pieces = p.k_tiles * (kW4K / 8);  // of 8 values per row
  int e = 0, few_cnt = -1;
  bool none = false;
  if constexpr (kList) {
    if (p.by_row && p.R <= 64) {
      // One id per lane: each wave finds its matrix and the rows that have it
      // by itself (all waves write the same list).
      const int id = lane < p.R ? p.ids[lane] : 0;
      e = __builtin_amdgcn_readlane(id, blockIdx.y);
      none = (unsigned)e >= (unsigned)p.n;
      const bool hit = lane < p.R && (none ? (unsigned)id >= (unsigned)p.n : id == e);
      const uint64_t hits = __ballot(hit);
      if (__ffsll((unsigned long long)hits) - 1 != (int)blockIdx.y) return;  // an earlier row's workgroup has this matrix
      if (hit) list[__popcll(hits & lanemask_lt())] = (uint16_t)lane;
      few_cnt = __popcll(hits);
    } else {
      e = p.by_row ? p.ids[blockIdx.y] : (int)blockIdx.y;
      none = (unsigned)e >= (unsigned)p.n;  // rows without a matrix (by matrix: one workgroup row for them)
    }
  }
  const uint4 ones = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
  const uint32_t mask = w4_scalar(kCodeMask), magic = w4_vector(kMagicBf16);
  const uint32_t lane16 = 16 * lane, lane_par = col * W4Params<KIND, SUB>::kBytes;
  const char *code0[RT], *par0[RT];  // first tile of each output block
#pragma unroll
  for (int a = 0; a < RT; ++a) {
    const int64_t t = (int64_t)min(rt0 + a, p.row_tiles - 1) * p.k_tiles;
    code0[a] = p.codes + (kSumUp ? 0 : e * p.code_stride) + t * kW4TileBytes;
    par0[a] = p.params + (kSumUp ? 0 : e * p.param_stride) + t * kW4Rows * W4Params<KIND, SUB>::kBytes;
  }

  // m rows from base (or from list[m0]): x into LDS, the products, y.
  auto block = [&](int base, int m0, int m) {
    // ---- x into LDS, kBatch pieces per thread in flight: along one row, or
    // of kBatch rows.  The first are asked for before the codes.
    const int x_rows = kSumUp ? (p.x_div == 1 ? p.k : 1) : m;
    XFrag<E> hold[kBatch];
    auto x_row = [&](int i) {
      uint32_t r = base + i;
      if constexpr (kList) r = base + __builtin_amdgcn_readfirstlane((int)list[m0 + i]);
      if constexpr (MODE != kRun) r /= (uint32_t)p.x_div;
      return p.x + (int64_t)r * p.ldx_bytes;
    };
    auto ask = [&](int row0, int c0, int along) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const uint32_t k = 8 * (c0 + i * along);
        const char* src = x_row(along ? row0 : min(row0 + i, x_rows - 1));
        hold[i] = XFrag<E>{};
        if (k < (uint32_t)p.d_in) hold[i].load(src + k * E::kBytes);
      }
    };
    auto put = [&](int row0, int c0, int along) {
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const int row = along ? row0 : min(row0 + i, x_rows - 1), at = c0 + i * along;
        if (at >= pieces) continue;
        uint4 parts[kParts];
        hold[i].parts(parts);
#pragma unroll
        for (int q = 0; q < kParts; ++q) *reinterpret_cast<uint4*>(xs + row * xrow_bytes + q * plane + 16 * at) = parts[q];
      }
    };
    constexpr int kThreads = 64 * W;
    if (x_rows == 1) ask(0, tid, kThreads);
    else ask(0, tid, 0);

    // ---- codes: U tiles of each output block in flight per wave, taken in
    // turn by the waves; loads past the last tile read it again (an
    // unconditional load keeps the waits of the earlier ones exact).
    uint4 code[U][RT];
    W4Params<KIND, SUB> par[U][RT];
    const int tiles = (kSumUp ? p.k : 1) * p.k_tiles;
    int cur_j = -1, cur_id = 0;
    float cur_w = 0.f;
    float slot_w[U];
    int slot_x[U];  // LDS offset of the tile's x; -1: a row without a matrix
    auto fetch = [&](int u, int i) {
      int kt = i;
      int64_t mat = 0;
      if constexpr (kSumUp) {
        const int j = (int)((uint32_t)i / (uint32_t)p.k_tiles);
        kt = i - j * p.k_tiles;
        if (j != cur_j) {
          cur_j = j;
          cur_id = p.ids[base + j];
          cur_w = p.weights[base + j];
        }
        const bool ok = (unsigned)cur_id < (unsigned)p.n;
        mat = ok ? cur_id : 0;
        slot_w[u] = cur_w;
        slot_x[u] = ok ? (p.x_div == 1 ? j * xrow_bytes : 0) + kt * kW4K * 2 : -1;
      } else {
        slot_x[u] = kt * kW4K * 2;
      }
#pragma unroll
      for (int a = 0; a < RT; ++a) {
        code[u][a] = ld16_stream(code0[a] + (mat * p.code_stride + (int64_t)kt * kW4TileBytes) + lane16);
        par[u][a].load(par0[a] + (mat * p.param_stride + (int64_t)kt * (kW4Rows * W4Params<KIND, SUB>::kBytes)) + lane_par);
      }
    };
#pragma unroll
    for (int u = 0; u < U; ++u) fetch(u, min(w + u * W, tiles - 1));
    if (x_rows == 1) {
      put(0, tid, kThreads);
      for (int c0 = tid + kBatch * kThreads; c0 - tid < pieces; c0 += kBatch * kThreads) {
        ask(0, c0, kThreads);
        put(0, c0, kThreads);
      }
    } else {
      put(0, tid, 0);
      for (int row0 = 0; row0 < x_rows; row0 += kBatch)
        for (int c0 = tid + (row0 == 0 ? kThreads : 0); c0 - tid < pieces; c0 += kThreads) {
          ask(row0, c0, 0);
          put(row0, c0, 0);
        }
    }
    lds_barrier();

    f32x4_t acc[RT];
#pragma unroll
    for (int a = 0; a < RT; ++a) acc[a] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    // Lanes of rows past m read the last row: their results are not used.
    const char* xl = xs + (kSumUp ? 0 : min(col, m - 1) * xrow_bytes) + 16 * h;
    auto compute = [&](int u) {
      const char* xk = xl + slot_x[u];
#pragma unroll
      for (int s = 0; s < SUB; ++s) {
        uint4 xp[kSteps][kParts];
        f32x4_t xsum = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
#pragma unroll
          for (int q = 0; q < kParts; ++q) xp[j][q] = ld16(xk + q * plane + 64 * (s * kSteps + j));
          if constexpr (!kExact) xsum = mfma_bf16_16x16x32(xp[j][0], ones, xsum);
        }
#pragma unroll
        for (int a = 0; a < RT; ++a) {
          const uint32_t cw[4] = {code[u][a].x, code[u][a].y, code[u][a].z, code[u][a].w};
          const float sc = kSumUp ? par[u][a].scale(s) * slot_w[u] : par[u][a].scale(s);
          const float z16 = par[u][a].zero16(s);
          f32x4_t c;
#pragma unroll
          for (int v = 0; v < 4; ++v) c[v] = kExact ? 0.f : -z16 * xsum[v];
#pragma unroll
          for (int j = 0; j < kSteps; ++j) {
            const uint4 b = kExact ? w4_expand_exact(cw[s * kSteps + j], mask, magic, z16)
                                   : w4_expand(cw[s * kSteps + j], mask, magic);
#pragma unroll
            for (int q = 0; q < kParts; ++q) c = mfma_bf16_16x16x32(xp[j][q], b, c);
          }
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[a][v] = fmaf(sc, c[v], acc[a][v]);
        }
      }
    };
    for (int i0 = w; i0 < tiles; i0 += U * W) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        if (i0 + u * W < tiles && (!kSumUp || slot_x[u] >= 0)) compute(u);
        if (i0 + U * W < tiles) fetch(u, min(i0 + (u + U) * W, tiles - 1));
      }
    }

    // ---- the waves' sums, in wave order
#pragma unroll
    for (int a = 0; a < RT; ++a)
#pragma unroll
      for (int v = 0; v < 4; ++v)
        if (4 * h + v < m) red[w][a][(4 * h + v) * kPad + col] = acc[a][v];
    __syncthreads();
    for (int i = tid; i < 16 * m * RT; i += kThreads) {
      const int o16 = i & 15, a = (i >> 4) % RT, row = (i >> 4) / RT;
      const int o = 16 * (rt0 + a) + o16;
      if (o >= p.d_out) continue;
      float v = 0.f;
#pragma unroll
      for (int ww = 0; ww < W; ++ww) v += red[ww][a][row * kPad + o16];
      const int r = kSumUp ? (int)blockIdx.y : base + (kList ? (int)list[m0 + row] : row);
      w4_store<E>(p.y + (int64_t)r * p.ldy_bytes, o, v, p.f32_out);
    }
  };

  if constexpr (MODE == kRun) {
    const int base = (int)blockIdx.y * p.row_cap;
    block(base, 0, min(p.row_cap, p.R - base));
  } else if constexpr (kSumUp) {
    block((int)blockIdx.y * p.k, 0, 1);
  } else {
    for (int win = 0; win < p.R; win += kListMax) {
      int cnt = few_cnt;
      if (cnt < 0) {
        cnt = w4_rows_of<W>(p, e, none, win, list, s_cnt);
        if (p.by_row && (int)list[0] != (int)blockIdx.y) return;
      }
      if (none) {
        w4_zero_rows<E>(p, win, list, cnt, 16 * rt0, 16 * RT);
      } else {
        for (int m0 = 0; m0 < cnt; m0 += p.row_cap) {
          block(win, m0, min(p.row_cap, cnt - m0));
          __syncthreads();  // the sums, x and the list are written again
        }
      }
      __syncthreads();
    }
  }
}

template <typename E, int KIND, int SUB, int RT, int U, int W, int MODE>
hipError_t launch_one(const W4RowsArgs& a, unsigned gy, hipStream_t stream) {
  const dim3 grid((unsigned)((a.row_tiles + RT - 1) / RT), gy);
  const size_t lds = (size_t)a.row_cap * w4_few_row_bytes(E::kBytes == 2 ? LORA_DTYPE_BF16 : LORA_DTYPE_F32, a.d_in);
  static DynLdsLimit lim;
  const hipError_t e = ensure_dynamic_lds(lim, reinterpret_cast<const void*>(w4_few_kernel<E, KIND, SUB, RT, U, W, MODE>), lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((w4_few_kernel<E, KIND, SUB, RT, U, W, MODE>), grid, dim3(64 * W), lds, stream, a);
  return hipGetLastError();
}

template <typename E, int KIND, int SUB, int MODE>
hipError_t launch_mode(const W4RowsArgs& a, unsigned gy, hipStream_t stream) {
  if constexpr (MODE == kSum) {
    return launch_one<E, KIND, SUB, 1, 4, 16, MODE>(a, gy, stream);
  } else {
    // Outputs per workgroup by the number of 16-output blocks in the call (of
    // all matrices with rows): 
    const int64_t blocks = (int64_t)a.row_tiles * (MODE == kRun || a.by_row ? gy : (a.R < a.n ? a.R : a.n));
    if (blocks < 512) return launch_one<E, KIND, SUB, 1, 2, 8, MODE>(a, gy, stream);
    if (blocks < 1280) return launch_one<E, KIND, SUB, 1, 4, 4, MODE>(a, gy, stream);
    if (blocks < 2816) return launch_one<E, KIND, SUB, 2, 2, 4, MODE>(a, gy, stream);
    return launch_one<E, KIND, SUB, 4, 1, 4, MODE>(a, gy, stream);
  }
}

template <typename E, int KIND, int SUB>
hipError_t launch_shape(const W4RowsArgs& a, unsigned gy, hipStream_t stream) {
  if (a.weights != nullptr) return launch_mode<E, KIND, SUB, kSum>(a, gy, stream);
  if (a.ids != nullptr) return launch_mode<E, KIND, SUB, kListed>(a, gy, stream);
  return launch_mode<E, KIND, SUB, kRun>(a, gy, stream);
}

template <typename E>
hipError_t launch_kind(const W4RowsArgs& a, int kind, int sub, unsigned gy, hipStream_t st) {
  switch (kind * 8 + sub) {
    case kW4Bf16 * 8 + 1: return launch_shape<E, kW4Bf16, 1>(a, gy, st);
    case kW4Bf16 * 8 + 2: return launch_shape<E, kW4Bf16, 2>(a, gy, st);
    case kW4Bf16 * 8 + 4: return launch_shape<E, kW4Bf16, 4>(a, gy, st);
    case kW4Bf16Zero * 8 + 1: return launch_shape<E, kW4Bf16Zero, 1>(a, gy, st);
    case kW4Bf16Zero * 8 + 2: return launch_shape<E, kW4Bf16Zero, 2>(a, gy, st);
    case kW4Bf16Zero * 8 + 4: return launch_shape<E, kW4Bf16Zero, 4>(a, gy, st);
    case kW4F32 * 8 + 1: return launch_shape<E, kW4F32, 1>(a, gy, st);
    case kW4F32 * 8 + 2: return launch_shape<E, kW4F32, 2>(a, gy, st);
    default: return launch_shape<E, kW4F32, 4>(a, gy, st);
  }
}

}  // namespace

hipError_t launch_w4_few(const W4RowsArgs& a, int dtype, int kind, int sub, unsigned gy, hipStream_t stream) {
  return dtype == LORA_DTYPE_BF16 ? launch_kind<BF16>(a, kind, sub, gy, stream) : launch_kind<F32>(a, kind, sub, gy, stream);
}

}  // namespace lora
