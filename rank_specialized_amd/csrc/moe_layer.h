// A mixture-of-experts layer for a few tokens, in two kernels:
//
//   h[t, e] = act(G_e x[t]) * (U_e x[t])          e = ids[t, j]
//   y[t]    = sum_j w[t, j] D_e h[t, e]
//
// with 4-bit matrices (w4.h).  What bounds both is the stream of codes.  In
// both, a workgroup owns some blocks of 16 outputs of one expert for the tokens that chose
// it: the rows lie in LDS, WK waves share the 128-input tiles of 16 outputs,
// and their sums meet in LDS, in wave order.  Codes enter the bf16 matrix cores
// as in the few-rows products (w4_rows.h): 32 + q with (32 + z) times the rows'
// sum taken off, or, for float32 rows, q - z itself.
//
// Rows that are more than one bf16 number wide are several rows of a product:
// of bf16 tokens x is one and h two, of float32 tokens three each.  For a few
// tokens they share one 16 x 16 product that would be mostly empty otherwise.
//
// Kernel 1 (gate and up): every wave finds the expert's tokens by itself, a
// token per lane.  h leaves as bf16 parts, the rows of the second kernel, and
// the tokens as an entry of a table.
// Kernel 2 (down): a workgroup leaves weighted float32 rows, and the one that
// comes last of those that share its outputs adds each token's, in order of its
// choices: sums have one order, whatever the schedule.
#pragma once
#include "host_util.h"
#include "moe_kernels.h"
#include "w4_ops.h"

namespace lora {
namespace {

constexpr int kMoeIds = 8;           // 64 choices each that a wave looks through in registers
constexpr int kMoePad = 17;          // LDS row stride of a 16 x 16 block of sums
constexpr int kMoeLds = 76 * 1024;   // of rows: two workgroups to a compute unit

// The tiles of codes of NB blocks of 16 outputs, U of each in flight, and their
// products with 16 NT rows.
template <int KIND, int SUB, bool EXACT, int NB, int NT, int WK, int U>
struct MoeStream {
  typedef W4Params<KIND, SUB> Par;
  const char *code0[NB], *par0[NB];  // uniform
  uint32_t lane_code, lane_par;
  uint4 code[U][NB];
  Par par[U][NB];
  uint32_t mask, magic;

  __device__ __forceinline__ void fetch(int u, int kt) {
#pragma unroll
    for (int a = 0; a < NB; ++a) {
      code[u][a] = ld16(code0[a] + (int64_t)kt * kW4TileBytes + lane_code);
      par[u][a].load(par0[a] + (int64_t)kt * (kW4Rows * Par::kBytes) + lane_par);
    }
  }
  __device__ __forceinline__ void start(int wk, int c0, int c1) {
#pragma unroll
    for (int u = 0; u < U; ++u) fetch(u, min(c0 + wk + u * WK, c1 - 1));
  }
  // The products of one tile: x at this lane's row and piece.
  __device__ __forceinline__ void tile(int u, const char* const (&x)[NT], uint32_t at, f32x4_t (&acc)[NB][NT]) {
    constexpr int kSteps = 4 / SUB;
    const uint4 ones = make_uint4(0x3f803f80u, 0x3f803f80u, 0x3f803f80u, 0x3f803f80u);
#pragma unroll
    for (int s = 0; s < SUB; ++s) {
      uint4 b[NB][kSteps];
#pragma unroll
      for (int a = 0; a < NB; ++a) {
        const uint32_t cw[4] = {code[u][a].x, code[u][a].y, code[u][a].z, code[u][a].w};
#pragma unroll
        for (int j = 0; j < kSteps; ++j)
          b[a][j] = EXACT ? w4_expand_exact(cw[s * kSteps + j], mask, magic, par[u][a].zero32(s))
                          : w4_expand(cw[s * kSteps + j], mask, magic);
      }
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        uint4 xp[kSteps];
        f32x4_t xsum = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
        for (int j = 0; j < kSteps; ++j) {
          xp[j] = ld16(x[t] + at + 64 * (s * kSteps + j));
          if constexpr (!EXACT) xsum = mfma_bf16_16x16x32(xp[j], ones, xsum);
        }
#pragma unroll
        for (int a = 0; a < NB; ++a) {
          const float sc = par[u][a].scale(s), z32 = par[u][a].zero32(s);
          f32x4_t c;
#pragma unroll
          for (int v = 0; v < 4; ++v) c[v] = EXACT ? 0.f : -z32 * xsum[v];
#pragma unroll
          for (int j = 0; j < kSteps; ++j) c = mfma_bf16_16x16x32(xp[j], b[a][j], c);
#pragma unroll
          for (int v = 0; v < 4; ++v) acc[a][t][v] = fmaf(sc, c[v], acc[a][t][v]);
        }
        if (NT > 1) asm volatile("" ::: "memory");  // the next rows' reads take these registers
      }
    }
  }
  __device__ __forceinline__ void tiles(int wk, int c0, int c1, const char* const (&x)[NT], f32x4_t (&acc)[NB][NT]) {
    for (int i0 = c0 + wk; i0 < c1; i0 += U * WK) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int i = i0 + u * WK;
        if (i < c1) tile(u, x, (uint32_t)(i - c0) * (kW4K * 2), acc);
        if (i0 + U * WK < c1) fetch(u, min(i + U * WK, c1 - 1));
      }
    }
  }
};

// Tiles of `rows` rows that LDS holds at a time.
__device__ __forceinline__ int moe_chunk(int lds_bytes, int rows, int k_tiles) {
  return min(k_tiles, (lds_bytes / rows - 16) / (kW4K * 2));
}
// An LDS barrier behind every load that the wave has asked for.
__device__ __forceinline__ void moe_loads_barrier() {
  __builtin_amdgcn_s_waitcnt(0);
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}
// Tiles [c0, c1) of rows of bf16 numbers into LDS by loads that write it
// directly, all of them in flight at once; row i from src(i), which is uniform.
// A wave-wide load takes four tiles of a row, pieces from `pieces` on repeat the
// one before.
template <int W, typename Src>
__device__ __forceinline__ void moe_dma(char* lds, int stride, int rows, int c0, int c1, int pieces, int w, int lane, Src src) {
  const int per_row = (c1 - c0 + 3) >> 2;
  for (int row = 0, f = w; row < rows; ++row, f -= per_row)
    for (; f < per_row; f += W)
      if (64 * f + lane < 16 * (c1 - c0)) {
        const uint32_t at = (uint32_t)min(16 * c0 + 64 * f + lane, pieces - 1) * 16;
        __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(src(row) + at),
                                         (__attribute__((address_space(3))) void*)(lds + row * stride + f * 1024), 16, 0, 0);
      }
}

// `rows` rows (at most 16 NT) of k_tiles tiles through a stream that `start`
// has begun: `fill(c0, c1, stride)` asks for tiles [c0, c1) of them to be
// written to LDS, `ends(c0, stride)` clears what lies behind a row's end in the
// last of them (`ragged`).  The sums of the wave land in red[wave][block][16-row
// tile].
template <int NB, int NT, typename Stream, typename Fill, typename Ends>
__device__ __forceinline__ void moe_products(Stream& st, int tid, int wk, int w, int k_tiles, int rows, char* lds, int chunk,
                                             bool ragged, Fill fill, Ends ends) {
  const int lane = tid & 63, col = lane & 15, h = lane >> 4;
  const int stride = chunk * kW4K * 2 + 16;
  const char* x[NT];
#pragma unroll
  for (int t = 0; t < NT; ++t) x[t] = lds + min(16 * t + col, rows - 1) * stride + 16 * h;
  f32x4_t acc[NB][NT];
#pragma unroll
  for (int a = 0; a < NB; ++a)
#pragma unroll
    for (int t = 0; t < NT; ++t) acc[a][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
  for (int c0 = 0; c0 < k_tiles; c0 += chunk) {
    const int c1 = min(k_tiles, c0 + chunk);
    if (c0 > 0) {
      __syncthreads();  // the chunk before has been read
      st.start(wk, c0, c1);
    }
    fill(c0, c1, stride);
    moe_loads_barrier();
    if (ragged && c1 == k_tiles) {
      ends(c0, stride);
      __syncthreads();
    }
    st.tiles(wk, c0, c1, x, acc);
  }
  __syncthreads();
  float* red = reinterpret_cast<float*>(lds) + (4 * h) * kMoePad + col;
#pragma unroll
  for (int a = 0; a < NB; ++a)
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
      for (int v = 0; v < 4; ++v) red[((w * NB + a) * NT + t) * 16 * kMoePad + v * kMoePad] = acc[a][t][v];
  __syncthreads();
}
// The sum of WK waves from w0 on, block a, of output c and a token's PARTS rows.
template <int NB, int NT, int WK, int PARTS>
__device__ __forceinline__ float moe_sum(const float* red, int w0, int a, int m, int r, int c) {
  float s = 0.f;
#pragma unroll
  for (int q = PARTS - 1; q >= 0; --q) {  // the small parts first
    const int row = q * m + r;
#pragma unroll
    for (int ww = 0; ww < WK; ++ww)
      s += red[(((w0 + ww) * NB + a) * NT + (row >> 4)) * 16 * kMoePad + (row & 15) * kMoePad + c];
  }
  return s;
}
// LDS bytes of the waves' sums.
constexpr int moe_sum_bytes(int waves, int nb, int nt) { return waves * nb * nt * 16 * kMoePad * 4; }
// An opaque copy of a lane's number, so that nothing that depends on it is held
// in registers across a loop.
__device__ __forceinline__ int moe_tid() {
  int tid = (int)threadIdx.x;
  asm volatile("" : "+v"(tid));
  return tid;
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
  uint8_t* counted;
  uint32_t* arrived;
  int groups, entries;
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

template <typename E, int KIND, int SUB, int NT, int WB, int WK, int U>
__global__ __launch_bounds__(64 * WB * WK) __attribute__((amdgpu_waves_per_eu(NT == 1 ? 4 : 2)))
void moe_up_kernel(const MoeUpArgs p) {
  constexpr int kParts = XFrag<E>::kParts, kHParts = kParts == 1 ? 2 : 3, W = WB * WK;
  constexpr int kTokens = 16 * NT / kParts;  // at a time
  extern __shared__ __align__(16) char lds[];  // x; then the waves' sums
  __shared__ uint16_t s_row[LORA_W4_MOE_MAX_TOKENS], s_tok[LORA_W4_MOE_MAX_TOKENS];
  __shared__ float s_sum[LORA_W4_MOE_MAX_TOKENS];
  const int tid = (int)threadIdx.x, lane = tid & 63, col = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6), wb = w / WK, wk = w % WK;

  const int R = p.T * p.k;
  if ((int)blockIdx.y == p.entries) {
    // For the second kernel: nobody has arrived, and the choices that count (an
    // expert's first in a token).
    if (blockIdx.x > 0) return;
    for (int i = tid; i < p.groups; i += 64 * W) p.arrived[i] = 0u;
    for (int r = tid; r < R; r += 64 * W) {
      const int own = p.ids[r], r0 = r / p.k * p.k;
      bool ok = (unsigned)own < (unsigned)p.n;
#pragma unroll 4
      for (int i = r0; i < r; ++i) ok = ok && p.ids[i] != own;
      p.counted[r] = ok;
    }
    return;
  }
  // ---- asked for in the order they are waited for: the choices, then the
  // expert's first codes
  int id[kMoeIds];
#pragma unroll
  for (int i = 0; i < kMoeIds; ++i) id[i] = p.ids[min(64 * i + lane, R - 1)];
  const int e = p.by_row ? p.ids[blockIdx.y] : (int)blockIdx.y, e0 = (unsigned)e < (unsigned)p.n ? e : 0;
  asm volatile("" ::: "memory");
  const int fb = (int)blockIdx.x * WB + wb;  // block of 16 features; from row_tiles on: pads of h
  const int64_t tile0 = (int64_t)min(fb, p.row_tiles - 1) * p.k_tiles;
  typedef MoeStream<KIND, SUB, (kParts > 1), 2, NT, WK, U> Stream;
  const int64_t code_at = e0 * p.code_stride + tile0 * kW4TileBytes;
  const int64_t par_at = e0 * p.param_stride + tile0 * kW4Rows * Stream::Par::kBytes;
  Stream st;
  st.code0[0] = p.gate + code_at;
  st.code0[1] = p.up + code_at;
  st.par0[0] = p.gate_par + par_at;
  st.par0[1] = p.up_par + par_at;
  st.mask = w4_scalar(kCodeMask);
  st.magic = w4_vector(kMagicBf16);
  st.lane_code = 16 * lane;
  st.lane_par = col * Stream::Par::kBytes;
  st.start(wk, 0, p.k_tiles);
  asm volatile("" ::: "memory");

  // ---- the expert's tokens, in order; every wave finds the same, and reads
  // what it has written itself
  int cnt = 0, first_row = -1;
  float wsum = 0.f;
  bool plain = R <= 64 * kMoeIds;  // every token names the expert once
  if (plain) {
#pragma unroll
    for (int i = 0; i < kMoeIds; ++i) {
      const int r = 64 * i + lane;
      const uint64_t hits = __ballot(r < R && id[i] == e);
      const int at = cnt + __popcll(hits & lanemask_lt());
      if (((hits >> lane) & 1) && at < LORA_W4_MOE_MAX_TOKENS) s_row[at] = (uint16_t)r;
      cnt += __popcll(hits);
    }
    plain = cnt <= LORA_W4_MOE_MAX_TOKENS;
    if (plain && lane < cnt) {
      first_row = s_row[lane];
      const int tok = first_row / p.k;
      s_tok[lane] = (uint16_t)tok;
      plain = lane == 0 || (int)s_row[lane - 1] / p.k != tok;
    }
    plain = __all(plain);
    if (plain && blockIdx.x == 0 && lane < cnt) wsum = p.weights[first_row];
  }
  if (!plain) {  // a token per lane, its weights added up
    __syncthreads();  // no wave writes the list above any more
    int first = -1;
    if (lane < p.T)
      for (int r = lane * p.k; r < (lane + 1) * p.k; ++r)
        if (p.ids[r] == e) {
          wsum = first < 0 ? p.weights[r] : wsum + p.weights[r];
          first = first < 0 ? r : first;
        }
    const uint64_t hits = __ballot(first >= 0);
    cnt = __popcll(hits);
    // Into the first lanes, through LDS.
    const int at = __popcll(hits & lanemask_lt());
    if (first >= 0) {
      s_row[at] = (uint16_t)first;
      s_tok[at] = (uint16_t)lane;
      s_sum[at] = wsum;
    }
    first_row = lane < cnt ? s_row[lane] : -1;
    wsum = lane < cnt ? s_sum[lane] : 0.f;
  }
  if ((unsigned)e >= (unsigned)p.n) cnt = 0;
  // By choice: the first row of an expert works for all of its rows.
  if (cnt > 0 && p.by_row && __builtin_amdgcn_readfirstlane(first_row) != (int)blockIdx.y) cnt = 0;
  if (blockIdx.x == 0 && w == 0) {
    MoeEntry& t = p.table[blockIdx.y];
    if (lane == 0) {
      t.e = e;
      t.cnt = cnt;
    }
    if (lane < cnt) {
      t.row[lane] = (uint16_t)first_row;
      t.w[lane] = wsum;
    }
  }
  if (cnt == 0) return;
  for (int m0 = 0; m0 < cnt; m0 += kTokens) {
    const int tid = moe_tid(), m = min(kTokens, cnt - m0), rows = m * kParts;
    const int chunk = moe_chunk(p.lds_bytes, rows, p.k_tiles);
    if (m0 > 0) {
      __syncthreads();  // the sums before have been read
      st.start(wk, 0, chunk);
    }
    moe_products<2, NT>(
        st, tid, wk, w, p.k_tiles, rows, lds, chunk, p.d % kW4K != 0,
        [&](int c0, int c1, int stride) {
          if constexpr (kParts == 1) {
            moe_dma<W>(lds, stride, m, c0, c1, p.d / 8, w, tid & 63, [&](int r) {
              return p.x + (int64_t)__builtin_amdgcn_readfirstlane((int)s_tok[m0 + r]) * p.ldx_bytes;
            });
          } else {
            constexpr int kBatch = 4;  // pieces in flight per lane
            const int pieces = (c1 - c0) * (kW4K / 8), total = m * pieces;
            for (int i0 = tid; i0 < total; i0 += 64 * W * kBatch) {
              XFrag<E> f[kBatch];
#pragma unroll
              for (int b = 0; b < kBatch; ++b) {
                const int i = min(i0 + 64 * W * b, total - 1), r = (int)((uint32_t)i / (uint32_t)pieces), pc = i - r * pieces;
                f[b].load(p.x + (int64_t)s_tok[m0 + r] * p.ldx_bytes + (int64_t)min(c0 * kW4K + 8 * pc, p.d - 8) * E::kBytes);
              }
#pragma unroll
              for (int b = 0; b < kBatch; ++b) {
                const int i = min(i0 + 64 * W * b, total - 1), r = (int)((uint32_t)i / (uint32_t)pieces), pc = i - r * pieces;
                uint4 parts[kParts];
                f[b].parts(parts);
#pragma unroll
                for (int q = 0; q < kParts; ++q) st16(lds + (q * m + r) * stride + 16 * pc, parts[q]);
              }
            }
          }
        },
        [&](int c0, int stride) {
          const int pads = (kW4K - p.d % kW4K) / 8;  // 16-byte pieces
          for (int i = tid; i < rows * pads; i += 64 * W)
            st16(lds + i / pads * stride + (p.k_tiles - c0) * kW4K * 2 - 16 * (1 + i % pads), make_uint4(0u, 0u, 0u, 0u));
        });
    const float* red = reinterpret_cast<const float*>(lds);
    for (int i = tid; i < WB * 16 * m; i += 64 * W) {
      const int c = i & 15, b = (i >> 4) % WB, r = (i >> 4) / WB;
      const float g = moe_sum<2, NT, WK, kParts>(red, b * WK, 0, m, r, c);
      const float u = moe_sum<2, NT, WK, kParts>(red, b * WK, 1, m, r, c);
      const int f = 16 * ((int)blockIdx.x * WB + b) + c, fp = p.h_tiles * kW4K;
      if (f >= fp) continue;
      uint16_t o[kHParts];
      moe_parts<kHParts>(f < p.ffn ? moe_act(p.act, g, u) : 0.f, o);
#pragma unroll
      for (int q = 0; q < kHParts; ++q) p.h[((int64_t)s_row[m0 + r] * kHParts + q) * fp + f] = o[q];
    }
  }
}

// ------------------------------------------------------------ down
struct MoeDownArgs {
  const char *codes, *params;
  int64_t code_stride, param_stride;
  int d_out, k_tiles, row_tiles;
  int T, k, lds_bytes;
  const uint16_t* h;
  const MoeEntry* table;
  float* part;  // by group of outputs
  const uint8_t* counted;
  uint32_t* arrived;
  char* y;
  int64_t ldy_bytes;
};

// Values that another workgroup of the kernel reads: stores and loads of the
// device's scope (bit sc1), which pass by the caches that are not coherent
// between the XCDs.  A wave's stores have reached memory once it has waited for
// them; then it may be counted as arrived.  (A fence of that scope writes back
// all of an XCD's L2: 26 us for the kernel of one token, 8 of 64 experts 1408 ->
// 2048, and 11 so.)
constexpr int kDeviceScope = 16;
__device__ __forceinline__ void moe_publish(float* p, float v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ void moe_published() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }
__device__ __forceinline__ f32x4_t moe_collect(rsrc_t r, uint32_t at) {
  return __builtin_bit_cast(f32x4_t, __builtin_amdgcn_raw_buffer_load_b128(r, at, 0, kDeviceScope));
}

// A wave owns NB blocks of 16 outputs.
template <typename E, int KIND, int SUB, int NT, int NB, int WK, int U>
__global__ __launch_bounds__(64 * (moe_down_blocks(NT == 2) / NB) * WK) __attribute__((amdgpu_waves_per_eu(NT == 1 ? 4 : 2)))
void moe_down_kernel(const MoeDownArgs p) {
  constexpr int kParts = E::kBytes == 2 ? 2 : 3, kBlocks = moe_down_blocks(NT == 2), W = kBlocks / NB * WK;
  constexpr int kTokens = 16 * NT / kParts;
  extern __shared__ __align__(16) char lds[];
  __shared__ uint16_t s_row[LORA_W4_MOE_MAX_TOKENS];
  __shared__ float s_w[LORA_W4_MOE_MAX_TOKENS];
  __shared__ int last;
  const int tid = (int)threadIdx.x, lane = tid & 63, col = lane & 15;
  const int w = __builtin_amdgcn_readfirstlane(tid >> 6), wb = w / WK, wk = w % WK;
  const MoeEntry& t = p.table[blockIdx.y];
  constexpr int kCols = 16 * kBlocks;
  const int e = t.e, cnt = t.cnt, o0 = (int)blockIdx.x * kCols, R = p.T * p.k;
  float* part = p.part + (int64_t)blockIdx.x * R * kCols;
  typedef MoeStream<KIND, SUB, (kParts > 2), NB, NT, WK, U> Stream;
  const int my_row = t.row[lane];  // behind cnt: not used
  const float my_w = t.w[lane];
  if (cnt > 0) {
    Stream st;
#pragma unroll
    for (int a = 0; a < NB; ++a) {
      const int64_t tile0 = (int64_t)min((int)blockIdx.x * kBlocks + wb * NB + a, p.row_tiles - 1) * p.k_tiles;
      st.code0[a] = p.codes + e * p.code_stride + tile0 * kW4TileBytes;
      st.par0[a] = p.params + e * p.param_stride + tile0 * kW4Rows * Stream::Par::kBytes;
    }
    st.mask = w4_scalar(kCodeMask);
    st.magic = w4_vector(kMagicBf16);
    st.lane_code = 16 * lane;
    st.lane_par = col * Stream::Par::kBytes;
    st.start(wk, 0, p.k_tiles);
    asm volatile("" ::: "memory");
    if (lane < cnt) {  // all waves write the same, and read what they have written
      s_row[lane] = (uint16_t)my_row;
      s_w[lane] = my_w;
    }
    const int plane = p.k_tiles * kW4K * 2;
    for (int m0 = 0; m0 < cnt; m0 += kTokens) {
      const int tid = moe_tid(), m = min(kTokens, cnt - m0), rows = m * kParts;
      const int chunk = moe_chunk(p.lds_bytes, rows, p.k_tiles);
      if (m0 > 0) {
        __syncthreads();
        st.start(wk, 0, chunk);
      }
      moe_products<NB, NT>(
          st, tid, wk, w, p.k_tiles, rows, lds, chunk, false,
          [&](int c0, int c1, int stride) {
            moe_dma<W>(lds, stride, rows, c0, c1, 16 * p.k_tiles, w, tid & 63, [&](int i) {
              const int q = i / m, r = __builtin_amdgcn_readfirstlane((int)s_row[m0 + i - q * m]);
              return reinterpret_cast<const char*>(p.h) + ((int64_t)r * kParts + q) * plane;
            });
          },
          [&](int, int) {});
      const float* red = reinterpret_cast<const float*>(lds);
      for (int i = tid; i < kBlocks * 16 * m; i += 64 * W) {
        const int c = i & 15, b = (i >> 4) % kBlocks, r = (i >> 4) / kBlocks, o = o0 + 16 * b + c;
        if (o < p.d_out)
          moe_publish(part + (int)s_row[m0 + r] * kCols + 16 * b + c,
                      s_w[m0 + r] * moe_sum<NB, NT, WK, kParts>(red, b / NB * WK, b % NB, m, r, c));
      }
    }
    moe_published();
  }
  // ---- the last workgroup of these outputs adds the choices' rows
  __syncthreads();
  if (tid == 0)
    last = __hip_atomic_fetch_add(&p.arrived[blockIdx.x], 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) == gridDim.y - 1;
  __syncthreads();
  if (!last) return;
  const rsrc_t pr = make_rsrc(part, (uint32_t)(R * kCols * 4));
  for (int i = tid; i < p.T * (kCols / 4); i += 64 * W) {
    const int tok = i / (kCols / 4), at = 4 * (i % (kCols / 4)), o = o0 + at;
    if (o >= p.d_out) continue;
    f32x4_t s = {0.f, 0.f, 0.f, 0.f};
    constexpr int kAhead = 8;  // choices asked for together
    for (int j0 = 0; j0 < p.k; j0 += kAhead) {
      f32x4_t v[kAhead];
      uint8_t counts[kAhead];
#pragma unroll
      for (int j = 0; j < kAhead; ++j) {
        const int r = tok * p.k + min(j0 + j, p.k - 1);
        counts[j] = p.counted[r];
        v[j] = moe_collect(pr, (uint32_t)(r * kCols + at) * 4u);
      }
#pragma unroll
      for (int j = 0; j < kAhead; ++j)
        if (j0 + j < p.k && counts[j]) s += v[j];
    }
    char* dst = p.y + (int64_t)tok * p.ldy_bytes + (int64_t)o * E::kBytes;
    if constexpr (E::kBytes == 2) *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(s[0], s[1]), pack_bf16x2(s[2], s[3]));
    else *reinterpret_cast<f32x4_t*>(dst) = s;
  }
}

// LDS of a call: the rows of as many tokens as come together, up to kMoeLds,
// and the waves' sums.
inline int moe_lds_bytes(int T, int parts, int nt, int k_tiles, int sums) {
  const int at_once = 16 * nt / parts;
  const int64_t rows = (int64_t)(T < at_once ? T : at_once) * parts * ((int64_t)k_tiles * kW4K * 2 + 16);
  const int64_t some = rows > kMoeLds ? kMoeLds : rows;
  return (int)(some > sums ? some : sums);
}

template <typename E, int KIND, int SUB, int NT, int WB, int WK, int U>
hipError_t run_up(const MoeCall& c, hipStream_t stream) {
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
  a.counted = reinterpret_cast<uint8_t*>(c.ws + c.plan.counted);
  a.arrived = reinterpret_cast<uint32_t*>(c.ws + c.plan.arrived);
  a.groups = c.plan.down_groups;
  a.entries = c.plan.entries;
  a.lds_bytes = moe_lds_bytes(c.T, XFrag<E>::kParts, NT, a.k_tiles, moe_sum_bytes(WB * WK, 2, NT));
  static DynLdsLimit lim;
  const auto kernel = moe_up_kernel<E, KIND, SUB, NT, WB, WK, U>;
  const hipError_t e = ensure_dynamic_lds(lim, reinterpret_cast<const void*>(kernel), (size_t)a.lds_bytes);
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)((a.h_tiles * 8 + WB - 1) / WB), (unsigned)c.plan.entries + 1);
  hipLaunchKernelGGL(kernel, grid, dim3(64 * WB * WK), (size_t)a.lds_bytes, stream, a);
  return hipGetLastError();
}

template <typename E, int KIND, int SUB, int NT, int NB, int WK, int U>
hipError_t run_down(const MoeCall& c, hipStream_t stream) {
  MoeDownArgs a{};
  a.codes = reinterpret_cast<const char*>(c.down.codes);
  a.params = reinterpret_cast<const char*>(c.down.params);
  a.d_out = c.down.d_out;
  a.code_stride = w4_code_bytes(1, c.down.d_in, a.d_out);
  a.param_stride = w4_params_bytes(1, c.down.d_in, a.d_out, KIND, SUB);
  a.k_tiles = c.plan.h_tiles;
  a.row_tiles = w4_row_tiles(a.d_out);
  a.T = c.T;
  a.k = c.k;
  a.h = reinterpret_cast<const uint16_t*>(c.ws + c.plan.h);
  a.table = reinterpret_cast<const MoeEntry*>(c.ws + c.plan.table);
  a.part = reinterpret_cast<float*>(c.ws + c.plan.part);
  a.counted = reinterpret_cast<const uint8_t*>(c.ws + c.plan.counted);
  a.arrived = reinterpret_cast<uint32_t*>(c.ws + c.plan.arrived);
  a.y = reinterpret_cast<char*>(c.y);
  a.ldy_bytes = c.ldy * E::kBytes;
  constexpr int kWaves = moe_down_blocks(NT == 2) / NB * WK;
  a.lds_bytes = moe_lds_bytes(c.T, moe_h_parts(c.dtype), NT, a.k_tiles, moe_sum_bytes(kWaves, NB, NT));
  static DynLdsLimit lim;
  const auto kernel = moe_down_kernel<E, KIND, SUB, NT, NB, WK, U>;
  const hipError_t e = ensure_dynamic_lds(lim, reinterpret_cast<const void*>(kernel), (size_t)a.lds_bytes);
  if (e != hipSuccess) return e;
  const dim3 grid((unsigned)c.plan.down_groups, (unsigned)c.plan.entries);
  hipLaunchKernelGGL(kernel, grid, dim3(64 * kWaves), (size_t)a.lds_bytes, stream, a);
  return hipGetLastError();
}

template <typename E, int KIND, int SUB, int F>
hipError_t run_up_form(const MoeCall& c, hipStream_t stream) {
  constexpr MoeForm f = kMoeUpForms[F];
  return run_up<E, KIND, SUB, f.tiles, f.blocks, f.waves, f.ahead>(c, stream);
}
template <typename E, int KIND, int SUB>
hipError_t launch_up(const MoeCall& c, hipStream_t stream) {
  const int form = moe_up_form(c.plan, c.dtype, SUB);
  if (form == kMoeUpTwo) return run_up_form<E, KIND, SUB, kMoeUpTwo>(c, stream);
  if constexpr (XFrag<E>::kParts > 1) {
    if (form == kMoeUpOne) return run_up_form<E, KIND, SUB, kMoeUpOne>(c, stream);
  } else if constexpr (SUB == 1) {
    if (form == kMoeUpWide) return run_up_form<E, KIND, SUB, kMoeUpWide>(c, stream);
  }
  return run_up_form<E, KIND, SUB, kMoeUpPlain>(c, stream);
}
template <typename E, int KIND, int SUB, int F>
hipError_t run_down_form(const MoeCall& c, hipStream_t stream) {
  constexpr MoeForm f = kMoeDownForms[F];
  return run_down<E, KIND, SUB, f.tiles, f.blocks, f.waves, f.ahead>(c, stream);
}
template <typename E, int KIND, int SUB>
hipError_t launch_down(const MoeCall& c, hipStream_t stream) {
  switch (moe_down_form(c.plan)) {
    case kMoeDownTwo: return run_down_form<E, KIND, SUB, kMoeDownTwo>(c, stream);
    case kMoeDownDeep: return run_down_form<E, KIND, SUB, kMoeDownDeep>(c, stream);
    default: return run_down_form<E, KIND, SUB, kMoeDownPlain>(c, stream);
  }
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
