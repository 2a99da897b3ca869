// 4-bit base products for few rows (the decode step), and for float32 rows:
//
//   y[r, o] = sum_g s[o, g] sum_{k in g} (q[o, k] - z[o, g]) x[r, k]
//
// with one matrix, with the matrix that ids[r] names, or summed over a
// token's k rows with weights.
//
// What bounds it is the stream of codes.  A workgroup owns 16 RT outputs of
// 16 NT rows, over all inputs or a split of them.  Its rows of x are copied
// into LDS, all inputs at once or a chunk at a time, so that a wave's loads
// in flight are codes alone: the waves take the 128-input tiles of the codes
// in turn (a tile is 1 KiB, one load per lane; the tiles of 16 outputs are
// consecutive in memory), U tiles x RT ahead, across chunks.  Their float32
// sums meet in LDS at the end and are added in wave order, the same order at
// every call; splits leave float32 rows that a last kernel adds in order.
// (With x loaded from memory beside the codes, a lane's four 16-byte pieces
// of x per tile took four times the registers of the codes and as many passes
// through the load path: 19.0 us for one token, 3584 -> 18944, against 9.3.)
//
// Measured (kernel times, three sets of weights in turn): one token 3584 ->
// 18944 9.3 to 9.7 us (35.6 MB, 3.7 TB/s); 23 rows 18944 -> 3584 in groups of
// 64 14.6 (2.6) and 3.9 for the splits' sum; one token's eight experts of 64,
// 2048 -> 2816, 8.1 (23.8 MB, 2.9), eight tokens' 28.7 (about 120 MB, 4.2);
// 180 rows of 32 experts 1408 -> 2048 in groups of 32 18.2 (2.9): with few
// bytes the launch, the copy of x and the last sums show, with fine groups the
// instructions per code.  The codes' loads go through the caches (past them,
// as data read once, one token took 10.4, the 23 rows 16.2).  More waves in a
// workgroup rather than more tiles in a wave's flight: one token 9.3 us with
// 8 waves of four tiles, 10.4 with 4.
//
// Products run on the matrix cores with x on the row side and the codes on
// the column side, 16 rows x 16 outputs.  A code enters as the bf16 number
// 32 + q, which costs one "and-or" per two codes; the excess is taken out
// with the sum of x over the group,
//
//   sum (q - z) x = sum (32 + q) x - (32 + z) sum x,
//
// where sum x comes from one more product against ones, in the same lane
// layout, and its multiple is the accumulator that the group's products
// start from.  All products are exact in float32 and only the sums round;
// 32 is a small base (16 is the smallest that bf16 holds with a step of one
// code, 32 lets the prefill kernel unpack the same layout with fewer shifts),
// which keeps the cancelled part small (a few times the result).  Float32
// rows, which take three products per step anyway (three bf16 parts), are
// multiplied with q - z itself: more work per code, no cancellation.
#pragma once
#include "host_util.h"
#include "w4_kernels.h"
#include "w4_ops.h"

namespace lora {
namespace {

struct W4RowsArgs {
  const char* codes;
  const char* params;
  int64_t code_stride, param_stride;  // bytes per matrix
  int n, k_tiles, row_tiles, d_in, d_out;
  const char* x;
  int64_t ldx_bytes;
  int x_div;
  char* y;  // rows of the output type, or float32 rows [splits][R] (f32_out)
  int64_t ldy_bytes;
  int R, k;
  const int32_t* ids;    // nullptr: matrix 0
  const float* weights;  // kSum
  int by_row;            // kListed: blockIdx.y is a row (the first row of its matrix works), else a matrix
  int f32_out;
  int row_cap;           // rows held in LDS at a time
  int per_split;         // tiles of inputs per split (blockIdx.z)
};

constexpr int kListMax = 4096;  // rows of a routed call that are listed at a time
constexpr int kPad = 17;        // LDS row stride of a 16 x 16 block of sums

template <typename E>
__device__ __forceinline__ void store_out(char* row, int o, float v, int f32_out) {
  if (E::kBytes == 4 || f32_out) reinterpret_cast<float*>(row)[o] = v;
  else reinterpret_cast<uint16_t*>(row)[o] = (uint16_t)f32_to_bf16(v);
}

// The rows of [win, win + kListMax) whose id is e (or, `none`, outside
// [0, n)), ascending, into `list`; returns their number.  Per chunk of 64 W
// rows, each wave counts its 64 by ballot and the waves' counts are added up
// in order.
template <int W>
__device__ __forceinline__ int rows_of(const W4RowsArgs& p, int e, bool none, int win, uint16_t* list, int* s_cnt) {
  const int tid = (int)threadIdx.x, lane = tid & 63, w = tid >> 6;
  const int end = min(p.R, win + kListMax);
  int cnt = 0;
  for (int r0 = win; r0 < end; r0 += 64 * W) {
    const int r = r0 + tid;
    const int id = r < end ? p.ids[r] : 0;
    const bool hit = r < end && (none ? (unsigned)id >= (unsigned)p.n : id == e);
    const uint64_t mask = __ballot(hit);
    if (lane == 0) s_cnt[w] = __popcll(mask);
    __syncthreads();
    int before = cnt, total = cnt;
#pragma unroll
    for (int i = 0; i < W; ++i) {
      before += i < w ? s_cnt[i] : 0;
      total += s_cnt[i];
    }
    if (hit) list[before + __popcll(mask & lanemask_lt())] = (uint16_t)(r - win);
    cnt = total;
    __syncthreads();
  }
  return __builtin_amdgcn_readfirstlane(cnt);  // the same in every lane: the loops over rows stay scalar
}

// Empty sums: outputs [o0, o0 + width) of `cnt` listed rows.
template <typename E>
__device__ __forceinline__ void zero_rows(const W4RowsArgs& p, int win, const uint16_t* list, int cnt, int o0, int width) {
  for (int i = (int)threadIdx.x; i < cnt * width; i += (int)blockDim.x) {
    const int o = o0 + i % width;
    if (o < p.d_out) store_out<E>(p.y + (int64_t)(win + list[i / width]) * p.ldy_bytes, o, 0.f, p.f32_out);
  }
}

// An LDS barrier that leaves loads from memory in flight (__syncthreads()
// waits for them: its fence).
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}
// Wait until at most N of the wave's loads are in flight (they end in order).
template <int N>
__device__ __forceinline__ void wait_loads() {
  static_assert(N >= 0 && N < 64, "vmcnt range");
  asm volatile("" ::: "memory");
  __builtin_amdgcn_s_waitcnt((N & 15) | ((N >> 4) << 14) | 0x0f70);
  asm volatile("" ::: "memory");
}

// What the rows of a workgroup are: a run of rows (one matrix); the rows whose
// id is its matrix; or one token's k rows, each with its own matrix, summed.
enum Mode { kRun, kListed, kSum };

// x in LDS.  Not CHUNKED: all of the rows' inputs.  CHUNKED: kChunk tiles of
// 16 NT rows; of 16 bf16 rows two such buffers, filled in turn.  More rows
// have one, which every chunk waits for with the codes in flight: of 64 rows a
// second costs the workgroups that would hide the loads (3584 -> 3584 13.7 us
// with two, 10.7 with one); of 32 it was not measured.
constexpr int kChunk = 4;
template <typename E, int NT, bool CHUNKED>
constexpr int x_buffers() {
  return CHUNKED && XFrag<E>::kParts == 1 && NT == 1 ? 2 : 1;
}

// At least two waves per SIMD: with up to 256 registers per lane the matrix
// instructions keep their results in ordinary registers, which the vector
// instructions around them read without a move.
template <typename E, int KIND, int SUB, int RT, int NT, int U, int W, int MODE, bool CHUNKED>
__global__ __launch_bounds__(64 * W) __attribute__((amdgpu_waves_per_eu(2)))
void w4_rows_kernel(const W4RowsArgs p) {
  constexpr int kParts = XFrag<E>::kParts;
  constexpr int kSteps = 4 / SUB;  // matrix-core steps per scale
  constexpr bool kExact = kParts > 1, kDma = kParts == 1;
  constexpr int kBatch = 4;  // float32: 32-byte pieces of x per lane and pass
  constexpr bool kSumUp = MODE == kSum, kList = MODE == kListed;
  static_assert(!CHUNKED || (kChunk % (U * W) == 0 && !kSumUp), "a wave's turns run on across chunks");
  // The loads of the codes in flight, per wave.
  constexpr int kCodeLoads = U * RT * (1 + (W4Params<KIND, SUB>::kBytes > 16 ? 2 : 1));
  // x, then (once it has been read) the waves' sums [W][RT][NT][16 * kPad].
  extern __shared__ __align__(16) char lds[];
  __shared__ uint16_t list[kList ? kListMax : 1];
  __shared__ int s_cnt[W];
  const int w = __builtin_amdgcn_readfirstlane((int)threadIdx.x >> 6);  // uniform: the codes' addresses stay scalar
  const int rt0 = (int)blockIdx.x * RT;
  // kSum: every tile of the token's rows, one row after the other
  const int t_begin = kSumUp ? 0 : (int)blockIdx.z * p.per_split;
  const int t_end = kSumUp ? p.k * p.k_tiles : min(p.k_tiles, t_begin + p.per_split);
  const int chunk = CHUNKED ? kChunk : p.k_tiles;
  const int plane = chunk * kW4K * 2, xrow_bytes = kParts * plane + 16;
  const int last_piece = p.d_in - 8;
  const bool ragged = p.d_in % kW4K != 0;
  int e = 0, few_cnt = -1;
  bool none = false;
  if constexpr (kList) {
    if (p.by_row && p.R <= 64) {
      // One id per lane: each wave finds its matrix and the rows that have it
      // by itself (all waves write the same list).
      const int lane = (int)threadIdx.x & 63;
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
  const char *code0[RT], *par0[RT];  // first tile of each output block
#pragma unroll
  for (int a = 0; a < RT; ++a) {
    const int64_t t = (int64_t)min(rt0 + a, p.row_tiles - 1) * p.k_tiles;
    code0[a] = p.codes + (kSumUp ? 0 : e * p.code_stride) + t * kW4TileBytes;
    par0[a] = p.params + (kSumUp ? 0 : e * p.param_stride) + t * kW4Rows * W4Params<KIND, SUB>::kBytes;
  }

  // m rows from base (or from list[m0]): x into LDS, the products, y.
  auto block = [&](int base, int m0, int m) {
    // A value the compiler cannot take out of the loop over a matrix's rows:
    // what depends on the lane is formed again for each block, and does not
    // hold registers across it.
    int tid = (int)threadIdx.x;
    if constexpr (kList) asm volatile("" : "+v"(tid));
    const int lane = tid & 63, col = lane & 15, h = lane >> 4;
    const uint32_t lane16 = 16 * lane, lane_par = col * W4Params<KIND, SUB>::kBytes;
    const int x_rows = kSumUp ? (p.x_div == 1 ? p.k : 1) : m;
    auto x_row = [&](int i) {  // uniform
      uint32_t r = base + i;
      if constexpr (kList) r = base + __builtin_amdgcn_readfirstlane((int)list[m0 + i]);
      if constexpr (MODE != kRun) r /= (uint32_t)p.x_div;
      return p.x + (int64_t)r * p.ldx_bytes;
    };
    // ---- x into LDS, bf16: loads that write LDS directly, 64 pieces of 8
    // values (4 tiles) of one row each.  Pieces past d_in repeat the last
    // one, until clear_pads.
    auto dma_row = [&](char* dst, const char* src, int k0) {
      const int k = min(k0 + 8 * lane, last_piece);
      __builtin_amdgcn_global_load_lds((const __attribute__((address_space(1))) void*)(src + (uint32_t)(2 * k)),
                                       (__attribute__((address_space(3))) void*)dst, 16, 0, 0);
    };
    // One chunk: the same number of loads in every wave and call, so that the
    // compiler can count past them.  Rows past m repeat the last.
    auto dma_chunk = [&](char* dst, int c0) {
#pragma unroll
      for (int i = 0; i < 16 * NT / W; ++i)
        dma_row(dst + (w + i * W) * xrow_bytes, x_row(min(w + i * W, m - 1)), c0 * kW4K);
    };
    auto dma_rows = [&](char* dst) {  // all inputs; the waves take the loads in turn
      const int per_row = (p.k_tiles + 3) >> 2;
      for (int row = 0, f = w; row < x_rows; ++row, f -= per_row)
        for (; f < per_row; f += W) {
          // The last load may cover tiles past the row's: its lanes stay out.
          if (f * 64 + lane < 16 * p.k_tiles) dma_row(dst + row * xrow_bytes + f * 1024, x_row(row), f * 4 * kW4K);
        }
    };
    // ---- x into LDS, float32: through registers, in its three parts.
    XFrag<E> hold[kBatch];
    auto part_rows = [&](int c0) {
      const int pieces = chunk * (kW4K / 8), per_row = (pieces + 63) >> 6, total = x_rows * per_row;
      for (int f0 = w; f0 < total; f0 += W * kBatch) {
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int f = min(f0 + i * W, total - 1), row = (int)((uint32_t)f / (uint32_t)per_row);
          const int k = c0 * kW4K + 8 * (64 * (f - row * per_row) + lane);
          hold[i].load(x_row(row) + (uint32_t)(min(k, last_piece) * E::kBytes));
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int f = min(f0 + i * W, total - 1), row = (int)((uint32_t)f / (uint32_t)per_row);
          const int at = 64 * (f - row * per_row) + lane;
          uint4 parts[kParts];
          hold[i].parts(parts);
          if (at < pieces)
#pragma unroll
            for (int q = 0; q < kParts; ++q) *reinterpret_cast<uint4*>(lds + row * xrow_bytes + q * plane + 16 * at) = parts[q];
        }
      }
    };

    // The last tile's pieces past d_in, at tile `kt` of x's rows in LDS, become
    // zeros once x is there: whatever their codes and scales, they then add
    // nothing, to sums near the largest float32 either.  (A choice of address
    // in the loads made 23 rows 18944 -> 3584 21.4 us a call, against 17.2; here
    // only a d_in that ends inside a tile pays, one barrier.)
    auto clear_pads = [&](char* dst, int kt) {
      int id = (int)threadIdx.x;
      asm volatile("" : "+v"(id));  // nothing of this is formed before, to hold registers
      const int pads = (kW4K - p.d_in % kW4K) / 2;  // dwords
#pragma unroll 1
      for (int row = id >> 6; row < x_rows; row += W)
#pragma unroll
        for (int q = 0; q < kParts; ++q)
          if ((id & 63) < pads)
            reinterpret_cast<uint32_t*>(dst + row * xrow_bytes + q * plane + (kt + 1) * kW4K * 2)[-1 - (id & 63)] = 0u;
      lds_barrier();
    };

    // ---- codes: U tiles of each output block in flight per wave, taken in
    // turn by the waves; loads past the last tile read it again (an
    // unconditional load keeps the waits of the earlier ones exact).
    uint4 code[U][RT];
    W4Params<KIND, SUB> par[U][RT];
    int cur_j = -1, cur_id = 0;
    float cur_w = 0.f;
    float slot_w[U];
    int slot_x[U];  // kSum: LDS offset of the tile's x, -1: a row without a matrix
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
      }
#pragma unroll
      for (int a = 0; a < RT; ++a) {
        code[u][a] = ld16(code0[a] + (mat * p.code_stride + (int64_t)kt * kW4TileBytes) + lane16);
        par[u][a].load(par0[a] + (mat * p.param_stride + (int64_t)kt * (kW4Rows * W4Params<KIND, SUB>::kBytes)) + lane_par);
      }
    };
    if constexpr (kDma) {
      if constexpr (CHUNKED) dma_chunk(lds, t_begin);
      else dma_rows(lds);
      asm volatile("" ::: "memory");  // the codes are asked for after x (wait_loads counts them)
    }
#pragma unroll
    for (int u = 0; u < U; ++u) fetch(u, min(t_begin + w + u * W, t_end - 1));

    f32x4_t acc[RT][NT];
#pragma unroll
    for (int a = 0; a < RT; ++a)
#pragma unroll
      for (int t = 0; t < NT; ++t) acc[a][t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
    // Lanes of rows past m read the last row: their results are not used.
    uint32_t xl[NT];
#pragma unroll
    for (int t = 0; t < NT; ++t) xl[t] = (kSumUp ? 0 : min(16 * t + col, m - 1) * xrow_bytes) + 16 * h;
    auto compute = [&](const char* x, int u) {
#pragma unroll
      for (int s = 0; s < SUB; ++s) {
        uint4 xp[NT][kSteps][kParts];
        f32x4_t xsum[NT];
#pragma unroll
        for (int t = 0; t < NT; ++t) {
          xsum[t] = f32x4_t{0.f, 0.f, 0.f, 0.f};
#pragma unroll
          for (int j = 0; j < kSteps; ++j) {
#pragma unroll
            for (int q = 0; q < kParts; ++q) xp[t][j][q] = ld16(x + xl[t] + q * plane + 64 * (s * kSteps + j));
            if constexpr (!kExact) xsum[t] = mfma_bf16_16x16x32(xp[t][j][0], ones, xsum[t]);
          }
        }
#pragma unroll
        for (int a = 0; a < RT; ++a) {
          const uint32_t cw[4] = {code[u][a].x, code[u][a].y, code[u][a].z, code[u][a].w};
          const float sc = par[u][a].scale(s);
          const float z32 = par[u][a].zero32(s);
          uint4 b[kSteps];
#pragma unroll
          for (int j = 0; j < kSteps; ++j)
            b[j] = kExact ? w4_expand_exact(cw[s * kSteps + j], mask, magic, z32) : w4_expand(cw[s * kSteps + j], mask, magic);
#pragma unroll
          for (int t = 0; t < NT; ++t) {
            f32x4_t c;
#pragma unroll
            for (int v = 0; v < 4; ++v) c[v] = kExact ? 0.f : -z32 * xsum[t][v];
#pragma unroll
            for (int j = 0; j < kSteps; ++j)
#pragma unroll
              for (int q = 0; q < kParts; ++q) c = mfma_bf16_16x16x32(xp[t][j][q], b[j], c);
#pragma unroll
            for (int v = 0; v < 4; ++v)
              // The weight multiplies what the scale gave: their own product
              // need not be a number that float32 holds.
              acc[a][t][v] = kSumUp ? fmaf(slot_w[u], sc * c[v], acc[a][t][v]) : fmaf(sc, c[v], acc[a][t][v]);
          }
        }
      }
    };
    // The tiles [c0, c1) of x at `rd`, while the next chunk's x goes to `wr`
    // (another buffer, which restrict tells the compiler: the reads need not
    // wait for the loads in flight).
    auto run = [&](const char* __restrict__ rd, char* __restrict__ wr, int c0, int c1, bool more) {
      if constexpr (CHUNKED && kDma && x_buffers<E, NT, CHUNKED>() > 1)
        if (more) {
          dma_chunk(wr, c1);
          asm volatile("" ::: "memory");
        }
      for (int i0 = c0 + w; i0 < c1; i0 += U * W) {
#pragma unroll
        for (int u = 0; u < U; ++u) {
          const int i = i0 + u * W;
          if constexpr (kSumUp) {
            if (i < c1 && slot_x[u] >= 0) compute(rd + slot_x[u], u);
          } else {
            if (i < c1) compute(rd + (i - c0) * kW4K * 2, u);
          }
          if (i0 + U * W < t_end) fetch(u, min(i + U * W, t_end - 1));
        }
      }
    };
    if constexpr (CHUNKED) {
      const int buf = x_buffers<E, NT, true>() > 1 ? 16 * NT * xrow_bytes : 0;
      int at = 0;
      for (int c0 = t_begin; c0 < t_end; c0 += kChunk) {
        if constexpr (kDma) {
          // This chunk's x is there once only the codes asked for after it
          // are in flight; where a wave has asked for fewer, once none is.
          if (buf == 0 && c0 > t_begin) {
            lds_barrier();  // every wave has read the last chunk
            dma_chunk(lds, c0);
            wait_loads<0>();
          } else if (c0 + w < t_end) wait_loads<kCodeLoads>();
          else wait_loads<0>();
        } else {
          if (c0 > t_begin) lds_barrier();  // every wave has read the last chunk
          part_rows(c0);
        }
        lds_barrier();
        if (ragged && c0 + kChunk >= p.k_tiles) clear_pads(lds + at, p.k_tiles - 1 - c0);
        run(lds + at, lds + (buf - at), c0, min(t_end, c0 + kChunk), c0 + kChunk < t_end);
        at = buf - at;
      }
    } else {
      if constexpr (kDma) wait_loads<kCodeLoads>();
      else part_rows(0);
      lds_barrier();
      if (ragged) clear_pads(lds, p.k_tiles - 1);
      run(lds, lds, t_begin, t_end, false);
    }

    // ---- the waves' sums, in wave order
    float* red = reinterpret_cast<float*>(lds);
    lds_barrier();  // x has been read
#pragma unroll
    for (int a = 0; a < RT; ++a)
#pragma unroll
      for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int v = 0; v < 4; ++v)
          if (16 * t + 4 * h + v < m) red[((w * RT + a) * NT + t) * 16 * kPad + (4 * h + v) * kPad + col] = acc[a][t][v];
    __syncthreads();
    char* y = p.y + (kSumUp ? 0 : (int64_t)blockIdx.z * p.R * p.ldy_bytes);
    for (int i = tid; i < 16 * m * RT; i += 64 * W) {
      const int o16 = i & 15, a = (i >> 4) % RT, rw = (i >> 4) / RT;
      const int o = 16 * (rt0 + a) + o16;
      if (o >= p.d_out) continue;
      float v = 0.f;
#pragma unroll
      for (int ww = 0; ww < W; ++ww) v += red[((ww * RT + a) * NT + (rw >> 4)) * 16 * kPad + (rw & 15) * kPad + o16];
      const int r = kSumUp ? (int)blockIdx.y : base + (kList ? (int)list[m0 + rw] : rw);
      store_out<E>(y + (int64_t)r * p.ldy_bytes, o, v, p.f32_out);
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
        cnt = rows_of<W>(p, e, none, win, list, s_cnt);
        if (p.by_row && (int)list[0] != (int)blockIdx.y) return;
      }
      if (none) {
        if (blockIdx.z == 0 && !p.f32_out) zero_rows<E>(p, win, list, cnt, 16 * rt0, 16 * RT);
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

template <typename E, int KIND, int SUB, int RT, int NT, int U, int W, int MODE, bool CHUNKED>
hipError_t launch_one(const W4RowsArgs& a, unsigned gy, hipStream_t stream) {
  const unsigned splits = MODE == kSum ? 1u : (unsigned)((a.k_tiles + a.per_split - 1) / a.per_split);
  const dim3 grid((unsigned)((a.row_tiles + RT - 1) / RT), gy, splits);
  const size_t row = (size_t)XFrag<E>::kParts * (CHUNKED ? kChunk : a.k_tiles) * kW4K * 2 + 16;
  const size_t x = CHUNKED ? x_buffers<E, NT, true>() * 16 * NT * row : a.row_cap * row;
  const size_t sums = (size_t)W * RT * NT * 16 * kPad * 4;
  const size_t lds = x > sums ? x : sums;
  static DynLdsLimit lim;
  const void* fn = reinterpret_cast<const void*>(w4_rows_kernel<E, KIND, SUB, RT, NT, U, W, MODE, CHUNKED>);
  const hipError_t e = ensure_dynamic_lds(lim, fn, lds);
  if (e != hipSuccess) return e;
  hipLaunchKernelGGL((w4_rows_kernel<E, KIND, SUB, RT, NT, U, W, MODE, CHUNKED>), grid, dim3(64 * W), lds, stream, a);
  return hipGetLastError();
}

template <typename E, int KIND, int SUB, int MODE>
hipError_t launch_mode(const W4RowsArgs& a, const W4Plan& pl, unsigned gy, hipStream_t stream) {
  if constexpr (MODE == kSum) {
    return launch_one<E, KIND, SUB, 1, 1, 4, 16, MODE, false>(a, gy, stream);
  } else {
    if constexpr (E::kBytes == 2) {
      if (pl.nt == 4) return launch_one<E, KIND, SUB, 2, 4, 1, 4, MODE, true>(a, gy, stream);
    }
    if (pl.nt == 2) return launch_one<E, KIND, SUB, 4, 2, 1, 4, MODE, true>(a, gy, stream);
    if (pl.chunked) return launch_one<E, KIND, SUB, 4, 1, 1, 4, MODE, true>(a, gy, stream);
    switch (pl.rt) {
      case 0: return launch_one<E, KIND, SUB, 1, 1, 2, 8, MODE, false>(a, gy, stream);
      case 1: return launch_one<E, KIND, SUB, 1, 1, 4, 8, MODE, false>(a, gy, stream);
      case 2: return launch_one<E, KIND, SUB, 2, 1, 2, 4, MODE, false>(a, gy, stream);
      default: return launch_one<E, KIND, SUB, 4, 1, 1, 4, MODE, false>(a, gy, stream);
    }
  }
}

template <typename E, int KIND, int SUB>
hipError_t launch_shape(const W4RowsArgs& a, const W4Plan& pl, unsigned gy, hipStream_t stream) {
  if (a.weights != nullptr) return launch_mode<E, KIND, SUB, kSum>(a, pl, gy, stream);
  if (a.ids != nullptr) return launch_mode<E, KIND, SUB, kListed>(a, pl, gy, stream);
  return launch_mode<E, KIND, SUB, kRun>(a, pl, gy, stream);
}

template <typename E>
hipError_t launch_kind(const W4RowsArgs& a, const W4Plan& pl, int kind, int sub, unsigned gy, hipStream_t st) {
  switch (kind * 8 + sub) {
    case kW4Bf16 * 8 + 1: return launch_shape<E, kW4Bf16, 1>(a, pl, gy, st);
    case kW4Bf16 * 8 + 2: return launch_shape<E, kW4Bf16, 2>(a, pl, gy, st);
    case kW4Bf16 * 8 + 4: return launch_shape<E, kW4Bf16, 4>(a, pl, gy, st);
    case kW4Bf16Zero * 8 + 1: return launch_shape<E, kW4Bf16Zero, 1>(a, pl, gy, st);
    case kW4Bf16Zero * 8 + 2: return launch_shape<E, kW4Bf16Zero, 2>(a, pl, gy, st);
    case kW4Bf16Zero * 8 + 4: return launch_shape<E, kW4Bf16Zero, 4>(a, pl, gy, st);
    case kW4F32 * 8 + 1: return launch_shape<E, kW4F32, 1>(a, pl, gy, st);
    case kW4F32 * 8 + 2: return launch_shape<E, kW4F32, 2>(a, pl, gy, st);
    default: return launch_shape<E, kW4F32, 4>(a, pl, gy, st);
  }
}

template <typename E>
hipError_t launch_rows_of(const W4Call& c, hipStream_t stream) {
  const lora_w4_store& s = c.s;
  const W4Plan& pl = c.plan;
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
  a.weights = pl.sum_in_kernel ? c.weights : nullptr;
  a.row_cap = pl.row_cap;
  a.per_split = pl.per_split;
  if (pl.keep_parts) {
    a.y = c.ws + pl.part;
    a.ldy_bytes = (int64_t)s.d_out * 4;
    a.f32_out = 1;
  }
  unsigned gy;
  if (pl.sum_in_kernel) {
    gy = (unsigned)(c.R / c.k);
  } else if (c.ids != nullptr) {
    a.by_row = c.R <= s.n && c.R <= kListMax;
    gy = a.by_row ? (unsigned)c.R : (unsigned)s.n + 1;
  } else {
    gy = (unsigned)((c.R + a.row_cap - 1) / a.row_cap);
  }
  return launch_kind<E>(a, pl, kind, sub, gy, stream);
}

}  // namespace
}  // namespace lora
