// The router: each token's k experts of E and their weights
// (lora_route in include/lora.h).
//
// One wave per token, expert e on lane e % 64, value e / 64, so that a row's
// logits are one coalesced load per 64 experts and stay in registers.  The
// choice runs on integer keys that order as the numbers do (0: cannot be
// chosen): without a bias, c orders as the logits themselves do, in both
// scores, so the keys are the float32 logits and no score is computed for the
// choice.  Where a group's score is the sum of two sigmoids, that sum is
// formed in float64 from its two largest logits, near one and two as its
// distance from there: sigmoids of more than 36.7 are 1.0 in float64 already.
// With a bias c itself is formed in float64, and scores that are equal there
// are ties (sigmoids above 36.7 with one bias, scores below 2^-53 of a bias).
// Each of the k steps takes the wave's largest key (four lane exchanges and a
// scalar maximum of the four rows) and its lowest index, and drops it; weights
// are computed at the end, by the k lanes that hold the chosen logits.
//
// What bounds it is the length of a wave's chain, not the bytes: one token of
// 64 experts 2.7 us (the shortest fill kernel: 1.3), 8192 tokens of 128 (4.7
// MB) 8.9, 250 tokens of 256 experts in groups with a bias 9.7, of which the
// float64 scores and eight choices of 64-bit keys are most.  So whatever is
// independent is asked for, exchanged and computed side by side: 10.9 us with
// the group scores one value after the other, 10.4 with a branch around each
// value's score and the bias read after it.
#include <float.h>
#include <math.h>

#include <type_traits>

#include "device_common.h"
#include "w4_kernels.h"

namespace lora {
namespace {

__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  const auto mx = [](uint32_t a, int b) { return a > (uint32_t)b ? a : (uint32_t)b; };
  v = mx(v, __builtin_amdgcn_mov_dpp((int)v, 0xB1, 0xF, 0xF, false));   // quad_perm 1,0,3,2
  v = mx(v, __builtin_amdgcn_mov_dpp((int)v, 0x4E, 0xF, 0xF, false));   // quad_perm 2,3,0,1
  v = mx(v, __builtin_amdgcn_mov_dpp((int)v, 0x141, 0xF, 0xF, false));  // row_half_mirror
  v = mx(v, __builtin_amdgcn_mov_dpp((int)v, 0x140, 0xF, 0xF, false));  // row_mirror
  uint32_t r = (uint32_t)__builtin_amdgcn_readlane((int)v, 0);
#pragma unroll
  for (int i = 1; i < 4; ++i) r = mx(r, __builtin_amdgcn_readlane((int)v, 16 * i));
  return r;
}

// Keys: unsigned integers in the order of the numbers, 0 below every number.
struct Key32 {
  uint32_t v;
  __device__ static Key32 none() { return {0u}; }
  __device__ static Key32 of(double) = delete;
  __device__ static Key32 of(float f) {
    const uint32_t u = __float_as_uint(f + 0.f);  // -0 as 0
    return {(u & 0x80000000u) ? ~u : u | 0x80000000u};
  }
  __device__ bool any() const { return v != 0u; }
  __device__ bool above(Key32 o) const { return v > o.v; }
  __device__ bool same(Key32 o) const { return v == o.v; }
  __device__ static Key32 wave_largest(Key32 k) { return {wave_max(k.v)}; }
  __device__ float value() const { return __uint_as_float((v & 0x80000000u) ? v & 0x7fffffffu : ~v); }
};
struct Key64 {
  uint64_t v;
  __device__ static Key64 none() { return {0ull}; }
  __device__ static Key64 of(double f) {
    const uint64_t u = (uint64_t)__double_as_longlong(f + 0.0);
    return {(u >> 63) ? ~u : u | (1ull << 63)};
  }
  __device__ bool any() const { return v != 0ull; }
  __device__ bool above(Key64 o) const { return v > o.v; }
  __device__ bool same(Key64 o) const { return v == o.v; }
  __device__ static Key64 wave_largest(Key64 k) {
    const uint32_t hi = wave_max((uint32_t)(k.v >> 32));
    const uint64_t at = __ballot((uint32_t)(k.v >> 32) == hi);
    // One lane has the largest upper half, nearly always.
    const uint32_t lo = (at & (at - 1)) == 0 ? (uint32_t)__builtin_amdgcn_readlane((int)k.v, __ffsll((unsigned long long)at) - 1)
                                             : wave_max((uint32_t)(k.v >> 32) == hi ? (uint32_t)k.v : 0u);
    return {((uint64_t)hi << 32) | lo};
  }
  __device__ double value() const {
    const uint64_t u = (v >> 63) ? v & ~(1ull << 63) : ~v;
    return __longlong_as_double((long long)u);
  }
};

__device__ __forceinline__ float wave_max_f(float v) {  // of numbers and -inf
  return Key32::wave_largest(Key32::of(v)).value();
}
__device__ __forceinline__ double wave_sum_f64(double v) {
#pragma unroll
  for (int d = 1; d < 64; d <<= 1) v += __shfl_xor(v, d);
  return v;
}

template <typename E>
__device__ __forceinline__ float logit_at(const void* p, int64_t i) {
  if constexpr (E::kBytes == 2) return bf16_lo(reinterpret_cast<const uint16_t*>(p)[i]);
  else return reinterpret_cast<const float*>(p)[i];
}

__device__ __forceinline__ uint32_t lane_xor(uint32_t v, int d) { return (uint32_t)__shfl_xor((int)v, d); }
__device__ __forceinline__ uint64_t lane_xor(uint64_t v, int d) {
  return ((uint64_t)lane_xor((uint32_t)(v >> 32), d) << 32) | lane_xor((uint32_t)v, d);
}
__device__ __forceinline__ uint32_t from_lane(uint32_t v, int l) { return (uint32_t)__shfl((int)v, l); }
__device__ __forceinline__ uint64_t from_lane(uint64_t v, int l) {
  return ((uint64_t)from_lane((uint32_t)(v >> 32), l) << 32) | from_lane((uint32_t)v, l);
}

// A group's score from its largest and second largest key, where it is the
// sum of two c (none, if there are no two).
__device__ __forceinline__ Key64 pair_score(Key64 a, Key64 b) {
  return a.any() && b.any() ? Key64::of(a.value() + b.value()) : Key64::none();
}
// The same from two logits, a >= b and c = sigmoid.  With p = sigmoid(-|a|) and
// q = sigmoid(-|b|), which hold their bits however small they are, the sum is
// p + q, 1 + (q - p) or 2 - (p + q).  Its key goes by itself below 1/2, by what
// it is from one up to 3/2, by what it lacks of two above.
__device__ __forceinline__ Key64 pair_score(Key32 a, Key32 b) {
  if (!a.any() || !b.any()) return Key64::none();
  const double x = (double)a.value(), y = (double)b.value();
  const double ex = exp(-fabs(x)), ey = exp(-fabs(y));
  const double p = ex / (1.0 + ex), q = ey / (1.0 + ey);
  const uint64_t low = 0x3fe0ull << 48, middle = 0x7fc0ull << 48;  // keys of [0, 1/2], of [-1/2, 1/2]
  const double s = p + q;
  if (s < 0.5 && (x <= 0.0 || y >= 0.0)) {
    const uint64_t at = (uint64_t)__double_as_longlong(s);
    return {x <= 0.0 ? 1 + at : 4 + low + middle + (low - at)};
  }
  const double from_one = x <= 0.0 ? s - 1.0 : (y >= 0.0 ? 1.0 - s : q - p);
  return {2 + low + (Key64::of(from_one).v - Key64::of(-0.5).v)};
}

// What the keys are: the logits; the logits, with groups by the sum of two
// scores; or the float64 c.
enum Keys { kLogits, kLogitPairs, kScores };
template <typename E, int NV, Keys KEYS>
__global__ __launch_bounds__(256) void route_kernel(const RouteArgs p) {
  constexpr bool WIDE = KEYS == kScores;
  typedef typename std::conditional<WIDE, Key64, Key32>::type Key;
  typedef typename std::conditional<KEYS == kLogits, Key32, Key64>::type GroupKey;
  const int lane = (int)threadIdx.x & 63;
  const int t = (int)blockIdx.x * 4 + ((int)threadIdx.x >> 6);
  if (t >= p.T) return;
  const int64_t row = (int64_t)t * p.ldl;
  constexpr float kNone = -INFINITY;
  float l[NV];  // logits; -inf: none (past E, NaN)
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int e = 64 * i + lane;
    const float v = e < p.E ? logit_at<E>(p.logits, row + e) : kNone;
    l[i] = v == v ? fminf(v, FLT_MAX) : kNone;
  }
  float bias[NV];  // asked for with the logits
  if constexpr (WIDE)
    if (p.bias)
#pragma unroll
      for (int i = 0; i < NV; ++i) bias[i] = p.bias[min(64 * i + lane, p.E - 1)];
  const bool softmax = p.score == LORA_ROUTE_SOFTMAX;
  // The softmax's maximum and sum over all experts, where the scores
  // themselves are needed (c with a bias; weights that keep their sum).
  float top = 0.f;
  double sum = 1.0;
  if (softmax && (WIDE || !p.renormalize)) {
    float m = kNone;
#pragma unroll
    for (int i = 0; i < NV; ++i) m = fmaxf(m, l[i]);
    top = wave_max_f(m);
    if (top == kNone) top = 0.f;
    double s = 0.0;
#pragma unroll
    for (int i = 0; i < NV; ++i) s += l[i] == kNone ? 0.0 : (WIDE ? exp((double)l[i] - (double)top) : (double)expf(l[i] - top));
    sum = wave_sum_f64(s);
  }

  Key key[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    if constexpr (WIDE) {
      // (The branch on the score is the same everywhere; none on l, so that
      // the values' long chains overlap.  exp of an infinity is one or 0.)
      double c = softmax ? exp((double)l[i] - (double)top) / sum : 1.0 / (1.0 + exp(-(double)l[i]));
      if (p.bias) c += bias[i] > FLT_MAX ? (double)FLT_MAX : (double)bias[i];  // a NaN stays one
      key[i] = l[i] != kNone && c == c && c != -INFINITY ? Key::of(c) : Key::none();
    } else {
      key[i] = l[i] != kNone ? Key::of(l[i]) : Key::none();
    }
  }

  if (p.groups > 1) {
    // Group g's score on lane g (groups <= 64): its largest key, or the sum
    // of its two largest c.
    const int n = p.E / p.groups;
    const bool pair = KEYS == kLogitPairs || (WIDE && !softmax && n > 1);
    Key first = Key::none(), second = Key::none();  // of the lane's group
    if (n <= 64 && (n & (n - 1)) == 0) {
      // A group is n neighbouring lanes of one value, and 64 / n groups are
      // reduced at once: (largest, second) pairs exchanged across n lanes.
      const int per = 64 / n;
      Key a[NV], b[NV];
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        a[i] = key[i];
        b[i] = Key::none();
      }
      for (int d = 1; d < n; d <<= 1) {
        Key oa[NV], ob[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          oa[i].v = lane_xor(a[i].v, d);
          if (pair) ob[i].v = lane_xor(b[i].v, d);
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const Key low = a[i].above(oa[i]) ? oa[i] : a[i];
          a[i] = a[i].above(oa[i]) ? a[i] : oa[i];
          if (pair) {
            b[i] = b[i].above(ob[i]) ? b[i] : ob[i];
            b[i] = b[i].above(low) ? b[i] : low;
          }
        }
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        Key fa, fb = Key::none();
        fa.v = from_lane(a[i].v, (lane % per) * n);
        if (pair) fb.v = from_lane(b[i].v, (lane % per) * n);
        if (lane / per == i) {
          first = fa;
          second = fb;
        }
      }
      if (lane >= p.groups) first = Key::none();
    } else {
      for (int g = 0; g < p.groups; ++g) {
        Key a = Key::none(), b = Key::none();
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const int e = 64 * i + lane;
          if (e >= g * n && e < (g + 1) * n) {
            if (key[i].above(a)) {
              b = a;
              a = key[i];
            } else if (key[i].above(b)) {
              b = key[i];
            }
          }
        }
        const Key top = Key::wave_largest(a);
        Key rest = Key::none();
        if (pair) {  // the largest is taken out on one lane
          const uint64_t at = __ballot(a.same(top));
          rest = Key::wave_largest(lane == __ffsll((unsigned long long)at) - 1 ? b : a);
        }
        if (lane == g) {
          first = top;
          second = rest;
        }
      }
    }
    GroupKey mine;
    if constexpr (KEYS == kLogits) mine = first;
    else mine = pair ? pair_score(first, second) : GroupKey{first.v};
    // A group's rank: those with a larger score, or the same and a lower index.
    int rank = 0;
    for (int g = 0; g < p.groups; ++g) {
      GroupKey o;
      if constexpr (sizeof(GroupKey) == 8) {
        o.v = ((uint64_t)(uint32_t)__builtin_amdgcn_readlane((int)(mine.v >> 32), g) << 32) |
              (uint32_t)__builtin_amdgcn_readlane((int)mine.v, g);
      } else {
        o.v = (uint32_t)__builtin_amdgcn_readlane((int)mine.v, g);
      }
      rank += o.above(mine) || (o.same(mine) && g < lane) ? 1 : 0;
    }
    const uint64_t keep = __ballot(lane < p.groups && rank < p.top_groups);
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int g = (64 * i + lane) / n;
      if (g >= p.groups || !((keep >> g) & 1)) key[i] = Key::none();
    }
  }

  // ---- the k largest, descending; lane j keeps the j-th
  int id = -1;
  float chosen = kNone;
  for (int j = 0; j < p.k; ++j) {
    Key best = key[0];
    int bi = 0;
#pragma unroll
    for (int i = 1; i < NV; ++i)
      if (key[i].above(best)) {
        best = key[i];
        bi = i;
      }
    const Key m = Key::wave_largest(best);
    if (!m.any()) break;  // no expert left (the same in every lane)
    const uint64_t at = __ballot(best.same(m));
    int win = __ffsll((unsigned long long)at) - 1;
    if (__popcll(at) > 1) {  // equal: the lowest index, value first
      const uint32_t far = best.same(m) ? (uint32_t)(64 * bi + lane) : 0xffffffffu;
      win = (int)(~wave_max(~far) & 63u);
    }
    float bl = l[0];
#pragma unroll
    for (int i = 1; i < NV; ++i) bl = bi == i ? l[i] : bl;
    const int we = __builtin_amdgcn_readlane(64 * bi + lane, win);
    const float wl = __int_as_float(__builtin_amdgcn_readlane(__float_as_int(bl), win));
    if (lane == j) {
      id = we;
      chosen = wl;
    }
#pragma unroll
    for (int i = 0; i < NV; ++i)
      if (64 * i + lane == we) key[i] = Key::none();
  }

  // ---- weights.  Renormalized ones are formed relative to the largest
  // chosen score, so that small scores do not vanish before the division.
  const bool have = id >= 0;
  double w = 0.0;
  if (softmax) {
    const float ref = p.renormalize ? wave_max_f(chosen) : top;
    if (have) w = WIDE ? exp((double)chosen - (double)ref) : (double)expf(chosen - ref);
    if (!p.renormalize) w /= sum;
  } else {
    const double ref = p.renormalize ? fmin((double)wave_max_f(chosen), 0.0) : 0.0;
    const double c = (double)chosen;
    if (have) w = c > 0.0 ? 1.0 / (1.0 + exp(-c)) : exp(c - ref) / (1.0 + exp(c));
  }
  if (p.renormalize) {
    const double s = wave_sum_f64(w);
    w = have ? w / s : 0.0;
  }
  if (lane < p.k) {
    const int64_t at = (int64_t)t * p.k + lane;
    p.ids[at] = id;
    // Without an expert w may be 0 / 0 (a softmax over none), or meet an
    // infinite scale: the weight is 0 whatever it is.
    p.weights[at] = have ? (float)(w * (double)p.scale) : 0.f;
  }
}

template <typename E, Keys KEYS>
hipError_t launch_sized(const RouteArgs& a, hipStream_t stream) {
  const dim3 grid((unsigned)((a.T + 3) / 4)), block(256);
  if (a.E <= 64) hipLaunchKernelGGL((route_kernel<E, 1, KEYS>), grid, block, 0, stream, a);
  else if (a.E <= 128) hipLaunchKernelGGL((route_kernel<E, 2, KEYS>), grid, block, 0, stream, a);
  else if (a.E <= 256) hipLaunchKernelGGL((route_kernel<E, 4, KEYS>), grid, block, 0, stream, a);
  else if (a.E <= 512) hipLaunchKernelGGL((route_kernel<E, 8, KEYS>), grid, block, 0, stream, a);
  else hipLaunchKernelGGL((route_kernel<E, 16, KEYS>), grid, block, 0, stream, a);
  return hipGetLastError();
}

}  // namespace

template <typename E>
static hipError_t launch_type(const RouteArgs& a, hipStream_t stream) {
  if (a.bias != nullptr) return launch_sized<E, kScores>(a, stream);
  if (a.groups > 1 && a.groups < a.E && a.score == LORA_ROUTE_SIGMOID) return launch_sized<E, kLogitPairs>(a, stream);
  return launch_sized<E, kLogits>(a, stream);
}

hipError_t launch_route(const RouteArgs& a, int dtype, hipStream_t stream) {
  return dtype == LORA_DTYPE_BF16 ? launch_type<BF16>(a, stream) : launch_type<F32>(a, stream);
}

}  // namespace lora
