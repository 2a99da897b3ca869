// Lays a checkpoint's 4-bit codes, scales and zero points out for the 4-bit
// base products (the layout: w4.h).  Run once when a layer is loaded: it
// moves bits and computes nothing but 32 + z, so every code, scale and zero
// point is held exactly.
#include "device_common.h"
#include "w4_kernels.h"

namespace lora {
namespace {

struct W4PackArgs {
  const uint8_t* q;      // [n][d_out][d_in / 2], input 2 i in the low four bits of byte i
  const void* scales;    // [n][d_out][groups], bf16 or float32
  const uint8_t* zeros;  // [n][d_out][groups] (0..15), or nullptr: 8
  int d_in, d_out, group, groups, sub, kind, k_tiles;
  int64_t tiles;  // n * row tiles * k_tiles
  int row_tiles;
  char* codes;
  char* params;
};

// One wave per tile; lane l fills its 16 bytes.  Inputs past d_in get the
// code of their zero point (a product of exactly zero with any finite x),
// outputs past d_out code 0 with scale 0.
__global__ __launch_bounds__(256) void w4_pack_kernel(const W4PackArgs p) {
  const int64_t tile = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * 4 + (threadIdx.x >> 6);
  if (tile >= p.tiles) return;
  const int lane = threadIdx.x & 63, row = lane & 15, h = lane >> 4;
  const int kt = (int)(tile % p.k_tiles);
  const int64_t t2 = tile / p.k_tiles;
  const int rt = (int)(t2 % p.row_tiles);
  const int64_t e = t2 / p.row_tiles;
  const int o = kW4Rows * rt + row;
  const int64_t orow = e * p.d_out + (o < p.d_out ? o : 0);
  const int gran = kW4K / p.sub;

  uint32_t w[4];
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const int k = kW4K * kt + 32 * j + 8 * h;
    uint32_t v = 0, out = 0;
    if (o < p.d_out) {
      if (k < p.d_in) {  // d_in is a multiple of 8: four whole bytes
        v = *reinterpret_cast<const uint32_t*>(p.q + orow * (p.d_in / 2) + k / 2);
      } else {
        // A chunk past the end: its group's zero point (the last group's, where its own does not exist).
        int g = k / p.group;
        g = g < p.groups ? g : p.groups - 1;
        const uint32_t z = p.zeros ? p.zeros[orow * p.groups + g] & 15u : 8u;
        v = z * 0x11111111u;
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      out |= ((v >> (8 * i)) & 15u) << (4 * i);
      out |= ((v >> (8 * i + 4)) & 15u) << (4 * i + 16);
    }
    w[j] = (out << 2) | (out >> 30);
  }
  st16(p.codes + tile * kW4TileBytes + 16 * lane, make_uint4(w[0], w[1], w[2], w[3]));

  // Scales: lanes 0..16 sub - 1, one value each.
  if (lane < kW4Rows * p.sub) {
    const int prow = lane / p.sub, s = lane % p.sub, po = kW4Rows * rt + prow;
    const int g = (kW4K * kt + gran * s) / p.group;
    const bool in = po < p.d_out && kW4K * kt + gran * s < p.d_in;
    const int64_t at = (e * p.d_out + po) * p.groups + g;
    const float zz = in && p.zeros ? 32.f + (float)(p.zeros[at] & 15) : 40.f;
    const int64_t idx = tile * kW4Rows * p.sub + lane;
    if (p.kind == kW4F32) {
      const float sc = in ? reinterpret_cast<const float*>(p.scales)[at] : 0.f;
      reinterpret_cast<float2*>(p.params)[idx] = make_float2(sc, zz);
    } else {
      const uint32_t sc = in ? reinterpret_cast<const uint16_t*>(p.scales)[at] : 0u;
      if (p.kind == kW4Bf16Zero)
        reinterpret_cast<uint32_t*>(p.params)[idx] = sc | (f32_to_bf16(zz) << 16);
      else
        reinterpret_cast<uint16_t*>(p.params)[idx] = (uint16_t)sc;
    }
  }
}

}  // namespace

hipError_t launch_w4_pack(const lora_w4_store& s, const uint8_t* q, const void* scales, const uint8_t* zeros,
                          void* codes, void* params, hipStream_t stream) {
  W4PackArgs a{};
  a.q = q;
  a.scales = scales;
  a.zeros = zeros;
  a.d_in = s.d_in;
  a.d_out = s.d_out;
  a.group = s.group;
  a.groups = (s.d_in - 1) / s.group + 1;
  a.sub = w4_sub(s.group);
  a.kind = w4_param_kind(s.scale_dtype, s.has_zeros);
  a.k_tiles = w4_k_tiles(s.d_in);
  a.row_tiles = w4_row_tiles(s.d_out);
  a.tiles = (int64_t)s.n * w4_tiles(s.d_in, s.d_out);
  a.codes = reinterpret_cast<char*>(codes);
  a.params = reinterpret_cast<char*>(params);
  // A grid holds less than 2^32 threads on an axis (64 GB of codes).
  const int64_t blocks = (a.tiles + 3) / 4, gx = blocks < (1 << 20) ? blocks : 1 << 20;
  const int64_t gy = (blocks + gx - 1) / gx;
  if (gy > 65535) return hipErrorInvalidValue;
  hipLaunchKernelGGL(w4_pack_kernel, dim3((unsigned)gx, (unsigned)gy), dim3(256), 0, stream, a);
  return hipGetLastError();
}

}  // namespace lora
