// Device helpers of the products of a few tokens.
#pragma once

#include <cuda_fp16.h>

#include "few_tokens.h"
#include "mx_device.cuh"

namespace mx {

// Load from shared memory of a CTA of the cluster (cluster_addr from mapa_shared).
__device__ __forceinline__ float4 ld_cluster_f32x4(uint32_t cluster_addr) {
  float4 v;
  asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
               : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w)
               : "r"(cluster_addr)
               : "memory");
  return v;
}

// Element i of a BF16 array, and a value's BF16 bits (round to nearest even).
__device__ __forceinline__ float bf16_value(const void *p, int64_t i) {
  return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(p)[i]) << 16);
}

__device__ __forceinline__ uint16_t bf16_bits(float v) {
  uint32_t out;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(out) : "f"(0.0f), "f"(v));
  return static_cast<uint16_t>(out & 0xFFFFu);
}

// The sum of output (row, token) of mx_linear_bf16, tensor scale included, with range for
// any x, scale and product of them: a block's elements in binary32 (each product by 2^-8, so
// exact and 32 of them below binary32's end), the blocks in binary64.  The kernels' sums
// have not that range: they are in units of an activation block's largest, and the tensor
// scale comes after them, so one can be infinite or NaN where the sum itself is finite.
// Outputs that are finite are the kernels' own; any other one is this (4096 of K: 100 us),
// which ends early once it is NaN.
template <int FMT>
__device__ __noinline__ float wide_sum(const LinearArgs &a, int64_t row, int token) {
  constexpr int kBlock = FMT == 0 ? 32 : 16;
  const int64_t tiles = (a.k / kBlock + 3) >> 2;
  const int64_t x_row = token * a.ld_x, c_row = row * (a.k >> 1);
  const int64_t s_row = (row >> 7) * tiles * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4;
  double sum = 0.0;
#pragma unroll 2
  for (int64_t k0 = 0; k0 < a.k; k0 += 32) {
    const int64_t block = k0 / kBlock, s_at = s_row + (block >> 2) * 512 + (block & 3);
    if (!in_bounds(s_at, 32 / kBlock, ((a.n + 127) >> 7) * tiles * 512, a.status) ||
        !in_bounds(x_row + k0, 32, (a.tokens - 1) * a.ld_x + a.k, a.status) ||
        !in_bounds(c_row + (k0 >> 1), 16, a.n * (a.k >> 1), a.status))
      continue;
    const uint4 *x_at = reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.x) + x_row + k0);
    const uint4 q = *reinterpret_cast<const uint4 *>(a.w.codes + c_row + (k0 >> 1));
    uint4 v[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] = x_at[i];
    double scale[32 / kBlock];
    if constexpr (FMT == 0) {
      const uint32_t b = a.w.scales[s_at];
      scale[0] = __longlong_as_double((b == 255u ? 0x7FFll : static_cast<long long>(b) + (1023 - 127)) << 52 |
                                      (b == 255u ? 1ll << 51 : 0ll));
    } else {
      uint32_t h;
      asm("cvt.rn.f16x2.e4m3x2 %0, %1;"
          : "=r"(h)
          : "h"(*reinterpret_cast<const uint16_t *>(a.w.scales + s_at)));
      const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
      scale[0] = f.x;
      scale[1] = f.y;
    }
    const uint32_t codes[4] = {q.x, q.y, q.z, q.w};
    float part[32 / kBlock] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t w[4] = {v[i].x, v[i].y, v[i].z, v[i].w};
      float &p = part[i * 8 / kBlock];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        uint32_t h;
        asm("{\n .reg .b8 t;\n cvt.u8.u32 t, %1;\n cvt.rn.f16x2.e2m1x2 %0, t;\n}\n"
            : "=r"(h)
            : "r"((codes[i] >> (8 * j)) & 0xFFu));
        const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
        p += __uint_as_float(w[j] << 16) * (f.x * 0x1p-8f);
        p += __uint_as_float(w[j] & 0xFFFF0000u) * (f.y * 0x1p-8f);
      }
    }
#pragma unroll
    for (int i = 0; i < 32 / kBlock; ++i) sum += static_cast<double>(part[i]) * scale[i];
    if (sum != sum) break;
  }
  return static_cast<float>((FMT == 1 ? sum * static_cast<double>(*a.w.ts) : sum) * 0x1p8);
}

// Stores output (row, token) of mx_linear_bf16 after its epilogue; v: alpha times the
// sum.  Each term is one binary32 operation, then one rounding to the output type.
__device__ __forceinline__ void put_linear(const LinearArgs &a, int64_t row, int token, float v) {
  const int64_t at = token * a.ld_y + row;
  if (!in_bounds(at, 1, (a.tokens - 1) * a.ld_y + a.n, a.status)) return;
  if (a.beta != 0.0f)
    v = __fmaf_rn(a.beta, a.out_fp32 ? static_cast<const float *>(a.y)[at] : bf16_value(a.y, at), v);
  if (a.bias != nullptr) v = __fadd_rn(v, a.bias[row]);
  if (a.gelu) v = gelu_f32x2(make_float2(v, v)).x;
  if (a.out_fp32)
    static_cast<float *>(a.y)[at] = v;
  else
    static_cast<uint16_t *>(a.y)[at] = bf16_bits(v);
}

}  // namespace mx
