// Device helpers of the products of a few tokens.
#pragma once

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
