// Products of a few tokens with FP4 weights: what mx_linear_bf16 (linear.cu)
// and the experts' products (moe.cu) share.
#pragma once

#include <cuda_fp16.h>

#include "mx_device.cuh"
#include "mx_internal.h"

namespace mx {

// Byte offset of the scale of (row, block) in the tcgen05 tile order; tiles =
// ceil(blocks of a row / 4).
__device__ __forceinline__ int64_t scale_offset(int64_t row, int64_t block, int64_t tiles) {
  return ((row >> 7) * tiles + (block >> 2)) * 512 + (row & 31) * 16 + ((row >> 5) & 3) * 4 +
         (block & 3);
}

// A scale byte's value: UE8M0 (255 is NaN) or E4M3.
template <int FMT>
__device__ __forceinline__ float scale_value(uint32_t byte) {
  if constexpr (FMT == 0) {
    return byte == 255u ? __uint_as_float(0x7FFFFFFFu)
                        : __uint_as_float(max(byte << 23, 0x00400000u));
  } else {
    uint32_t h;
    asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(byte)));
    return __half2float(__ushort_as_half(static_cast<unsigned short>(h & 0xFFFFu)));
  }
}

// The two E2M1 codes of a byte as FP16 (low nibble in the low half), exact.
__device__ __forceinline__ uint32_t e2m1x2_f16x2(uint32_t byte) {
  uint32_t h;
  asm("{\n .reg .b8 t;\n cvt.u8.u32 t, %1;\n cvt.rn.f16x2.e2m1x2 %0, t;\n}\n" : "=r"(h) : "r"(byte));
  return h;
}

// One warp: sum over k of weight (row) times x for `count` (<= N) rows of x,
// the full sum in every lane.  x(i, k) gives element k of the i-th row.
template <int FMT, int N, typename X>
__device__ __forceinline__ void warp_row_dot(const uint8_t *codes, const uint8_t *scales,
                                             int64_t row, int64_t k, int count, const X &x,
                                             float (&acc)[N]) {
  const int lane = threadIdx.x & 31;
  const int64_t tiles = (k / (FMT == 0 ? 32 : 16) + 3) / 4;
#pragma unroll
  for (int i = 0; i < N; ++i) acc[i] = 0.0f;
  for (int64_t w = lane; w < k / 8; w += 32) {
    const uint32_t word = *reinterpret_cast<const uint32_t *>(codes + row * (k / 2) + w * 4);
    const float s = scale_value<FMT>(scales[scale_offset(row, FMT == 0 ? w / 4 : w / 2, tiles)]);
    float v[8];
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const float2 f = __half22float2(__halves2half2(
          __ushort_as_half(static_cast<unsigned short>(e2m1x2_f16x2(word >> (8 * b)) & 0xFFFFu)),
          __ushort_as_half(static_cast<unsigned short>(e2m1x2_f16x2(word >> (8 * b)) >> 16))));
      v[2 * b] = f.x * s;
      v[2 * b + 1] = f.y * s;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i < count) {
#pragma unroll
        for (int j = 0; j < 8; ++j) acc[i] = __fmaf_rn(v[j], x(i, w * 8 + j), acc[i]);
      }
    }
  }
#pragma unroll
  for (int i = 0; i < N; ++i) {
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) acc[i] += __shfl_xor_sync(0xFFFFFFFFu, acc[i], m);
  }
}

__device__ __forceinline__ float bf16_value(const void *p, int64_t i) {
  return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(p)[i]) << 16);
}

__device__ __forceinline__ uint16_t bf16_bits(float v) {
  uint32_t out;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(out) : "f"(0.0f), "f"(v));
  return static_cast<uint16_t>(out & 0xFFFFu);
}

}  // namespace mx
