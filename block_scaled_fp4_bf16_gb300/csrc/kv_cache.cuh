// Device helpers of the paged cache (kv_append.cu, attention.cu).
#pragma once

#include "decode.h"
#include "mx_device.cuh"

namespace mx {

// The length of sequence b as it stands in memory.
__device__ __forceinline__ int64_t stated_length(const CacheArgs &c, int b) {
  return in_bounds(b, 1, c.sequences, c.status) ? c.lengths[b] : 0;
}

// Tokens of sequence b: its length within 0 .. max_pages * page_tokens.
__device__ __forceinline__ int64_t cache_length(const CacheArgs &c, int b) {
  const int64_t n = stated_length(c, b);
  const int64_t most = c.max_pages * c.page_tokens;
  if (n < 0 || n > most) {
    atomicOr(c.status, kStatusIndexBit);
    return n < 0 ? 0 : most;
  }
  return n;
}

// Page that holds token t (within the length) of sequence b; -1, and recorded, if it is
// none of the pool.
__device__ __forceinline__ int64_t cache_page(const CacheArgs &c, int b, int64_t t) {
  const int64_t at = b * c.max_pages + t / c.page_tokens;
  if (!in_bounds(at, 1, c.sequences * c.max_pages, c.status)) return -1;
  const int64_t page = c.table[at];
  if (page >= 0 && page < c.pages) return page;
  atomicOr(c.status, kStatusIndexBit);
  return -1;
}

// 2^e for e in -149 .. 127.
__device__ __forceinline__ float exp2_int(int e) {
  return e >= -126 ? __int_as_float((e + 127) << 23) : __int_as_float(1 << (e + 149));
}

// Two E4M3 codes (the lower byte first) as binary32.
__device__ __forceinline__ float2 e4m3x2_value(uint32_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(static_cast<uint16_t>(codes)));
  float2 v;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, h;\n}\n"
      : "=f"(v.x), "=f"(v.y)
      : "r"(h));
  return v;
}

}  // namespace mx
