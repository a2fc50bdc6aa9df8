// Stores new keys and values in the paged cache: E4M3 codes under one power of two for each
// 32 tokens and head.
//
// The scale is 2^e, e the least with amax <= 448 2^e: a power of two moves only E4M3's
// exponent, so that when a later token raises e, rounding the held codes again loses
// nothing but what falls below 2^-6 of the new range.
//
// A CTA takes the new tokens of one block of 32 of one sequence, for as many heads as come to
// 256 channels (one head a CTA: 23 us for 16384 x 8 x 128, 35 for 16 x 64, where this takes 19 and
// 19 on one input again and again; 21.5 for the first over inputs in turn).  A unit of its threads has the keys or the values of a head: it reads each once, holds
// it in registers (8 channels a lane) while the largest magnitude goes across its warps, and
// writes its codes.  What a value costs bounds a prompt (so the largest of two at a time, one
// factor, no test for infinities where the block has none), the chain starts and lengths,
// page, scale a single token; the values are read beside it.
#include <cuda_fp16.h>

#include "kv_cache.cuh"

namespace mx {
namespace {

constexpr int kThreads = 256;

// The least e with amax <= 448 * 2^e, -127 .. 120 (-127 for 0).
__device__ __forceinline__ int block_exponent(uint32_t amax) {
  const int e = static_cast<int>(amax >> 23);  // 448 = 1.75 * 2^8
  if (e == 0) return -127;                     // (below 2^-126: less than 448 * 2^-127)
  const int up = (amax & 0x7FFFFFu) > 0x600000u;
  return max(e - 127 - 8 + up, -127);
}

// The larger of each of two unsigned 16-bit numbers.
__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

__device__ __forceinline__ int64_t start_of(const AppendArgs &a, int i) {
  return in_bounds(i, 1, a.c.sequences + 1, a.c.status) ? a.starts[i] : 0;
}

template <int DIM>
__global__ void __launch_bounds__(kThreads) append_kernel(const __grid_constant__ AppendArgs a) {
  constexpr int kLanes = DIM / 8, kRows = 4, kPasses = kCacheBlock / kRows;
  constexpr int kUnit = kLanes * kRows, kUnits = kThreads / kUnit;  // a unit: keys or values of a head
  __shared__ int found, descends, shared_slots;  // the sequence; are starts out of order; a slot that two take
  __shared__ uint32_t largest[kThreads / 32];
  griddep_launch_dependents();
  griddep_wait();
  const CacheArgs &c = a.c;
  const int unit = threadIdx.x / kUnit, thread = threadIdx.x % kUnit;
  const int which = unit & 1, head = blockIdx.y * (kUnits / 2) + (unit >> 1);
  // Slots of sequence b begin at starts[b] / 32 + 2 b, which leaves room for any place
  // of its tokens in their blocks.
  int b = 0;
  int64_t row0 = 0, n = 0, index = 0, stated = 0;
  if (a.starts == nullptr) {
    n = a.tokens / c.sequences;
    const int per = static_cast<int>((n + kCacheBlock - 2) / kCacheBlock + 1);
    b = static_cast<int>(blockIdx.x) / per;
    index = static_cast<int>(blockIdx.x) % per;
    row0 = b * n;
    stated = stated_length(c, b);
  } else {
    if (threadIdx.x == 0) found = 0x7FFFFFFF, descends = shared_slots = 0;
    __syncthreads();
    const int64_t slot = blockIdx.x;
    for (int i = threadIdx.x; i < c.sequences; i += kThreads) {
      const int64_t s0 = start_of(a, i), s1 = start_of(a, i + 1);
      if (s0 < 0 || s1 < s0 || s1 > a.tokens) {
        if (slot == 0 && blockIdx.y == 0) atomicOr(c.status, kStatusIndexBit);
        descends = 1;
        continue;
      }
      // (starts in order make a slot that of one sequence; out of order, the first one takes it, see below)
      if (slot >= s0 / kCacheBlock + 2 * static_cast<int64_t>(i) &&
          slot < s1 / kCacheBlock + 2 * static_cast<int64_t>(i) + 2)
        atomicMin(&found, i);
    }
    __syncthreads();
    b = found;
    if (b == 0x7FFFFFFF) return;
    row0 = start_of(a, b);
    n = start_of(a, b + 1) - row0;
    if (descends) {
      // a sequence with slots that an earlier one has, too, is left out as a whole
      for (int i = threadIdx.x; i < b; i += kThreads) {
        const int64_t s0 = start_of(a, i), s1 = start_of(a, i + 1);
        if (s0 >= 0 && s1 >= s0 && s1 <= a.tokens && s1 / kCacheBlock + 2 * static_cast<int64_t>(i) + 2 >
                                                        row0 / kCacheBlock + 2 * static_cast<int64_t>(b))
          shared_slots = 1;
      }
      __syncthreads();
      if (shared_slots) return;
    }
    stated = stated_length(c, b);
    index = slot - (row0 / kCacheBlock + 2 * static_cast<int64_t>(b));
  }
  if (head >= c.heads) return;
  // positions first .. first + n - 1, of which those from 0 on are stored
  const int64_t length = cache_length(c, b);
  const int64_t first = stated - n, begin = first > 0 ? first : 0;
  const int64_t block0 = (begin / kCacheBlock + index) * kCacheBlock;
  const int64_t from = begin > block0 ? begin : block0;
  const int64_t to = length < block0 + kCacheBlock ? length : block0 + kCacheBlock;
  if (from >= to) return;
  const int held = static_cast<int>(from - block0), count = static_cast<int>(to - from);

  const int lane = thread % kLanes, sub = thread / kLanes;
  const int64_t rows = row0 + (from - first);
  const int64_t extent = (a.tokens - 1) * a.ld[which] + static_cast<int64_t>(c.heads) * DIM;
  const int64_t x_at = (rows + sub) * a.ld[which] + head * DIM + lane * 8;
  uint4 x[kPasses];
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    x[i] = make_uint4(0, 0, 0, 0);
    const int64_t at = x_at + i * kRows * a.ld[which];
    if (i * kRows + sub < count && in_bounds(at, 8, extent, c.status))
      x[i] = *reinterpret_cast<const uint4 *>(a.x[which] + at);
  }
  const int64_t page = cache_page(c, b, block0);
  if (page < 0) return;
  const int in_page = static_cast<int>(block0 % c.page_tokens);
  const int64_t base = (page * c.heads + head) * c.page_tokens + in_page;
  uint8_t *scale = c.scales[which] + base / kCacheBlock;
  const int64_t scales = c.pages * c.heads * (c.page_tokens / kCacheBlock);
  const int before = held > 0 && in_bounds(base / kCacheBlock, 1, scales, c.status) ? *scale - 127 : -127;
  __syncwarp();  // (the scale is written at the end; a unit of several warps meets below)

  // magnitudes are ordered as the bits without the sign: two at a time
  uint32_t most = 0;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    most = max_u16x2(most, max_u16x2(x[i].x & 0x7FFF7FFFu, x[i].y & 0x7FFF7FFFu));
    most = max_u16x2(most, max_u16x2(x[i].z & 0x7FFF7FFFu, x[i].w & 0x7FFF7FFFu));
  }
  uint32_t amax = __reduce_max_sync(0xFFFFFFFFu, max(most & 0xFFFFu, most >> 16)) << 16;
  auto across = [&] {  // the largest of the unit's warps
    if constexpr (kUnit > 32) {
      if ((threadIdx.x & 31) == 0) largest[threadIdx.x >> 5] = amax;
      named_barrier_sync(1 + unit, kUnit);
#pragma unroll
      for (int w = 0; w < kUnit / 32; ++w) amax = max(amax, largest[unit * (kUnit / 32) + w]);
    }
  };
  across();
  const bool wild = amax >= 0x7F800000u;  // infinities or NaN: the scale goes by the others
  if (wild) {
    amax = 0;
#pragma unroll
    for (int i = 0; i < kPasses; ++i) {
      const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
#pragma unroll
      for (int k = 0; k < 4; ++k) {
        const uint32_t lo = (w[k] & 0x7FFFu) << 16, hi = w[k] & 0x7FFF0000u;
        amax = max(amax, max(lo < 0x7F800000u ? lo : 0u, hi < 0x7F800000u ? hi : 0u));
      }
    }
    amax = __reduce_max_sync(0xFFFFFFFFu, amax);
    if constexpr (kUnit > 32) named_barrier_sync(1 + unit, kUnit);  // (the others have read the first ones)
    across();
  }
  const int e = max(block_exponent(amax), before);
  const float f = exp2_int(-e);
  uint8_t *codes = c.codes[which] + base * DIM;
  const int64_t code_extent = c.pages * c.heads * c.page_tokens * DIM - base * DIM;
#pragma unroll
  for (int i = 0; i < kPasses; ++i) {
    const int r = i * kRows + sub;
    if (r >= count) continue;
    const uint32_t w[4] = {x[i].x, x[i].y, x[i].z, x[i].w};
    uint16_t out[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const float2 v = mul_f32x2(make_float2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xFFFF0000u)),
                                 make_float2(f, f));
      float lo = v.x, hi = v.y;
      if (wild) {  // (the conversion would make an infinity 448)
        if (fabsf(lo) == INFINITY) lo = NAN;
        if (fabsf(hi) == INFINITY) hi = NAN;
      }
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(out[k]) : "f"(hi), "f"(lo));
    }
    const int at = (held + r) * DIM + lane * 8;
    if (in_bounds(at, 8, code_extent, c.status))
      *reinterpret_cast<uint2 *>(codes + at) =
          make_uint2(out[0] | static_cast<uint32_t>(out[1]) << 16, out[2] | static_cast<uint32_t>(out[3]) << 16);
  }
  if (e > before && held > 0) {
    // what the block holds, rounded again under the new scale
    const float g = exp2_int(max(before - e, -149));
    for (int i = thread; i < held * (DIM / 4); i += kUnit) {
      if (!in_bounds(static_cast<int64_t>(i) * 4, 4, code_extent, c.status)) continue;
      uint32_t *p = reinterpret_cast<uint32_t *>(codes) + i;
      const float2 lo = e4m3x2_value(*p & 0xFFFFu), hi = e4m3x2_value(*p >> 16);
      uint16_t l, h;
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(l) : "f"(lo.y * g), "f"(lo.x * g));
      asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(h) : "f"(hi.y * g), "f"(hi.x * g));
      const uint32_t nan = ((((*p & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) >> 7) * 0xFFu;  // (stays as it is)
      *p = (*p & nan) | ((l | static_cast<uint32_t>(h) << 16) & ~nan);
    }
  }
  if (thread == 0 && in_bounds(base / kCacheBlock, 1, scales, c.status)) *scale = static_cast<uint8_t>(e + 127);
}

template <int DIM>
cudaError_t launch(const AppendArgs &a, cudaStream_t s) {
  int64_t slots;
  if (a.starts == nullptr) {
    const int64_t n = a.tokens / a.c.sequences;
    slots = a.c.sequences * ((n + kCacheBlock - 2) / kCacheBlock + 1);
  } else {
    slots = a.tokens / kCacheBlock + 2 * static_cast<int64_t>(a.c.sequences);
  }
  constexpr int kHeads = kThreads / (DIM / 2) / 2;  // of a CTA
  return launch_pdl(append_kernel<DIM>, dim3(static_cast<unsigned>(slots), (a.c.heads + kHeads - 1) / kHeads),
                    dim3(kThreads), 0, s, a);
}

}  // namespace

cudaError_t launch_kv_append(const AppendArgs &a, cudaStream_t s) {
  switch (a.c.head_dim) {
    case 64: return launch<64>(a, s);
    case 128: return launch<128>(a, s);
    default: return launch<256>(a, s);
  }
}

}  // namespace mx
