// Activations as sums of FP4, for products of a few tokens on the FP4 tensor cores
// (moe_mma.cu, linear_mma.cu).
//
// The weights' bytes bound such products, so no instruction should touch a
// weight: codes and scales go from memory to the block-scaled FP4 product as
// they lie.  For that the activations have to be FP4 too, without losing their
// digits: a value is written as a sum of eight E2M1 digits,
//     x = 2^e (q_0 + 2^-2 q_1 + 2^-5 q_2 + ... + 2^-20 q_7),   e for its block,
// each digit the rounding of what the ones before it left (what is left after
// q_0 is at most 1 of 6, after every other at most 1/2 of 4, so eight digits
// reach 2^-21 of the block's scale: a BF16 value is exact unless its last bit
// lies below that).  The digits of a token are eight rows of the product's
// narrow operand, and the epilogue adds their eight sums in binary32.  The FP4
// rate makes the eightfold product cheaper than converting the weights.
#pragma once

#include <cuda_fp16.h>

#include "few_tokens.cuh"

namespace mx {

constexpr int kDigits = 8;
constexpr int kImageK = 256;                   // elements of K of a stage
constexpr int kImageCodes = kDigits * 128;     // bytes of codes
// Bytes of a scale tile's scales in a stage: 128 rows (16 activations' digits) and four
// blocks, two (MXFP4) or four (NVFP4) of them a stage.
template <int FMT>
constexpr int kImageScales = (FMT == 0 ? 2 : 4) * 512;
constexpr int kTileRows = 16;  // rows of activations whose digits fill a scale tile
static_assert(kTileRows * kDigits == 128 && kMoeGroupMax == kTileRows, "digits of a scale tile");
// Weight of digit p: 2^-kShift[p].
__host__ __device__ constexpr int digit_shift(int p) { return p == 0 ? 0 : 3 * p - 1; }

// Where digits go.  Rows are places.
struct Image {
  uint8_t *codes;       // [stages][rows][kImageCodes]
  uint8_t *scales;      // [stages][tiles][kImageScales]
  float *factors;       // NVFP4: [rows], the power of two of a place
  int rows, tiles;
};

// Largest e with |v| <= 6 * 2^e for |v| <= top, as small as it can be; top > 0.
__device__ __forceinline__ int block_exponent(float top) {
  const uint32_t u = __float_as_uint(top);
  if (u < 0x00800000u) return -127;  // subnormal: 2^-126 at most
  const int e = static_cast<int>(u >> 23) - 127;
  return (u & 0x007FFFFFu) > 0x00400000u ? e - 1 : e - 2;
}

// 2^e for -149 <= e <= 127.
__device__ __forceinline__ float pow2(int e) {
  return e >= -126 ? __uint_as_float(static_cast<uint32_t>(e + 127) << 23)
                   : __uint_as_float(1u << (e + 149));
}

// NVFP4: exponent of a row's factor, the largest finite magnitude being `top`: the
// largest block's scale becomes 2^8, the largest power of two of E4M3.
__device__ __forceinline__ int row_exponent(float top) { return max(block_exponent(top) - 8, -118); }

__device__ __forceinline__ void raise_finite(float &top, const float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float a = fabsf(v[i]);
    if (a < __uint_as_float(0x7F800000u)) top = fmaxf(top, a);
  }
}

__device__ __forceinline__ float warp_max(float v) {  // v >= 0
  return __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(v)));
}

// Whole warp.  The digits of 256 elements (eight a lane), written to `copies` places
// of an image's stage (`codes`, `scales`): places[j] (0xFFFF: none), or `place` where
// places is null; members[place] (null: place) is its scale tile * kTileRows + its row
// there.  MXFP4: UE8M0 scales for 32 (four lanes), digit p with the scale
// 2^(e - shift p); NVFP4: E4M3 for 16 (two lanes), a power of two relative to 2^row_e,
// the digits' weights left to the reader.  A block that holds an infinity or NaN gets
// the scale NaN.
//
// Not inlined, and the digits a loop: instructions that run for the first time are
// fetched behind the weights that stream meanwhile (unrolled and inlined, 8 KB of code,
// the digits of x were there 1 us later: 4.5 us and 3.6 us into the experts' kernel, 1 x
// 2048).  Kernels call it once with no copies before there is such a stream
// (warm_digits).
template <int FMT>
__device__ __noinline__ void write_digits(uint8_t *codes, uint8_t *scales, float v0, float v1,
                                          float v2, float v3, float v4, float v5, float v6,
                                          float v7, int row_e, int copies, const uint16_t *places,
                                          int place, const uint16_t *members) {
  float v[8] = {v0, v1, v2, v3, v4, v5, v6, v7};
  const int lane = threadIdx.x & 31;
  float top = 0.0f;
  uint32_t odd = 0;  // an infinity or NaN here
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    top = fmaxf(top, fabsf(v[i]));
    odd |= (__float_as_uint(v[i]) & 0x7F800000u) == 0x7F800000u;
  }
#pragma unroll
  for (int m = 1; m < (FMT == 0 ? 4 : 2); m <<= 1) {
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, m));
    odd |= __shfl_xor_sync(0xFFFFFFFFu, odd, m);
  }
  int e = block_exponent(top);
  uint32_t byte;
  if constexpr (FMT == 0) {
    e = max(e, -127);
    byte = odd ? 255u : static_cast<uint32_t>(e + 127);
  } else {
    const int j = min(max(e - row_e, -9), 8);  // 2^-9 is E4M3's least
    e = row_e + j;
    byte = odd ? 0x7Fu : j >= -6 ? static_cast<uint32_t>(j + 7) << 3 : 1u << (j + 9);
  }
  // v 2^-e, in two steps where one power of two would not be a normal number
  const float f0 = pow2(min(-e, 100)), f1 = pow2(-e - min(-e, 100));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = odd ? 0.0f : v[i] * f0 * f1;
  uint32_t digits[kDigits] = {};
#pragma unroll 1
  for (int d = 0; d < kDigits; ++d) {
    const float up = d == 0 ? 4.0f : 8.0f;
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t c = cvt_e2m1x2(v[2 * i], v[2 * i + 1]);
      uint32_t h;
      asm("{\n .reg .b8 t;\n cvt.u8.u32 t, %1;\n cvt.rn.f16x2.e2m1x2 %0, t;\n}\n" : "=r"(h) : "r"(c));
      const float2 q = __half22float2(*reinterpret_cast<const __half2 *>(&h));
      v[2 * i] = (v[2 * i] - q.x) * up;
      v[2 * i + 1] = (v[2 * i + 1] - q.y) * up;
      w |= c << (8 * i);
    }
    if (FMT == 0 && digit_shift(d) > e + 127) w = 0;  // (no scale that small)
#pragma unroll
    for (int i = 0; i + 1 < kDigits; ++i) digits[i] = digits[i + 1];
    digits[kDigits - 1] = w;
  }
  // scale words of four blocks, for each digit's row
  constexpr int kWords = FMT == 0 ? 2 : 4;
  uint32_t words[kWords] = {};
#pragma unroll
  for (int b = 0; b < 4 * kWords; ++b)
    words[b / 4] |= __shfl_sync(0xFFFFFFFFu, byte, b * (8 / kWords)) << (8 * (b % 4));
  if constexpr (FMT == 0) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      // 255 stays NaN; a digit whose scale would lie below 2^-127 is 0
      const uint32_t nan = __vcmpeq4(words[i], 0xFFFFFFFFu);
      words[i] = __vsubus4(words[i], ((lane & 7) == 0 ? 0u : 3u * (lane & 7) - 1u) * 0x01010101u) | nan;
    }
  }
  // row d of the 8 x 128 byte tile, 16-byte chunk lane / 4, swizzled
  uint32_t at[kDigits];
#pragma unroll
  for (int d = 0; d < kDigits; ++d) at[d] = d * 128 + (((lane >> 2) ^ d) << 4) + (lane & 3) * 4;
#pragma unroll 1
  for (int j = 0; j < copies; ++j) {
    const int to = places != nullptr ? places[j] : place;
    if (to == 0xFFFF) continue;
    uint8_t *c = codes + static_cast<int64_t>(to) * kImageCodes;
#pragma unroll
    for (int d = 0; d < kDigits; ++d) *reinterpret_cast<uint32_t *>(c + at[d]) = digits[d];
    if (lane < kDigits) {
      // digit rows of a group in the order of a scale tile: row c at c % 32, word c / 32
      const int mem = members != nullptr ? members[to] : to, m = mem % kTileRows;
      uint8_t *dst = scales + (mem / kTileRows) * kImageScales<FMT> +
                     ((m & 3) * kDigits + lane) * 16 + (m >> 2) * 4;
#pragma unroll
      for (int i = 0; i < kWords; ++i) *reinterpret_cast<uint32_t *>(dst + i * 512) = words[i];
    }
  }
}

// The digits of v for `copies` places of stage `stage`.
template <int FMT>
__device__ __forceinline__ void write_digits(const Image &out, int stage, const float (&v)[8],
                                             int row_e, int copies, const uint16_t *places,
                                             int place, const uint16_t *members) {
  write_digits<FMT>(out.codes + static_cast<int64_t>(stage) * out.rows * kImageCodes,
                    out.scales + static_cast<int64_t>(stage) * out.tiles * kImageScales<FMT>, v[0],
                    v[1], v[2], v[3], v[4], v[5], v[6], v[7], row_e, copies, places, place, members);
}
template <int FMT>
__device__ __forceinline__ void warm_digits(const Image &out) {
  const float v[8] = {};
  write_digits<FMT>(out, 0, v, 0, 0, nullptr, 0, nullptr);
}

// Warps of a CTA that makes digits of x.
template <int FMT>
constexpr int kDigitWarps = FMT == 0 ? 4 : 8;

// The CTA's W warps: the digits of token t, stages group * W and on, one a warp, places
// by token.  NVFP4's factor needs the token's largest magnitude, which the CTA looks for
// together (tops: W words of shared memory).
template <int FMT, int W>
__device__ __forceinline__ void token_digits(const Image &out, const void *x, int64_t ld_x,
                                             int tokens, int64_t k, int t, int group,
                                             uint32_t *tops, uint32_t *status) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int64_t extent = (tokens - 1) * ld_x + k;
  const auto load = [&](int64_t at) {
    const int64_t off = t * ld_x + at;
    return at < k && in_bounds(off, 8, extent, status)
               ? *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(x) + off)
               : make_uint4(0, 0, 0, 0);
  };
  // (its own part first: later loads queue behind the next kernel's first weights)
  const int st = group * W + warp;
  const uint4 q = load(static_cast<int64_t>(st) * kImageK + lane * 8);
  int row_e = 0;
  if constexpr (FMT == 1) {
    // magnitudes compare as integers; one of 0x7F80 or more is no number and counts as 0
    uint32_t top = 0;
    for (int64_t at = threadIdx.x * 8; at < k; at += 8 * W * kImageK) {
      uint4 u[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) u[i] = load(at + i * W * kImageK);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t w[4] = {u[i].x, u[i].y, u[i].z, u[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t m = w[j] & 0x7FFF7FFFu;
          top = __vmaxu2(top, m & ~__vcmpgeu2(m, 0x7F807F80u));
        }
      }
    }
    top = __reduce_max_sync(0xFFFFFFFFu, max(top & 0xFFFFu, top >> 16));
    if (lane == 0) tops[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < W; ++w) top = max(top, tops[w]);
    __syncthreads();  // (before another call writes them)
    row_e = row_exponent(__uint_as_float(top << 16));
    if (group == 0 && threadIdx.x == 0) out.factors[t] = pow2(row_e);
  }
  if (static_cast<int64_t>(st) * kImageK >= k) return;
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
  float v[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
  write_digits<FMT>(out, st, v, row_e, 1, nullptr, t, nullptr);
}

// The images in the experts' workspace: codes of x, scales of x, codes of h, scales of
// h.  Rows are pairs sorted by expert; of x, for so few tokens that all of them fit any
// group, the tokens (moe_by_token).
inline Image moe_image_of(const MoeArgs &a, bool of_h) {
  const int64_t pairs = static_cast<int64_t>(a.tokens) * a.top_k;
  const bool by_token = !of_h && moe_by_token(a.fmt, a.tokens);
  const int64_t rows = by_token ? a.tokens : pairs;
  uint8_t *at = a.image + (of_h ? moe_image_bytes(pairs, a.hidden) : 0);
  const int64_t stages = ((of_h ? a.inter : a.hidden) + kImageK - 1) / kImageK;
  return Image{at, at + rows * stages * kImageCodes, a.factors + (of_h ? pairs : 0),
               static_cast<int>(rows), by_token ? 1 : static_cast<int>(pairs)};
}

// ---------------------------------------------------------------- grid-wide counts
// Kernels whose CTAs are resident together (a cooperative launch) count the CTAs
// that have finished a part; a wait for the count is bounded all the same.

__device__ __forceinline__ uint32_t load_acquire(const uint32_t *count) {
  uint32_t v;
  asm volatile("ld.acquire.gpu.u32 %0, [%1];" : "=r"(v) : "l"(count) : "memory");
  return v;
}

// Adds one after all that this thread has seen done, and what a barrier ordered before
// it (a release is cumulative; a __threadfence before it only took 0.3 us more of each).
__device__ __forceinline__ void release_add(uint32_t *count) {
  asm volatile("red.release.gpu.global.add.u32 [%0], 1;" ::"l"(count) : "memory");
}

// The same, and what others had done when they added is seen after it; what it was.
__device__ __forceinline__ uint32_t acquire_release_add(uint32_t *count) {
  uint32_t was;
  asm volatile("atom.acq_rel.gpu.global.add.u32 %0, [%1], 1;" : "=r"(was) : "l"(count) : "memory");
  return was;
}

// One thread, or a whole warp together (a warp of which one lane waits comes out
// diverged, and every shuffle after it then takes 330 clocks: measured, 4 us of a
// write_digits; experts 1 x 2048 x 1024 of 64 25.3 us, so 20.7).  False when the wait
// ran out (abort is raised then) or abort was up.
__device__ __forceinline__ bool count_reached(const uint32_t *count, uint32_t target,
                                              volatile uint32_t *abort, uint32_t *status) {
  const uint64_t t0 = globaltimer_ns();
  while (true) {
    if (load_acquire(count) >= target) return true;
    if (*abort) return false;
    if (globaltimer_ns() - t0 > kWaitTimeoutNs) {
      *abort = 1u;
      atomicOr(status, kStatusTimeout);
      return false;
    }
  }
}

// `threads` threads of the CTA (named barrier 1; `leader` is one of them): what they
// wrote is counted once.
__device__ __forceinline__ void add_count(uint32_t *count, int threads, bool leader) {
  named_barrier_sync(1, threads);
  if (leader) release_add(count);
}

// The same threads: every CTA has counted (false: given up).  The leader's warp looks.
__device__ __forceinline__ bool all_counted(const uint32_t *count, int threads, bool leader,
                                            volatile uint32_t *flag, volatile uint32_t *abort,
                                            uint32_t *status) {
  if (__any_sync(0xFFFFFFFFu, leader)) {
    const bool ok = __all_sync(0xFFFFFFFFu, count_reached(count, gridDim.x, abort, status));
    if (leader) *flag = ok ? 1u : 0u;
  }
  named_barrier_sync(1, threads);
  return *flag != 0u;
}

}  // namespace mx
