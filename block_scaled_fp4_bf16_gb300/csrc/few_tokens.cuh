// Products of a few tokens with FP4 weights: the core of mx_linear_bf16
// (linear.cu) and of the experts' products (moe.cu).
//
// out[n, t] = sum_k W[n, k] x[t, k] for R = 16 MT weight rows and up to 8 NT
// tokens.  The weights' bytes bound it (4.25 or 4.5 bits each; at 6.8 TB/s an
// SM has to take 45 codes a clock), so the kernel is built to keep weight
// copies in flight and to spend few instructions on a code:
//   - a warp owns a range of K and walks it in stages of 128: codes, scales and
//     activations of a stage come by cp.async into the warp's own ring in shared
//     memory, and run on over the end of one tile into the next; warps meet
//     only to add their partial sums;
//   - E2M1 becomes FP16 by the conversion instruction, two codes at once, and
//     multiplies on the 16 x 8 x 16 FP16 product with binary32 sums, the
//     weights on its 16-row side (measured: 90 codes a clock per SM converted,
//     128 multiplied; the tcgen05 forms would multiply faster, but want codes of
//     either format at both operands or FP16 tiles written back to memory);
//   - MXFP4 scales apply to the sum of a 32-block (any UE8M0 power of two), the
//     E4M3 scales of NVFP4 to the FP16 weights (code * scale has 6 bits: exact);
//   - activations become FP16 times a power of two for each (token, 128): BF16
//     values keep all their bits unless they lie 2^-31 below the largest of the
//     128.
#pragma once

#include <cuda_fp16.h>

#include "mx_device.cuh"
#include "mx_internal.h"

namespace mx {
namespace few {

constexpr int kStageK = 128;  // K elements of a stage

// Bytes of a token's row in a stage, padded so that a quarter warp's 16-byte
// reads (two tokens) fall on distinct banks.
template <typename XT>
constexpr int x_pitch() {
  return sizeof(XT) == 2 ? 256 + 64 : 512 + 16;
}

// A multiple of 64: stage_product steps between chunks by flipping address bits.
template <int FMT, int MT, typename XT>
__host__ __device__ constexpr int stage_bytes(int tokens) {
  return (16 * MT * (64 + (FMT == 0 ? 4 : 8)) + tokens * x_pitch<XT>() + 63) / 64 * 64;
}

// One matrix of a stack: codes, scales and their extents (of the whole stack,
// for the bounds-checked build).
struct Rows {
  const uint8_t *codes;
  const uint8_t *scales;
  int64_t code_off, scale_off;    // of this matrix in the stack
  int64_t code_end, scale_end;    // extents of the stack
};

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *base, int64_t off, bool valid,
                                           int64_t extent, uint32_t *status) {
  valid = valid && in_bounds(off, 16, extent, status);
  asm volatile("cp.async.cg.shared.global.L2::128B [%0], [%1], 16, %2;" ::"r"(dst),
               "l"(static_cast<const char *>(base) + (valid ? off : 0)), "r"(valid ? 16 : 0)
               : "memory");
}

__device__ __forceinline__ void cp_async4(uint32_t dst, const void *base, int64_t off, bool valid,
                                          int64_t extent, uint32_t *status) {
  valid = valid && in_bounds(off, 4, extent, status);
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst),
               "l"(static_cast<const char *>(base) + (valid ? off : 0)), "r"(valid ? 4 : 0)
               : "memory");
}

__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }

template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t addr, uint32_t (&r)[4]) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];"
               : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
               : "r"(addr)
               : "memory");
  return v;
}

__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr) : "memory");
  return v;
}

__device__ __forceinline__ uint32_t lds32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}

// d = a b + c: 16 x 16 times 16 x 8, FP16 operands, binary32 sums.
__device__ __forceinline__ void mma_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                          uint32_t a3, uint32_t b0, uint32_t b1,
                                          const float (&c)[4]) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%10, %11, %12, %13};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c[0]), "f"(c[1]), "f"(c[2]),
        "f"(c[3]));
}

// Eight codes (a word) as four FP16 pairs, in the order of K.
__device__ __forceinline__ void e2m1x8_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n .reg .b8 x0, x1, x2, x3;\n mov.b32 {x0, x1, x2, x3}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, x0;\n cvt.rn.f16x2.e2m1x2 %1, x1;\n"
      " cvt.rn.f16x2.e2m1x2 %2, x2;\n cvt.rn.f16x2.e2m1x2 %3, x3;\n}\n"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}

// Two UE8M0 bytes (the low half of `b`) as BF16 pair, and two E4M3 as FP16 pair.
__device__ __forceinline__ uint32_t ue8m0x2_bf16x2(uint32_t b) {
  uint32_t r;
  asm("cvt.rn.bf16x2.ue8m0x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(b)));
  return r;
}
__device__ __forceinline__ uint32_t e4m3x2_f16x2(uint32_t b) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(b)));
  return r;
}
__device__ __forceinline__ uint32_t mul_f16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t mul_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// ---------------------------------------------------------------- copies in

// Copies the codes and scales of stage `s` of R = 16 MT rows into `dst`.  The
// rows are two halves of 8 MT that begin at row first[0] of m[0] and first[1] of
// m[1] (the same matrix, 8 MT apart, unless the tile holds gate and up rows);
// rows at or past n and K blocks at or past k become zeros.
template <int FMT, int MT>
__device__ __forceinline__ void load_weights(uint32_t dst, const Rows (&m)[2], const int (&first)[2],
                                             int n, int k, int s, uint32_t *status) {
  constexpr int R = 16 * MT, kHalf = R / 2;
  const int lane = threadIdx.x & 31;
  // codes: 64 bytes of a row in four 16-byte chunks (one 32-block each), chunk c
  // of row r at c ^ (r / 2 % 4): ldmatrix then reads without bank conflicts
  const int chunk = lane & 3, row0 = lane >> 2;
  const int64_t ldb = k >> 1;
  const bool k_in = s * kStageK + chunk * 32 < k;
#pragma unroll
  for (int j = 0; j < R / 8; ++j) {
    const int h = j * 8 >= kHalf ? 1 : 0;
    const int row = row0 + j * 8;
    const int at = first[h] + row - h * kHalf;
    cp_async16(dst + row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4), m[h].codes,
               m[h].code_off + at * ldb + (s * 64 + chunk * 16), k_in && at < n, m[h].code_end,
               status);
  }
  // scales: the four (MXFP4) or eight bytes of a row, one tile column each word
  constexpr int kCols = FMT == 0 ? 1 : 2;
  const int tiles = (k / (FMT == 0 ? 32 : 16) + 3) >> 2;
  const uint32_t sdst = dst + R * 64;
#pragma unroll
  for (int i0 = 0; i0 < R * kCols; i0 += 32) {
    const int i = i0 + lane;
    const int row = i % R, q = i / R;
    if (i < R * kCols) {
      const bool h = row >= kHalf;
      const int at = h ? first[1] + row - kHalf : first[0] + row, col = s * kCols + q;
      const int64_t off = (h ? m[1].scale_off : m[0].scale_off) +
                          (static_cast<int64_t>(at >> 7) * tiles + col) * 512 + (at & 31) * 16 +
                          ((at >> 5) & 3) * 4;
      cp_async4(sdst + row * (4 * kCols) + q * 4, h ? m[1].scales : m[0].scales, off,
                col < tiles && at < n, h ? m[1].scale_end : m[0].scale_end, status);
    }
  }
}

// Copies stage `s` of `count` rows of x (row r of the stage at offset
// row_off(r), in elements) into `dst`.
template <typename XT, typename RowOff>
__device__ __forceinline__ void load_x(uint32_t dst, const void *x, int64_t extent, int count, int k,
                                       int s, const RowOff &row_off, uint32_t *status) {
  constexpr int kChunk = 16 / sizeof(XT), kChunks = kStageK / kChunk;
  const int lane = threadIdx.x & 31;
  for (int i = lane; i < count * kChunks; i += 32) {
    const int r = i / kChunks, c = i % kChunks;
    const int64_t at = row_off(r) + s * kStageK + c * kChunk;
    cp_async16(dst + r * x_pitch<XT>() + c * 16, x, at * static_cast<int64_t>(sizeof(XT)),
               s * kStageK + c * kChunk < k, extent, status);
  }
}

// ---------------------------------------------------------------- a stage's product

// The activations of one 8-token tile as the product's right operand: b[block]
// holds K elements 8 t .. 8 t + 7 of the 32-block for token g (lane = 4 g + t),
// as FP16 after a multiplication by 2^(14 - floor(log2 max)) of the token's 128.
// Returns the inverse, 2^(floor(log2 max) - 14).
template <typename XT>
__device__ __forceinline__ float x_fragments(uint32_t row, bool valid, uint32_t (&b)[4][4]) {
  const int t = threadIdx.x & 3;
  if constexpr (sizeof(XT) == 2) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 v = valid ? lds128(row + i * 64 + t * 16) : make_uint4(0, 0, 0, 0);
      b[i][0] = v.x, b[i][1] = v.y, b[i][2] = v.z, b[i][3] = v.w;
#pragma unroll
      for (int j = 0; j < 4; j += 2)
        top = __vimax3_u16x2(top, b[i][j] & 0x7FFF7FFFu, b[i][j + 1] & 0x7FFF7FFFu);
    }
    uint32_t e = max(top & 0xFFFFu, top >> 16);
    e = max(e, __shfl_xor_sync(0xFFFFFFFFu, e, 1));
    e = max(e, __shfl_xor_sync(0xFFFFFFFFu, e, 2));
    e = max(e >> 7, 15u);  // exponent field of the largest, kept where both factors are normal
    const uint32_t f = (268u - e) * 0x00800080u;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const uint32_t v = mul_bf16x2(b[i][j], f);
        b[i][j] = pack_f16x2(__uint_as_float(v << 16), __uint_as_float(v & 0xFFFF0000u));
      }
    }
    return __uint_as_float((e - 14u) << 23);
  } else {
    float v[4][8], top = 0.0f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const uint4 q = valid ? lds128(row + i * 128 + t * 32 + j * 16) : make_uint4(0, 0, 0, 0);
        v[i][4 * j] = __uint_as_float(q.x), v[i][4 * j + 1] = __uint_as_float(q.y);
        v[i][4 * j + 2] = __uint_as_float(q.z), v[i][4 * j + 3] = __uint_as_float(q.w);
      }
#pragma unroll
      for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(v[i][j]));
    }
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 1));
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, 2));
    const uint32_t e = max(__float_as_uint(top) >> 23, 15u);
    const float f = __uint_as_float((268u - e) << 23);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
      for (int j = 0; j < 4; ++j) b[i][j] = pack_f16x2(v[i][2 * j] * f, v[i][2 * j + 1] * f);
    }
    return __uint_as_float((e - 14u) << 23);
  }
}

// total += the product of the stage at `st`: element [m][n][i] is row 16 m + g
// (+ 8 for i >= 2), token 8 n + 2 t + (i & 1).
template <int FMT, int MT, int NT, typename XT>
__device__ __forceinline__ void stage_product(uint32_t st, int count, float (&total)[MT][NT][4]) {
  constexpr int R = 16 * MT;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint32_t scales = st + R * 64, xs = scales + R * (FMT == 0 ? 4 : 8);
  uint32_t b[NT][4][4];
  float sx[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const float s = x_fragments<XT>(xs + (8 * n + g) * x_pitch<XT>(), 8 * n + g < count, b[n]);
    sx[n][0] = __shfl_sync(0xFFFFFFFFu, s, t * 8);
    sx[n][1] = __shfl_sync(0xFFFFFFFFu, s, t * 8 + 4);
  }
  // ldmatrix lane addresses: rows l % 8 (+ 8), blocks l / 16 (+ 2)
  const int lrow = (lane & 7) + ((lane >> 3) & 1) * 8;
  const uint32_t lbase = st + lrow * 64 + (((lane >> 4) ^ ((lrow >> 1) & 3)) << 4);
#pragma unroll
  for (int m = 0; m < MT; ++m) {
    float acc[NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[n][0] = acc[n][1] = acc[n][2] = acc[n][3] = 0.0f;
    float s0[4], s1[4];       // MXFP4: scales of rows g, g + 8 for the four blocks
    uint32_t q0[4], q1[4];    // NVFP4: this lane's group scale as FP16 pairs
    if constexpr (FMT == 0) {
      const uint32_t w0 = lds32(scales + (16 * m + g) * 4), w1 = lds32(scales + (16 * m + g + 8) * 4);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const uint32_t p0 = ue8m0x2_bf16x2(w0 >> (16 * i)), p1 = ue8m0x2_bf16x2(w1 >> (16 * i));
        s0[2 * i] = __uint_as_float(p0 << 16), s0[2 * i + 1] = __uint_as_float(p0 & 0xFFFF0000u);
        s1[2 * i] = __uint_as_float(p1 << 16), s1[2 * i + 1] = __uint_as_float(p1 & 0xFFFF0000u);
      }
    } else {
      const uint2 w0 = lds64(scales + (16 * m + g) * 8), w1 = lds64(scales + (16 * m + g + 8) * 8);
      // lanes t = 0, 1 hold the first 16 of a 32-block, t = 2, 3 the second
      const uint32_t pick = t < 2 ? 0x2200u : 0x3311u;
      const uint32_t u[4] = {__byte_perm(w0.x, 0, pick), __byte_perm(w0.y, 0, pick),
                             __byte_perm(w1.x, 0, pick), __byte_perm(w1.y, 0, pick)};
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        q0[2 * i] = e4m3x2_f16x2(u[i]), q0[2 * i + 1] = e4m3x2_f16x2(u[i] >> 16);
        q1[2 * i] = e4m3x2_f16x2(u[2 + i]), q1[2 * i + 1] = e4m3x2_f16x2(u[2 + i] >> 16);
      }
    }
#pragma unroll
    for (int half = 0; half < 2; ++half) {
      uint32_t w[4];  // rows g, g + 8 of block 2 half, then of block 2 half + 1
      ldmatrix_x4((lbase + m * 1024) ^ (half * 32), w);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int blk = 2 * half + i;
        uint32_t a0[4], a1[4];
        e2m1x8_f16(w[2 * i], a0);
        e2m1x8_f16(w[2 * i + 1], a1);
        if constexpr (FMT == 1) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            a0[j] = mul_f16x2(a0[j], q0[blk]);
            a1[j] = mul_f16x2(a1[j], q1[blk]);
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          if constexpr (FMT == 0) {
            const float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            float d[4];
            mma_16816(d, a0[0], a1[0], a0[1], a1[1], b[n][blk][0], b[n][blk][1], zero);
            mma_16816(d, a0[2], a1[2], a0[3], a1[3], b[n][blk][2], b[n][blk][3], d);
            acc[n][0] = __fmaf_rn(s0[blk], d[0], acc[n][0]);
            acc[n][1] = __fmaf_rn(s0[blk], d[1], acc[n][1]);
            acc[n][2] = __fmaf_rn(s1[blk], d[2], acc[n][2]);
            acc[n][3] = __fmaf_rn(s1[blk], d[3], acc[n][3]);
          } else {
            mma_16816(acc[n], a0[0], a1[0], a0[1], a1[1], b[n][blk][0], b[n][blk][1], acc[n]);
            mma_16816(acc[n], a0[2], a1[2], a0[3], a1[3], b[n][blk][2], b[n][blk][3], acc[n]);
          }
        }
      }
    }
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        total[m][n][i] = __fmaf_rn(sx[n][i & 1], acc[n][i], total[m][n][i]);
    }
  }
}

// ---------------------------------------------------------------- joining the warps

// The sums of a CTA's warps: each writes its totals to `red` (float4 [warps][MT NT
// 32]), and after a barrier unit u (= (m NT + n) 32 + lane) is their sum in the
// order of the warps.
template <int MT, int NT>
__device__ __forceinline__ void write_totals(float4 *red, int warp, const float (&total)[MT][NT][4]) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int m = 0; m < MT; ++m) {
#pragma unroll
    for (int n = 0; n < NT; ++n)
      red[(warp * MT * NT + m * NT + n) * 32 + lane] =
          make_float4(total[m][n][0], total[m][n][1], total[m][n][2], total[m][n][3]);
  }
}

template <int UNITS>
__device__ __forceinline__ float4 sum_totals(const float4 *red, int warps, int unit) {
  float4 s = red[unit];
  for (int w = 1; w < warps; ++w) {
    const float4 v = red[w * UNITS + unit];
    s.x += v.x, s.y += v.y, s.z += v.z, s.w += v.w;
  }
  return s;
}

}  // namespace few

__device__ __forceinline__ float bf16_value(const void *p, int64_t i) {
  return __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(p)[i]) << 16);
}

__device__ __forceinline__ uint16_t bf16_bits(float v) {
  uint32_t out;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(out) : "f"(0.0f), "f"(v));
  return static_cast<uint16_t>(out & 0xFFFFu);
}

}  // namespace mx
