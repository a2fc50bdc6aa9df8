// Products of a few tokens with FP4 weights: the core of mx_linear_bf16
// (linear.cu) and of the experts' products (moe.cu).
//
// out[n, t] = sum_k W[n, k] x[t, k] for R = 16 MT weight rows and up to 8 NT
// tokens.  The weights' bytes bound it (4.25 or 4.5 bits each; at 6.8 TB/s an
// SM has to take 45 codes a clock), so the kernel is built to keep weight
// copies in flight and to spend few instructions on a code:
//   - a warp owns a range of K and walks it in stages of 128: codes come by one
//     TMA copy, scales and activations by bulk copies, into the warp's own ring
//     in shared memory, and run on over the end of one tile into the next;
//     warps meet only to add their partial sums;
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
// What bounds the arithmetic is the integer pipe (two instructions a clock per
// SM), where the conversions run: half an instruction a code.
#pragma once

#include <cuda_fp16.h>

#include "mx_device.cuh"
#include "mx_internal.h"

namespace mx {
namespace few {

constexpr int kStageK = 128;  // K elements of a stage

// Bytes of a stage's scales: 512-byte tiles of 128 rows, one (MXFP4) or two
// (NVFP4) for each of the SEGS runs of rows.
template <int FMT, int SEGS>
constexpr int kScaleBytes = (FMT == 0 ? 512 : 1024) * SEGS;

// Codes and scales; a multiple of 512 (the period of the codes' 64-byte swizzle).
template <int FMT, int MT, int SEGS>
constexpr int kStageBytes = 16 * MT * 64 + kScaleBytes<FMT, SEGS>;

// Bytes of a warp's decoded scales: four FP32 (MXFP4) or eight FP16 pairs a row.
template <int FMT, int MT>
constexpr int kDecodedBytes = 16 * MT * (FMT == 0 ? 16 : 32);

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

__device__ __forceinline__ void sts128(uint32_t addr, uint4 v) {
  asm volatile("st.shared.v4.u32 [%0], {%1, %2, %3, %4};" ::"r"(addr), "r"(v.x), "r"(v.y), "r"(v.z),
               "r"(v.w)
               : "memory");
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
__device__ __forceinline__ uint32_t pack_f16x2(float lo, float hi) {
  uint32_t r;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
  return r;
}

// ---------------------------------------------------------------- copies in

// One run of rows of a stage: the codes' map (rows of the whole stack), its
// first row there, and the scales of its matrix.
struct Run {
  const CUtensorMap *codes;
  int code_row;            // first row in the map
  const uint8_t *scales;   // of this matrix
  int row;                 // first row in this matrix
  int64_t scale_end;       // bytes of its scales
};

// A warp's ring of stages, each with a barrier that counts its copies' bytes.
// `abort` (shared by the CTA) is raised when a wait runs out: the copies stop,
// the waits return at once, and the CTA ends after its outstanding copies.
struct Ring {
  uint32_t base, bars;
  int stage_size, slots;
  volatile uint32_t *abort;
  uint32_t *status;
  int put = 0, get = 0;
  uint32_t get_phase = 0;
  int outstanding = 0;

  __device__ __forceinline__ uint32_t stage(int slot) const { return base + slot * stage_size; }

  // Whole warp.  Starts the copies of stage s of 16 MT rows in SEGS runs; tiles:
  // scale tiles along K.
  template <int FMT, int MT, int SEGS>
  __device__ __forceinline__ void fill(const Run (&runs)[SEGS], int s, int tiles) {
    constexpr int kRunRows = 16 * MT / SEGS;
    if (*abort) return;
    const uint32_t dst = stage(put), bar = bars + put * 8;
    const uint32_t scale_bytes = FMT == 0 ? 512u : (tiles - 2 * s > 1 ? 1024u : 512u);
    if (elect_one()) {
      mbar_arrive_expect_tx(bar, 16 * MT * 64 + SEGS * scale_bytes);
#pragma unroll
      for (int i = 0; i < SEGS; ++i) {
        tma_load_2d(dst + i * kRunRows * 64, runs[i].codes, s * 64, runs[i].code_row, bar);
        const int64_t off = (static_cast<int64_t>(runs[i].row >> 7) * tiles +
                             s * (FMT == 0 ? 1 : 2)) * 512;
        bulk_load(dst + 16 * MT * 64 + i * kScaleBytes<FMT, 1>,
                  runs[i].scales + (in_bounds(off, scale_bytes, runs[i].scale_end, status) ? off : 0),
                  scale_bytes, bar);
      }
    }
    if (++put == slots) put = 0;
    ++outstanding;
  }

  // Whole warp.  Waits for the next stage; false when a wait ran out.
  __device__ __forceinline__ bool wait() {
    return mbar_wait_warp(bars + get * 8, get_phase, abort, status);
  }

  // The stage that wait() gave is read (after a __syncwarp it may be filled again).
  __device__ __forceinline__ void next() {
    --outstanding;
    if (++get == slots) get = 0, get_phase ^= 1u;
  }

  // After an abort: no copy may still be writing when the CTA ends.
  __device__ __forceinline__ void drain() {
    for (; outstanding > 0; next()) mbar_drain(bars + get * 8, get_phase);
  }
};

// ---------------------------------------------------------------- a stage's product

// The activations in shared memory: FP16 [token][K of the slice], rows `pitch`
// bytes apart, and for each stage of 128 the tokens' factors.  The padding of a
// row makes a quarter warp's 16-byte reads (two tokens) fall on distinct banks.
__host__ __device__ constexpr int x_pitch(int stages) { return stages * kStageK * 2 + 64; }

// Whole CTA (W warps).  Writes `count` rows of x, K elements [k0, k0 + 128
// stages), as FP16 at xs: each 128 times 2^(14 - floor(log2 max)), and the
// inverse to factors[stage * kTokens + token].  Elements at or past k are 0.
// row(i): the i-th row; extent: elements of x from its base (bounds-checked
// build).  A half warp takes 128 elements, eight a lane.
template <typename XT, int W, int kTokens, typename Row>
__device__ __forceinline__ void stage_x(uint32_t xs, float *factors, const void *x, int64_t extent,
                                        int count, int stages, int k0, int k, const Row &row,
                                        uint32_t *status) {
  constexpr int kBatch = sizeof(XT) == 2 ? 8 : 4;  // tasks whose loads are in flight
  const int half = threadIdx.x >> 4, l = threadIdx.x & 15;
  const int tasks = count * stages, pitch = x_pitch(stages);
  // task / stages by a multiplication (tasks * stages < 2^32)
  const uint32_t inv = (0xFFFFFFFFu / stages) + 1u;
  const auto token = [&](int task) {
    return stages == 1 ? task : static_cast<int>(__umulhi(static_cast<uint32_t>(task), inv));
  };
  for (int base = 0; base < tasks; base += kBatch * 2 * W) {
    uint4 raw[kBatch][sizeof(XT) / 2];
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int task = base + j * 2 * W + half;
      const int r = token(task), at = k0 + (task - r * stages) * kStageK + l * 8;
#pragma unroll
      for (int q = 0; q < static_cast<int>(sizeof(XT) / 2); ++q) raw[j][q] = make_uint4(0, 0, 0, 0);
      if (task < tasks && at < k) {
        const int64_t off = row(r) + at;
        if (in_bounds(off, 8, extent, status)) {
          const uint4 *p = reinterpret_cast<const uint4 *>(static_cast<const XT *>(x) + off);
#pragma unroll
          for (int q = 0; q < static_cast<int>(sizeof(XT) / 2); ++q) raw[j][q] = p[q];
        }
      }
    }
#pragma unroll
    for (int j = 0; j < kBatch; ++j) {
      const int task = base + j * 2 * W + half;
      float v[8];
      if constexpr (sizeof(XT) == 2) {
        const uint32_t w[4] = {raw[j][0].x, raw[j][0].y, raw[j][0].z, raw[j][0].w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[2 * i] = __uint_as_float(w[i] << 16);
          v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
        }
      } else {
#pragma unroll
        for (int q = 0; q < 2; ++q) {
          v[4 * q] = __uint_as_float(raw[j][q].x), v[4 * q + 1] = __uint_as_float(raw[j][q].y);
          v[4 * q + 2] = __uint_as_float(raw[j][q].z), v[4 * q + 3] = __uint_as_float(raw[j][q].w);
        }
      }
      float top = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) top = fmaxf(top, fabsf(v[i]));
#pragma unroll
      for (int m = 8; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, m));
      // exponent field of the largest, kept where both factors are normal
      const uint32_t e = max(__float_as_uint(top) >> 23, 15u);
      const float f = __uint_as_float((268u - e) << 23);
      if (task < tasks) {
        const int r = token(task), s = task - r * stages;
        sts128(xs + r * pitch + s * (kStageK * 2) + l * 16,
               make_uint4(pack_f16x2(v[0] * f, v[1] * f), pack_f16x2(v[2] * f, v[3] * f),
                          pack_f16x2(v[4] * f, v[5] * f), pack_f16x2(v[6] * f, v[7] * f)));
        if (l == 0) factors[s * kTokens + r] = __uint_as_float((e - 14u) << 23);
      }
    }
  }
}

// Decodes the scales of a stage (`raw`: SEGS runs of 512-byte tiles) once for
// the warp: row r of the 16 MT gets its scales of the stage at dec, as four FP32
// (MXFP4) or, for each half of a 32-block, four FP16 pairs (NVFP4).  A 16-byte
// row of a tile holds the words of rows l, l + 32, l + 64, l + 96; run i starts
// at row first[i] of its matrix.
// Blocks past K (`blocks` of the four are inside) get the scale 0: their codes
// are 0, but the bytes there need not be.
template <int FMT, int MT, int SEGS>
__device__ __forceinline__ void decode_scales(uint32_t raw, const int (&first)[SEGS], int blocks,
                                              uint32_t dec) {
  constexpr int kRunRows = 16 * MT / SEGS;
  constexpr int kWordBlocks = FMT == 0 ? 4 : 2;  // 32-blocks of a word
  const uint32_t keep0 = blocks >= kWordBlocks ? ~0u : (1u << (32 / kWordBlocks * blocks)) - 1u;
  const uint32_t keep1 = blocks >= 4 ? ~0u : blocks <= 2 ? 0u : 0xFFFFu;  // NVFP4's second word
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int i = 0; i < SEGS; ++i) {
#pragma unroll
    for (int r0 = 0; r0 < kRunRows; r0 += 32) {
      if (kRunRows < 32 && lane >= kRunRows) continue;
      const int in_tile = (first[i] & 127) + r0 + lane;  // a run does not cross a tile
      const uint32_t at = raw + i * kScaleBytes<FMT, 1> + (in_tile & 31) * 16 + (in_tile >> 5) * 4;
      const uint32_t row = i * kRunRows + r0 + lane;
      if constexpr (FMT == 0) {
        const uint32_t w = lds32(at) & keep0;
        const uint32_t p = ue8m0x2_bf16x2(w), q = ue8m0x2_bf16x2(w >> 16);
        sts128(dec + row * 16, make_uint4(p << 16, p & 0xFFFF0000u, q << 16, q & 0xFFFF0000u));
      } else {
        const uint32_t w0 = lds32(at) & keep0, w1 = lds32(at + 512) & keep1;
        const uint32_t a = e4m3x2_f16x2(w0), b = e4m3x2_f16x2(w0 >> 16), c = e4m3x2_f16x2(w1),
                       d = e4m3x2_f16x2(w1 >> 16);
        sts128(dec + row * 32, make_uint4(__byte_perm(a, 0, 0x1010), __byte_perm(b, 0, 0x1010),
                                          __byte_perm(c, 0, 0x1010), __byte_perm(d, 0, 0x1010)));
        sts128(dec + row * 32 + 16,
               make_uint4(__byte_perm(a, 0, 0x3232), __byte_perm(b, 0, 0x3232),
                          __byte_perm(c, 0, 0x3232), __byte_perm(d, 0, 0x3232)));
      }
    }
  }
  __syncwarp();
}

// total += the product of the stage at `st` (scales decoded at `dec`) and the
// activations at `xs` (`count` tokens, rows `pitch` apart, factors at `sx`):
// element [m][n][i] is row 16 m + g (+ 8 for i >= 2), token 8 n + 2 t + (i & 1),
// lane = 4 g + t.  Lane t holds K elements 8 t .. 8 t + 7 of each 32-block, of
// the codes and of x alike.
template <int FMT, int MT, int NT, int NTM>
__device__ __forceinline__ void stage_product(uint32_t st, uint32_t dec, uint32_t xs, int pitch,
                                              uint32_t sx, int count, float (&total)[MT][NTM][4]) {
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  // ldmatrix lane addresses: rows l % 8 (+ 8), blocks l / 16 (+ 2)
  const int lrow = (lane & 7) + ((lane >> 3) & 1) * 8;
  const uint32_t lbase = st + lrow * 64 + (((lane >> 4) ^ ((lrow >> 1) & 3)) << 4);
  float acc[MT][NT][4];
#pragma unroll
  for (int m = 0; m < MT; ++m) {
#pragma unroll
    for (int n = 0; n < NT; ++n) acc[m][n][0] = acc[m][n][1] = acc[m][n][2] = acc[m][n][3] = 0.0f;
  }
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    uint4 b[NT][2];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        b[n][i] = make_uint4(0, 0, 0, 0);
        if (8 * n + g < count)
          b[n][i] = lds128(xs + (8 * n + g) * pitch + (2 * half + i) * 64 + t * 16);
      }
    }
#pragma unroll
    for (int m = 0; m < MT; ++m) {
      uint32_t w[4];  // rows g, g + 8 of block 2 half, then of block 2 half + 1
      ldmatrix_x4((lbase + m * 1024) ^ (half * 32), w);
      // scales of rows g and g + 8 for the two blocks: FP32 (MXFP4), or this
      // lane's half of each block as FP16 pairs (NVFP4)
      constexpr int kRow = FMT == 0 ? 16 : 32;
      const uint32_t at = dec + (16 * m + g) * kRow + (FMT == 0 ? 0 : (t >> 1) * 16) + half * 8;
      const uint2 s0 = lds64(at), s1 = lds64(at + 8 * kRow);
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        uint32_t a0[4], a1[4];
        e2m1x8_f16(w[2 * i], a0);
        e2m1x8_f16(w[2 * i + 1], a1);
        const uint32_t q0 = i == 0 ? s0.x : s0.y, q1 = i == 0 ? s1.x : s1.y;
        if constexpr (FMT == 1) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            a0[j] = mul_f16x2(a0[j], q0);
            a1[j] = mul_f16x2(a1[j], q1);
          }
        }
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float(&c)[4] = acc[m][n];
          if constexpr (FMT == 0) {
            const float zero[4] = {0.0f, 0.0f, 0.0f, 0.0f};
            float d[4];
            mma_16816(d, a0[0], a1[0], a0[1], a1[1], b[n][i].x, b[n][i].y, zero);
            mma_16816(d, a0[2], a1[2], a0[3], a1[3], b[n][i].z, b[n][i].w, d);
            c[0] = __fmaf_rn(__uint_as_float(q0), d[0], c[0]);
            c[1] = __fmaf_rn(__uint_as_float(q0), d[1], c[1]);
            c[2] = __fmaf_rn(__uint_as_float(q1), d[2], c[2]);
            c[3] = __fmaf_rn(__uint_as_float(q1), d[3], c[3]);
          } else {
            mma_16816(c, a0[0], a1[0], a0[1], a1[1], b[n][i].x, b[n][i].y, c);
            mma_16816(c, a0[2], a1[2], a0[3], a1[3], b[n][i].z, b[n][i].w, c);
          }
        }
      }
    }
  }
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const uint2 f = lds64(sx + (8 * n + 2 * t) * 4);
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int i = 0; i < 4; ++i)
        total[m][n][i] =
            __fmaf_rn(__uint_as_float(i & 1 ? f.y : f.x), acc[m][n][i], total[m][n][i]);
    }
  }
}

// ---------------------------------------------------------------- the whole walk

// How a CTA's W warps and its shared memory serve its items.  An item is
// 16 MT rows_w rows times a group's tokens; rows_w warps stand side by side along
// the rows, the W / rows_w others along K.  Up to `batch` items of a group are
// taken together, and x is held `x_stages` stages of K at a time: the slices are
// the outer loop, so that x is converted once for a batch, and the sums of a
// batch's items wait in shared memory from slice to slice.
struct Split {
  int rows_w;
  int x_stages;
  int batch;
};

// Shared memory of a CTA, in order: the warps' rings, the warps' sums [batch][W]
// (the decoded scales of the item at work lie in its own part: its sums are in
// registers meanwhile), barriers and the abort flag, factors and activations.
template <int FMT, int MT, int NT, int SEGS, int W, int S>
struct Layout {
  static constexpr int kRing = W * S * kStageBytes<FMT, MT, SEGS>;
  static constexpr int kWarpRed = MT * NT * 512;
  static_assert(kDecodedBytes<FMT, MT> <= kWarpRed, "the decoded scales' place");
  static constexpr int kBars = W * S * 8 + 16;
  static int total(int tokens, const Split &s) {
    return kRing + s.batch * W * kWarpRed + kBars + tokens * x_pitch(s.x_stages) +
           s.x_stages * NT * 8 * 4;
  }
  // The split for `items` items a CTA (at rows_w = 1) of `stages` stages: along K
  // while every warp has at least `least` stages, else along the rows; as many
  // items together as a CTA has (if the sums of all K do not come at once); all
  // of x where it fits.
  static Split split(int tokens, int stages, int least, int items, int bytes) {
    Split s{1, 0, 1};
    while (s.rows_w < W && stages < least * (W / s.rows_w)) s.rows_w *= 2;
    items = (items + s.rows_w - 1) / s.rows_w;
    const auto fitting = [&](int batch) {
      return (bytes - kRing - batch * W * kWarpRed - kBars - tokens * 64) /
             (tokens * kStageK * 2 + NT * 8 * 4);
    };
    s.x_stages = fitting(1);
    if (s.x_stages >= stages) {
      s.x_stages = stages;
      while (s.batch < 2 && s.batch < items && fitting(s.batch + 1) >= stages) ++s.batch;
      return s;
    }
    while (s.batch < items && fitting(s.batch + 1) >= W / s.rows_w) ++s.batch;
    // whole rounds of the warps along K
    s.x_stages = fitting(s.batch);
    if (s.x_stages > W / s.rows_w) s.x_stages = s.x_stages / (W / s.rows_w) * (W / s.rows_w);
    return s;
  }
};

// Walks this CTA's items.  Policy gives
//   start(item, end)     whole CTA, once, after the set-up that touches no global
//                        memory: waits for the previous kernel, sets the items
//   group(item)          the tokens' group (items of a group are consecutive)
//   count(item)          its tokens (<= 8 NT)
//   row_off(item, i)     offset in x (elements) of its i-th token
//   runs(item, wr, runs) the rows of row-warp wr
//   put(item, wr, m, n, lane, sums)  the four sums (or, with SEGS == 2, those of
//                        the first run's and of the second run's rows) of a unit
// The warps meet where activations are staged, and, if K is divided among them,
// around the sums of a batch.
template <int FMT, int MT, int NT, int SEGS, int W, int S, typename XT, typename Policy>
__device__ __forceinline__ void walk(char *smem, Policy &policy, const void *x, int64_t x_extent,
                                     int k, const Split &split, uint32_t *status) {
  using L = Layout<FMT, MT, NT, SEGS, W, S>;
  constexpr int kUnits = MT * NT * 32;  // float4 of a warp's sums
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int wr = warp % split.rows_w, wk = warp / split.rows_w, kw = W / split.rows_w;
  char *at = smem + L::kRing;
  float4 *red = reinterpret_cast<float4 *>(at);
  at += split.batch * W * L::kWarpRed;
  const uint32_t bars = smem_u32(at);
  volatile uint32_t *abort = reinterpret_cast<volatile uint32_t *>(at + W * S * 8);
  at += L::kBars;
  const uint32_t factors = smem_u32(at);
  const uint32_t xs = factors + split.x_stages * NT * 8 * 4;
  if (threadIdx.x == 0) *abort = 0;
  if (threadIdx.x < W * S) mbar_init(bars + threadIdx.x * 8, 1);
  fence_barrier_init();
  Ring ring{smem_u32(smem) + warp * S * kStageBytes<FMT, MT, SEGS>, bars + warp * S * 8,
            kStageBytes<FMT, MT, SEGS>, S, abort, status};

  const int stages = (k + kStageK - 1) / kStageK, tiles = (k / (FMT == 0 ? 32 : 16) + 3) >> 2;
  const int slices = (stages + split.x_stages - 1) / split.x_stages;
  // this warp's stages of slice i: [lo, hi)
  const auto share = [&](int i, int &lo, int &hi) {
    const int first = i * split.x_stages, len = min(split.x_stages, stages - first);
    lo = first + len * wk / kw;
    hi = first + len * (wk + 1) / kw;
  };
  int item = 0, item_end = 0;
  // items of the batch that begins at `first`
  const auto batch_of = [&](int first) {
    int n = 1;
    while (n < split.batch && first + n < item_end && policy.group(first + n) == policy.group(first))
      ++n;
    return n;
  };
  // the copies' place in the warp's sequence of batches, slices, items and
  // stages, ahead of the product's
  int put_first = 0, put_n = 0, put_i = 0, put_slice = 0, put_s = 0, put_lo = 0, put_hi = 0;
  Run put_runs[SEGS];
  const auto fill = [&]() {
    while (put_first < item_end && put_s == put_hi) {
      if (++put_i == put_n) {
        put_i = 0;
        if (++put_slice == slices) {
          put_slice = 0;
          put_first += put_n;
          if (put_first >= item_end) break;
          put_n = batch_of(put_first);
        }
        share(put_slice, put_lo, put_hi);
      }
      put_s = put_lo;
      if (put_n > 1 || put_slice == 0) policy.runs(put_first + put_i, wr, put_runs);
    }
    if (put_first < item_end) ring.fill<FMT, MT, SEGS>(put_runs, put_s++, tiles);
  };
  __syncthreads();
  policy.start(item, item_end);
  put_first = item;
  share(0, put_lo, put_hi);
  put_s = put_lo;
  if (put_first < item_end) {
    put_n = batch_of(put_first);
    policy.runs(put_first, wr, put_runs);
  }
  if (slices == 1 && put_lo == put_hi) put_first = item_end;  // no share of K
  for (int i = 0; i < S - 1; ++i) fill();

  int staged = -1;
  while (item < item_end) {
    const int n_items = batch_of(item), count = policy.count(item), group = policy.group(item);
    for (int slice = 0; slice < slices; ++slice) {
      const int len = min(split.x_stages, stages - slice * split.x_stages);
      if (slices > 1 || group != staged) {
        if (staged >= 0) __syncthreads();
        stage_x<XT, W, 8 * NT>(xs, reinterpret_cast<float *>(at), x, x_extent, count, len,
                               slice * split.x_stages * kStageK, k,
                               [&](int i) { return policy.row_off(item, i); }, status);
        __syncthreads();
        staged = group;
      }
      const int pitch = x_pitch(len);
      int lo, hi;
      share(slice, lo, hi);
      for (int i = 0; i < n_items; ++i) {
        float4 *sums = red + (i * W + warp) * kUnits;
        const uint32_t dec = smem_u32(sums);
        Run runs[SEGS];
        policy.runs(item + i, wr, runs);
        int first[SEGS];
#pragma unroll
        for (int j = 0; j < SEGS; ++j) first[j] = runs[j].row;
        float total[MT][NT][4];
#pragma unroll
        for (int m = 0; m < MT; ++m) {
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            const float4 v = slice == 0 ? make_float4(0.0f, 0.0f, 0.0f, 0.0f)
                                        : sums[(m * NT + n) * 32 + lane];
            total[m][n][0] = v.x, total[m][n][1] = v.y, total[m][n][2] = v.z, total[m][n][3] = v.w;
          }
        }
        __syncwarp();
        for (int s = lo; s < hi; ++s) {
          const bool ok = ring.wait();
          fill();
          if (!ok) break;
          const uint32_t st = ring.stage(ring.get);
          decode_scales<FMT, MT, SEGS>(st + 16 * MT * 64, first, min((k >> 5) - 4 * s, 4), dec);
          const int sl = s - slice * split.x_stages;
          const uint32_t sx = factors + sl * NT * 8 * 4, xa = xs + sl * kStageK * 2;
          if (NT == 1 || count > (NT == 4 ? 16 : 8))
            stage_product<FMT, MT, NT, NT>(st, dec, xa, pitch, sx, count, total);
          else if (NT == 4 && count > 8)
            stage_product<FMT, MT, (NT == 4 ? 2 : 1), NT>(st, dec, xa, pitch, sx, count, total);
          else
            stage_product<FMT, MT, 1, NT>(st, dec, xa, pitch, sx, count, total);
          ring.next();
          __syncwarp();
        }
#pragma unroll
        for (int m = 0; m < MT; ++m) {
#pragma unroll
          for (int n = 0; n < NT; ++n)
            sums[(m * NT + n) * 32 + lane] =
                make_float4(total[m][n][0], total[m][n][1], total[m][n][2], total[m][n][3]);
        }
      }
    }
    // the warps' sums, added in the order of the warps
    constexpr int kM = MT / SEGS;
    const int col_tiles = (count + 7) / 8;
    const auto add = [&](int i, int r, int unit) {
      float4 v = red[(i * W + r) * kUnits + unit];
      for (int w = r + split.rows_w; w < W; w += split.rows_w) {
        const float4 o = red[(i * W + w) * kUnits + unit];
        v.x += o.x, v.y += o.y, v.z += o.z, v.w += o.w;
      }
      return v;
    };
    // kw == 1: a warp's sums are its own
    if (kw > 1) __syncthreads();
    const int step = kw > 1 ? W : 1;
    for (int i = 0; i < n_items; ++i) {
      const int units = (kw > 1 ? split.rows_w : 1) * kM * col_tiles;
      for (int u = kw > 1 ? warp : 0; u < units; u += step) {
        const int n = u % col_tiles, q = u / col_tiles, m = q % kM;
        const int r = kw > 1 ? q / kM : wr;
        float4 v[SEGS];
#pragma unroll
        for (int j = 0; j < SEGS; ++j) v[j] = add(i, r, ((m + j * kM) * NT + n) * 32 + lane);
        policy.put(item + i, r, m, n, lane, v);
      }
    }
    if (kw > 1) __syncthreads();
    item += n_items;
  }
  ring.drain();
}

constexpr int kMaxSmem = 227 * 1024;

}  // namespace few

}  // namespace mx
