// mx_linear_bf16: a few BF16 rows times an FP4 weight.
//
// y[t, n] = sum_k W[n, k] x[t, k] for up to 8 NT tokens.  Two kernels; the rule that
// chooses (linear_mma_better) has both sides' times.  This one is for the smaller
// calls, where a launch and one pass of dependent steps are what counts:
//   - an item is R = 16 MT weight rows; the CTA's warps divide K, each walks its range
//     in stages of 128 that come by cp.async into a ring of its own, over the end
//     of one item into the next; the warps meet only to add their sums;
//   - with fewer items than SMs the CTAs of a cluster divide K and add their sums
//     through each other's shared memory (1 x 1024 x 8192: 7.3 us, so 4.9; 13 x 1312 x
//     25408 NVFP4 31.7 us, so 14.7);
//   - E2M1 becomes FP16 by the conversion instruction, two codes at once, and
//     multiplies on the 16 x 8 x 16 FP16 product with binary32 sums, the weights on
//     its 16-row side (measured: 90 codes a clock per SM converted, 128 multiplied);
//   - MXFP4 scales apply to the sum of a 32-block, the E4M3 scales of NVFP4 to the FP16
//     weights (code * scale has 6 bits: exact);
//   - activations become FP16 times a power of two for each (token, 128): BF16
//     values keep all their bits unless they lie 2^-31 below the largest of the 128.
//     The sums of a block are then up to 2^22.6, with which a UE8M0 scale above 2^104
//     overflows, as may the whole sum before a small tensor scale: an output that is not
//     finite is summed again with more range (wide_sum).
// It issues about 2.5 instructions a code, which bounds it at 4 TB/s of weights
// for up to 8 tokens (8 x 28672 x 8192: 32 us); linear_mma.cu leaves the weights to the
// tensor cores.  At 8 x 4096 x 4096 (5.0 us; its bytes 1.4) latency bounds it: a launch,
// two rounds of copies from memory, the join of the warps.  Above 16 tokens instructions do
// (32 x 4096 x 4096: 12.8 us): every item of 32 rows converts all of x again, as many
// elements as weights, and shared memory holds two stages a warp.
#include <cuda_fp16.h>

#include "few_tokens.cuh"

namespace mx {
namespace {

constexpr int kMaxSmem = 227 * 1024;
constexpr int kStageK = 128;  // K elements of a stage

// Bytes of a token's row in a stage, padded so that a quarter warp's 16-byte reads
// (two tokens) fall on distinct banks.
constexpr int kXPitch = 256 + 64;

// Codes, scales, activations; a multiple of 64 (stage_product steps between chunks
// by flipping address bits).
template <int FMT, int MT>
constexpr int stage_bytes(int tokens) {
  return (16 * MT * (64 + (FMT == 0 ? 4 : 8)) + tokens * kXPitch + 63) / 64 * 64;
}

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

__device__ __forceinline__ void cp_async_commit() {
  asm volatile("cp.async.commit_group;" ::: "memory");
}

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
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
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

// Copies the codes and scales of stage `s` of the R = 16 MT rows from row0 into
// `dst`; rows at or past n and blocks of K at or past k become zeros.
template <int FMT, int MT>
__device__ __forceinline__ void load_weights(uint32_t dst, const LinearArgs &a, int64_t row0, int s) {
  constexpr int R = 16 * MT;
  const int lane = threadIdx.x & 31;
  // codes: 64 bytes of a row in four 16-byte chunks (one 32-block each), chunk c
  // of row r at c ^ (r / 2 % 4): ldmatrix then reads without bank conflicts
  const int chunk = lane & 3, r0 = lane >> 2;
  const int64_t ldb = a.k >> 1;
  const bool k_in = s * kStageK + chunk * 32 < a.k;
#pragma unroll
  for (int j = 0; j < R / 8; ++j) {
    const int row = r0 + j * 8;
    cp_async16(dst + row * 64 + ((chunk ^ ((row >> 1) & 3)) << 4), a.w.codes,
               (row0 + row) * ldb + (s * 64 + chunk * 16), k_in && row0 + row < a.n, a.n * ldb,
               a.status);
  }
  // scales: the four (MXFP4) or eight bytes of a row, one tile column each word
  constexpr int kCols = FMT == 0 ? 1 : 2;
  const int tiles = static_cast<int>((a.k / (FMT == 0 ? 32 : 16) + 3) >> 2);
  const int64_t extent = ((a.n + 127) >> 7) * tiles * 512;
  const uint32_t sdst = dst + R * 64;
#pragma unroll
  for (int i0 = 0; i0 < R * kCols; i0 += 32) {
    const int row = (i0 + lane) % R, q = (i0 + lane) / R;
    const int64_t at = row0 + row;
    const int col = s * kCols + q;
    cp_async4(sdst + row * (4 * kCols) + q * 4, a.w.scales,
              ((at >> 7) * tiles + col) * 512 + (at & 31) * 16 + ((at >> 5) & 3) * 4,
              col < tiles && at < a.n, extent, a.status);
  }
}

// Copies stage `s` of x into `dst`.
__device__ __forceinline__ void load_x(uint32_t dst, const LinearArgs &a, int s) {
  const int lane = threadIdx.x & 31;
  for (int i = lane; i < a.tokens * 16; i += 32) {
    const int r = i >> 4, at = s * kStageK + (i & 15) * 8;
    cp_async16(dst + r * kXPitch + (i & 15) * 16, a.x, (r * a.ld_x + at) * 2, at < a.k,
               ((a.tokens - 1) * a.ld_x + a.k) * 2, a.status);
  }
}

// The activations of one 8-token tile as the product's right operand: b[block]
// holds K elements 8 t .. 8 t + 7 of the 32-block for token g (lane = 4 g + t),
// as FP16 after a multiplication by 2^(14 - floor(log2 max)) of the token's 128.
// Returns the inverse, 2^(floor(log2 max) - 14).
__device__ __forceinline__ float x_fragments(uint32_t row, bool valid, uint32_t (&b)[4][4]) {
  const int t = threadIdx.x & 3;
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
}

// total += the product of the stage at `st`: element [m][n][i] is row 16 m + g
// (+ 8 for i >= 2), token 8 n + 2 t + (i & 1).
template <int FMT, int MT, int NT>
__device__ __forceinline__ void stage_product(uint32_t st, int count, float (&total)[MT][NT][4]) {
  constexpr int R = 16 * MT;
  const int lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const uint32_t scales = st + R * 64, xs = scales + R * (FMT == 0 ? 4 : 8);
  uint32_t b[NT][4][4];
  float sx[NT][2];
#pragma unroll
  for (int n = 0; n < NT; ++n) {
    const float s = x_fragments(xs + (8 * n + g) * kXPitch, 8 * n + g < count, b[n]);
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

constexpr int kMaxCtas = 8;  // of a cluster

// CTAs of a cluster for `tiles` tiles: at least two stages a warp.
int cluster_ctas(int warps, int64_t tiles, int64_t k, int num_sms) {
  const int64_t stages = (k + kStageK - 1) / kStageK;
  int64_t c = num_sms / tiles;
  if (c > stages / (2 * warps)) c = stages / (2 * warps);
  return static_cast<int>(c < 1 ? 1 : c > kMaxCtas ? kMaxCtas : c);
}

struct LinearParams {
  LinearArgs a;
  int tiles;  // row tiles of 16 MT rows
  int ctas;   // of a cluster
};

// Persistent over row tiles: tile blockIdx.x, + gridDim.x, ...  Each of the W
// warps takes its share of K in every tile.
template <int FMT, int MT, int NT, int W, int S>
__global__ void __launch_bounds__(W * 32, 1) linear_kernel(const __grid_constant__ LinearParams p) {
  extern __shared__ __align__(128) char smem[];
  constexpr int R = 16 * MT, kUnits = MT * NT * 32;
  const LinearArgs &a = p.a;
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5;
  const int stage_size = stage_bytes<FMT, MT>(a.tokens);
  float4 *red = reinterpret_cast<float4 *>(smem);
  const uint32_t ring = smem_u32(smem) + W * kUnits * 16 + warp * S * stage_size;
  const int all = static_cast<int>((a.k + kStageK - 1) / kStageK);
  const int rank = p.ctas > 1 ? static_cast<int>(cluster_ctarank()) : 0;
  const int first_tile = blockIdx.x / p.ctas, tile_step = gridDim.x / p.ctas;
  const int share = rank * W + warp, shares = p.ctas * W;  // of K
  const int s_begin = static_cast<int>(static_cast<int64_t>(all) * share / shares);
  const int s_end = static_cast<int>(static_cast<int64_t>(all) * (share + 1) / shares);

  // the copies' place: tile and stage, ahead of the product's
  int ptile = first_tile, ps = s_begin, pslot = 0;
  const auto issue = [&]() {
    if (s_begin < s_end && ptile < p.tiles) {
      const uint32_t dst = ring + pslot * stage_size;
      load_weights<FMT, MT>(dst, a, static_cast<int64_t>(ptile) * R, ps);
      load_x(dst + R * (64 + (FMT == 0 ? 4 : 8)), a, ps);
      if (++ps == s_end) ps = s_begin, ptile += tile_step;
      if (++pslot == S) pslot = 0;
    }
    cp_async_commit();
  };

  griddep_wait();
#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue();
  const float alpha = FMT == 1 ? *a.w.ts : 1.0f;
  int slot = 0;
  for (int tile = first_tile; tile < p.tiles; tile += tile_step) {
    float total[MT][NT][4] = {};
    for (int s = s_begin; s < s_end; ++s) {
      cp_async_wait<S - 2>();
      __syncwarp();
      issue();
      stage_product<FMT, MT, NT>(ring + slot * stage_size, a.tokens, total);
      if (++slot == S) slot = 0;
    }
    // the warps' sums, added in the order of the warps
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int m = 0; m < MT; ++m) {
#pragma unroll
      for (int n = 0; n < NT; ++n)
        red[(warp * MT * NT + m * NT + n) * 32 + lane] =
            make_float4(total[m][n][0], total[m][n][1], total[m][n][2], total[m][n][3]);
    }
    __syncthreads();
    if (p.ctas > 1) cluster_sync();
    // (of a cluster each CTA takes a part of the outputs)
    for (int u = threadIdx.x * p.ctas + rank; u < kUnits; u += W * 32 * p.ctas) {
      float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
      for (int c = 0; c < p.ctas; ++c) {
        float4 o[W];
#pragma unroll
        for (int w = 0; w < W; ++w) {
          const float4 *from = red + w * kUnits + u;
          o[w] = p.ctas > 1 ? ld_cluster_f32x4(mapa_shared(smem_u32(from), static_cast<uint32_t>(c)))
                            : *from;
        }
#pragma unroll
        for (int w = 0; w < W; ++w) v.x += o[w].x, v.y += o[w].y, v.z += o[w].z, v.w += o[w].w;
      }
      const int ul = u & 31, mn = u >> 5;
      const int64_t row0 = static_cast<int64_t>(tile) * R + (mn / NT) * 16 + (ul >> 2);
      const int col0 = (mn % NT) * 8 + (ul & 3) * 2;
      float f[4] = {v.x, v.y, v.z, v.w};
      const auto in = [&](int i) { return row0 + (i >> 1) * 8 < a.n && col0 + (i & 1) < a.tokens; };
      bool finite = true;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (FMT == 1) f[i] *= alpha;
        finite = finite && fabsf(f[i]) < __uint_as_float(0x7F800000u);
      }
      if (!finite) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          if (in(i) && !(fabsf(f[i]) < __uint_as_float(0x7F800000u)))
            f[i] = wide_sum<FMT>(a, row0 + (i >> 1) * 8, col0 + (i & 1));
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i)
        if (in(i)) put_linear(a, row0 + (i >> 1) * 8, col0 + (i & 1), f[i]);
    }
    __syncwarp();  // (an output may have taken some lanes through wide_sum)
    if (p.ctas > 1)
      cluster_sync();
    else
      __syncthreads();
  }
}

template <int FMT, int MT, int NT, int W, int S>
cudaError_t launch(const LinearArgs &a, cudaStream_t s) {
  const auto kernel = linear_kernel<FMT, MT, NT, W, S>;
  const void *func = reinterpret_cast<const void *>(kernel);
  if (!kernel_setup_get(func, nullptr)) {
    const cudaError_t e =
        cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e != cudaSuccess) return e;
    kernel_setup_put(func, 0);
  }
  size_t smem = W * MT * NT * 512 + static_cast<size_t>(W) * S * stage_bytes<FMT, MT>(a.tokens);
  // One CTA an SM: two on one, launched while the kernel before it still holds the
  // others, share what one SM can do (1 x 4096 x 8192: 11.9 us, so 8.1).
  if (smem <= kMaxSmem / 2) smem = kMaxSmem / 2 + 1024;
  LinearParams p{a, static_cast<int>((a.n + 16 * MT - 1) / (16 * MT)), 1};
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.blockDim = dim3(W * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  // Fewer tiles than SMs: the CTAs of a cluster divide K, so many as leave every tile a
  // cluster at once (a cluster lies within a part of the GPU: fewer fit than SMs / CTAs).
  for (p.ctas = cluster_ctas(W, p.tiles, a.k, a.num_sms); p.ctas > 1; --p.ctas) {
    static const char keys[kMaxCtas + 1] = {};  // their addresses name the instance and count
    int fit = 0;
    attr[1].val.clusterDim.x = static_cast<unsigned>(p.ctas);
    cfg.gridDim = dim3(static_cast<unsigned>(p.ctas));
    cfg.numAttrs = 2;
    if (!kernel_setup_get(&keys[p.ctas], &fit)) {
      // (the most shared memory the instance can ask for, so that the answer holds)
      cfg.dynamicSmemBytes = kMaxSmem;
      const cudaError_t e = cudaOccupancyMaxActiveClusters(&fit, kernel, &cfg);
      if (e != cudaSuccess) return e;
      cfg.dynamicSmemBytes = smem;
      kernel_setup_put(&keys[p.ctas], fit);
    }
    if (fit >= p.tiles) break;
  }
  const int clusters = p.tiles < a.num_sms ? p.tiles : a.num_sms;
  cfg.gridDim = dim3(static_cast<unsigned>(clusters * p.ctas));
  cfg.numAttrs = p.ctas > 1 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, kernel, p);
}

// Rows of an item: 64 where every SM gets one, else 32.
bool tall_items(int64_t tokens, int64_t n, int num_sms) {
  return tokens <= 16 && n >= 64 * static_cast<int64_t>(num_sms);
}

// Warps and depth of the rings: what shared memory holds.
template <int FMT>
cudaError_t launch_fmt(const LinearArgs &a, cudaStream_t s) {
  const bool tall = tall_items(a.tokens, a.n, a.num_sms);
  if (a.tokens <= 8) return tall ? launch<FMT, 4, 1, 8, 3>(a, s) : launch<FMT, 2, 1, 8, 4>(a, s);
  if (a.tokens <= 16) return tall ? launch<FMT, 4, 2, 8, 2>(a, s) : launch<FMT, 2, 2, 8, 3>(a, s);
  return launch<FMT, 2, 4, 6, 2>(a, s);
}

}  // namespace

// Which is the faster, by the weights that an SM's share of this kernel's grid has (with
// the rows and SMs that the last round of items leaves idle), times the 152 SMs: it takes
// 0.2 us for 2^20 of them up to 8 tokens, 0.3 up to 16, 0.55 above; linear_mma.cu's two
// launches take 9 to 12 us and then 6 TB/s.  Measured (us, this kernel / that one):
//                      4096 x 4096   8192 x 4096   8192 x 8192   28672 x 8192   3360 x 19552
//   (2^20 weights            19            38            76            228            91)
//   MXFP4   8 tokens:   5.0 /  9.9    9.0 / 13.0   15.2 / 13.9    32.5 / 24.6    17.8 / 13.3
//          16 tokens:   6.7 / 11.8   12.2 / 14.9   21.3 / 15.5    45.9 / 26.0    24.6 / 14.8
//          32 tokens:  12.8 / 14.8   24.5 / 15.6   44.5 / 20.0   130.5 / 32.9    50.8 / 22.9
//   NVFP4   8 tokens:   5.4 / 10.8    9.8 / 13.3   16.8 / 14.4    36.4 / 26.3    19.7 / 14.2
//          32 tokens:  12.4 / 14.7   23.6 / 15.5   42.9 / 19.4   125.4 / 36.1    49.0 / 26.7
// The workspace's size follows from it, so it asks no device: it assumes 152 SMs, and that
// as many clusters of the CTAs wanted are resident as there are tiles (launch() takes fewer
// CTAs where they are not).
bool linear_mma_better(int64_t tokens, int64_t n, int64_t k) {
  constexpr int kSms = 152;
  const int64_t rows = tall_items(tokens, n, kSms) ? 64 : 32, tiles = (n + rows - 1) / rows;
  const int64_t ctas = cluster_ctas(tokens <= 16 ? 8 : 6, tiles, k, kSms);
  const int64_t rounds = ctas > 1 ? 1 : (tiles + kSms - 1) / kSms;
  const int64_t least = tokens <= 8 ? 72 : tokens <= 16 ? 50 : 28;
  return rounds * rows * kSms * k / ctas >= least << 20;
}

cudaError_t launch_linear(const LinearArgs &a, cudaStream_t s) {
  return a.fmt == 0 ? launch_fmt<0>(a, s) : launch_fmt<1>(a, s);
}

}  // namespace mx
