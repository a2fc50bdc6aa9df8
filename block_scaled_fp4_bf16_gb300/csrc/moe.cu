// Mixture of experts for a few tokens: the router, and the two products of the
// chosen experts.
#include "few_tokens.cuh"

namespace mx {
namespace {

constexpr int kWarps = 8;

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

// Order of the logits as unsigned integers: NaN first, then descending.
__device__ __forceinline__ uint32_t logit_key(float v) {
  const uint32_t u = __float_as_uint(v);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// One CTA per token: the logits by warps, the choice by the first warp.
__global__ void __launch_bounds__(kWarps * 32) route_kernel(const RouteArgs a) {
  __shared__ float logits[kMoeMaxExperts];
  griddep_launch_dependents();
  griddep_wait();
  const int t = blockIdx.x, warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  for (int e = warp; e < a.experts; e += kWarps) {
    float acc = 0.0f;
    for (int k = lane; k < a.hidden; k += 32)
      acc = __fmaf_rn(bf16_value(a.router, static_cast<int64_t>(e) * a.hidden + k),
                      bf16_value(a.x, t * a.ld_x + k), acc);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) acc += __shfl_xor_sync(0xFFFFFFFFu, acc, m);
    if (lane == 0) logits[e] = a.bias ? acc + a.bias[e] : acc;
  }
  __syncthreads();
  if (warp != 0) return;
  float chosen[kMoeMaxTopK];
  int ids[kMoeMaxTopK];
  uint32_t taken = 0;  // bit i: this lane's i-th logit is taken
  for (int j = 0; j < a.top_k; ++j) {
    uint32_t best = 0, at = 0xFFFFFFFFu;
    for (int e = lane, i = 0; e < a.experts; e += 32, ++i) {
      const uint32_t key = logit_key(logits[e]);
      if (!((taken >> i) & 1u) && key > best) best = key, at = e;
    }
    const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best);
    const uint32_t id = __reduce_min_sync(0xFFFFFFFFu, best == top ? at : 0xFFFFFFFFu);
    const bool none = top <= logit_key(-INFINITY);
    ids[j] = none ? -1 : static_cast<int>(id);
    chosen[j] = none ? -INFINITY : logits[id];
    if (!none && (id & 31u) == lane) taken |= 1u << (id / 32);
  }
  float sum = 0.0f;
  if (a.normalize) {
    for (int j = 0; j < a.top_k; ++j) sum += ids[j] < 0 ? 0.0f : expf(chosen[j] - chosen[0]);
  } else {
    for (int e = lane; e < a.experts; e += 32) sum += expf(logits[e] - chosen[0]);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, m);
  }
  if (lane < a.top_k) {
    int id = -1;
    float l = 0.0f;
    for (int j = 0; j < a.top_k; ++j)
      if (j == lane) id = ids[j], l = chosen[j];
    a.ids[t * a.top_k + lane] = id;
    a.weights[t * a.top_k + lane] = id < 0 ? 0.0f : expf(l - chosen[0]) / sum;
  }
}

// h[p, i] = act(G_e x)[i] (U_e x)[i] for pair p = t * top_k + j, e = ids[p].
template <int FMT>
__global__ void __launch_bounds__(kWarps * 32) up_kernel(const MoeArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int p = blockIdx.y, t = p / a.top_k;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32;
  const int e = a.ids[p];
  if (e < 0 || e >= a.experts || row >= a.inter) return;
  const int64_t blocks = a.hidden / (FMT == 0 ? 32 : 16);
  const int64_t code_bytes = static_cast<int64_t>(a.inter) * (a.hidden / 2);
  const int64_t scale_bytes = ((a.inter + 127ll) / 128) * ((blocks + 3) / 4) * 512;
  const auto x = [&](int, int64_t k) { return bf16_value(a.x, t * a.ld_x + k); };
  float g[1], u[1];
  warp_row_dot<FMT, 1>(a.gate.codes + e * code_bytes, a.gate.scales + e * scale_bytes, row,
                       a.hidden, 1, x, g);
  warp_row_dot<FMT, 1>(a.up.codes + e * code_bytes, a.up.scales + e * scale_bytes, row, a.hidden, 1,
                       x, u);
  if ((threadIdx.x & 31) != 0) return;
  const float gv = FMT == 1 ? g[0] * a.gate.ts[e] : g[0];
  const float uv = FMT == 1 ? u[0] * a.up.ts[e] : u[0];
  const float act = a.gelu ? gelu_f32x2(make_float2(gv, gv)).x : gv / (1.0f + expf(-gv));
  a.h[static_cast<int64_t>(p) * a.inter + row] = act * uv;
}

// y[t, n] = sum_j w_tj (D_e h_p)[n].
template <int FMT>
__global__ void __launch_bounds__(kWarps * 32) down_kernel(const MoeArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int t = blockIdx.y;
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32;
  if (row >= a.hidden) return;
  const int64_t blocks = a.inter / (FMT == 0 ? 32 : 16);
  const int64_t code_bytes = static_cast<int64_t>(a.hidden) * (a.inter / 2);
  const int64_t scale_bytes = ((a.hidden + 127ll) / 128) * ((blocks + 3) / 4) * 512;
  float y = 0.0f;
  for (int j = 0; j < a.top_k; ++j) {
    const int p = t * a.top_k + j, e = a.ids[p];
    if (e < 0 || e >= a.experts) continue;
    float z[1];
    warp_row_dot<FMT, 1>(
        a.down.codes + e * code_bytes, a.down.scales + e * scale_bytes, row, a.inter, 1,
        [&](int, int64_t k) { return a.h[static_cast<int64_t>(p) * a.inter + k]; }, z);
    y = __fmaf_rn(a.weights[p], FMT == 1 ? z[0] * a.down.ts[e] : z[0], y);
  }
  if ((threadIdx.x & 31) == 0) static_cast<uint16_t *>(a.y)[t * a.ld_y + row] = bf16_bits(y);
}

template <int FMT>
cudaError_t launch_experts(const MoeArgs &a, cudaStream_t s) {
  const dim3 block(kWarps * 32);
  const cudaError_t e = launch_pdl(
      up_kernel<FMT>, dim3((a.inter + kWarps - 1) / kWarps, a.tokens * a.top_k), block, 0, s, a);
  if (e != cudaSuccess) return e;
  return launch_pdl(down_kernel<FMT>, dim3((a.hidden + kWarps - 1) / kWarps, a.tokens), block, 0, s,
                    a);
}

}  // namespace

cudaError_t launch_moe_route(const RouteArgs &a, cudaStream_t s) {
  return launch_pdl(route_kernel, dim3(a.tokens), dim3(kWarps * 32), 0, s, a);
}

cudaError_t launch_moe_experts(const MoeArgs &a, cudaStream_t s) {
  return a.fmt == 0 ? launch_experts<0>(a, s) : launch_experts<1>(a, s);
}

}  // namespace mx
