// Mixture of experts for a few tokens: the router, and the two products of the
// chosen experts.
#include "few_tokens.cuh"

namespace mx {
namespace {

constexpr int kWarps = 8;

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

// ---------------------------------------------------------------- the experts

// y[t] = sum_j w_tj z[t, j], in the order of the slots.
__global__ void __launch_bounds__(256) combine_kernel(const MoeArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int t = blockIdx.y, c = (blockIdx.x * 256 + threadIdx.x) * 2;
  if (c >= a.hidden) return;
  float y0 = 0.0f, y1 = 0.0f;
  for (int j = 0; j < a.top_k; ++j) {
    const int p = t * a.top_k + j, e = a.ids[p];
    if (e < 0 || e >= a.experts) continue;
    const float w = a.weights[p];
    float2 z = make_float2(0.0f, 0.0f);
    for (int i = 0; i < a.down_parts; ++i) {
      const int64_t o = (static_cast<int64_t>(i) * a.tokens * a.top_k + p) * a.hidden + c;
      if (!in_bounds(o, 2, static_cast<int64_t>(a.down_parts) * a.tokens * a.top_k * a.hidden,
                     a.status))
        continue;
      const float2 v = *reinterpret_cast<const float2 *>(a.z + o);
      z.x += v.x;
      z.y += v.y;
    }
    y0 = __fmaf_rn(w, z.x, y0);
    y1 = __fmaf_rn(w, z.y, y1);
  }
  const int64_t o = t * a.ld_y + c;
  if (!in_bounds(o, 2, (a.tokens - 1) * a.ld_y + a.hidden, a.status)) return;
  uint16_t *y = static_cast<uint16_t *>(a.y) + o;
  y[0] = bf16_bits(y0);
  y[1] = bf16_bits(y1);
}

}  // namespace

cudaError_t launch_moe_route(const RouteArgs &a, cudaStream_t s) {
  return launch_pdl(route_kernel, dim3(a.tokens), dim3(kWarps * 32), 0, s, a);
}

cudaError_t launch_moe_experts(const MoeArgs &a, cudaStream_t s) {
  const cudaError_t e = launch_expert_products(a, s);
  if (e != cudaSuccess) return e;
  return launch_pdl(combine_kernel, dim3((a.hidden + 511) / 512, a.tokens), dim3(256), 0, s, a);
}

}  // namespace mx
