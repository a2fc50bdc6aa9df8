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
  if (a.counts != nullptr && t == 0 && threadIdx.x < kMoeCounts) a.counts[threadIdx.x] = 0;
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

}  // namespace

cudaError_t launch_moe_route(const RouteArgs &a, cudaStream_t s) {
  return launch_pdl(route_kernel, dim3(a.tokens), dim3(kWarps * 32), 0, s, a);
}

}  // namespace mx
