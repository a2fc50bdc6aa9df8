// The grouping of a mixture-of-experts call's (token, slot) pairs by expert.
#pragma once

#include <cuda_fp16.h>

#include "mx_device.cuh"
#include "mx_internal.h"

namespace mx {

// The (token, slot) pairs by expert, in shared memory: groups of up to
// kGroup pairs of one expert.  Every CTA makes them from the ids (at most 1024).
struct Groups {
  uint16_t *list;    // pairs, sorted by expert
  uint16_t *expert;  // of a group
  uint16_t *begin;   // of a group in list
  uint16_t *size;
  int count;

  static constexpr int bytes(int pairs) { return pairs * 8 + 16; }
};

// Whole CTA of W warps.  `at`: Groups::bytes(pairs) bytes; `scratch`: 2 * W *
// experts bytes.  An expert's pairs are in ascending order (every CTA has to
// make the same groups): a warp counts its run of the pairs, and an expert's
// pairs of the earlier warps come first.
template <int W>
__device__ __forceinline__ Groups make_groups(char *at, char *scratch, const int32_t *ids, int pairs,
                                              int experts, int group, uint32_t *status) {
  Groups g;
  g.list = reinterpret_cast<uint16_t *>(at);
  g.expert = g.list + pairs;
  g.begin = g.expert + pairs;
  g.size = g.begin + pairs;
  constexpr int kRuns = (kMoeMaxTokens * kMoeMaxTopK + 32 * W - 1) / (32 * W);  // of 32, a warp
  int *total = reinterpret_cast<int *>(at + pairs * 8);
  uint16_t *counts = reinterpret_cast<uint16_t *>(scratch);  // [W][experts]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int chunks = (pairs + 31) / 32, per_warp = (chunks + W - 1) / W;
  for (int i = threadIdx.x; i < W * experts; i += W * 32) counts[i] = 0;
  __syncthreads();
  int expert[kRuns], rank[kRuns];
#pragma unroll
  for (int c = 0; c < kRuns; ++c) {
    const int p = (warp * per_warp + c) * 32 + lane;
    expert[c] = c < per_warp && p < pairs && in_bounds(p, 1, pairs, status) ? ids[p] : -1;
    if (expert[c] >= experts) expert[c] = -1;
  }
#pragma unroll
  for (int c = 0; c < kRuns; ++c) {
    if (c >= per_warp) break;
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, expert[c]);
    const int before = __popc(same & ((1u << lane) - 1u));
    uint16_t *count = counts + warp * experts + expert[c];
    if (expert[c] >= 0) rank[c] = *count + before;
    __syncwarp();
    if (expert[c] >= 0 && before == 0) *count += static_cast<uint16_t>(__popc(same));
    __syncwarp();
  }
  __syncthreads();
  if (warp == 0) {
    uint32_t pair0 = 0, group0 = 0;
    for (int e0 = 0; e0 < experts; e0 += 32) {
      const int e = e0 + lane;
      uint32_t n = 0;
      if (e < experts)
        for (int w = 0; w < W; ++w) n += counts[w * experts + e];
      const uint32_t q = (n + group - 1) / group;
      uint32_t sum = n | (q << 16);  // both prefix sums at once (each below 2^16)
#pragma unroll
      for (int d = 1; d < 32; d <<= 1) {
        const uint32_t v = __shfl_up_sync(0xFFFFFFFFu, sum, d);
        if (lane >= d) sum += v;
      }
      const uint32_t pair = pair0 + (sum & 0xFFFFu) - n, first = group0 + (sum >> 16) - q;
      if (e < experts) {
        uint32_t base = pair;  // where the expert's pairs of each warp begin
        for (int w = 0; w < W; ++w) {
          const uint32_t c = counts[w * experts + e];
          counts[w * experts + e] = static_cast<uint16_t>(base);
          base += c;
        }
      }
      for (uint32_t j = 0; j < q; ++j) {
        g.expert[first + j] = static_cast<uint16_t>(e);
        g.begin[first + j] = static_cast<uint16_t>(pair + j * group);
        g.size[first + j] = static_cast<uint16_t>(min(n - j * group, static_cast<uint32_t>(group)));
      }
      const uint32_t last = __shfl_sync(0xFFFFFFFFu, sum, 31);
      pair0 += last & 0xFFFFu;
      group0 += last >> 16;
    }
    if (lane == 0) *total = static_cast<int>(group0);
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < kRuns; ++c) {
    if (c < per_warp && expert[c] >= 0)
      g.list[counts[warp * experts + expert[c]] + rank[c]] =
          static_cast<uint16_t>((warp * per_warp + c) * 32 + lane);
  }
  __syncthreads();
  g.count = *total;
  return g;
}

}  // namespace mx
