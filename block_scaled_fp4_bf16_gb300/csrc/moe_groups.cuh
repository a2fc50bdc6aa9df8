// The grouping of a mixture-of-experts call's (token, slot) pairs by expert.
#pragma once

#include "few_tokens.cuh"

namespace mx {

// The pairs sorted by expert (an expert's in ascending order), divided into groups
// of up to a given size of one expert.  A pair's place is its index in the list.
// The arrays lie one after the other (bytes(pairs) in all, 16-byte aligned) in shared
// memory; every CTA makes its own.
struct Groups {
  uint16_t *list;    // pairs
  uint16_t *expert;  // of a group
  uint16_t *begin;   // place of a group's first pair
  uint16_t *size;
  int *count;        // groups

  __host__ __device__ static constexpr int bytes(int pairs) { return (pairs * 8 + 16 + 15) / 16 * 16; }
  __device__ __forceinline__ static Groups at(void *p, int pairs) {
    Groups g;
    g.list = static_cast<uint16_t *>(p);
    g.expert = g.list + pairs;
    g.begin = g.expert + pairs;
    g.size = g.begin + pairs;
    g.count = reinterpret_cast<int *>(g.size + pairs);
    return g;
  }
};

// A place's group and its index there.
__device__ __forceinline__ uint16_t pack_member(int group, int index) {
  return static_cast<uint16_t>(group * kMoeGroupMax + index);
}

// Whole CTA of W warps.  Fills g; place[pair]: its place (0xFFFF: an empty slot);
// member[place]: pack_member.  scratch: 2 * (W + 2) * experts bytes.
// Every CTA that does this gets the same groups.
template <int W>
__device__ __forceinline__ void make_groups(const Groups &g, uint16_t *place, uint16_t *member,
                                            char *scratch, const int32_t *ids, int pairs,
                                            int experts, int group, uint32_t *status) {
  if (pairs <= 32) {
    // A pair a lane: its place is the number of pairs before it in the order
    // (expert, pair), its group the number of groups that begin before it.
    // (the comparisons of a pair are one vote, the pairs divided among the warps)
    const int lane = threadIdx.x & 31;
    int e = lane < pairs && in_bounds(lane, 1, pairs, status) ? ids[lane] : -1;
    if (e < 0 || e >= experts) e = -1;
    for (int i = threadIdx.x >> 5; i < pairs; i += W) {
      const int o = __shfl_sync(0xFFFFFFFFu, e, i);
      const uint32_t before =
          __ballot_sync(0xFFFFFFFFu, e >= 0 && (e < o || (e == o && lane < i)));
      if (lane == 0) place[i] = static_cast<uint16_t>(o >= 0 ? __popc(before) : 0xFFFF);
    }
    __syncthreads();
    if (threadIdx.x < 32) {
      const int at = lane < pairs ? place[lane] : 0xFFFF;
      const uint32_t same = __match_any_sync(0xFFFFFFFFu, e);
      const int rank = __popc(same & ((1u << lane) - 1u));
      const bool first = e >= 0 && rank % group == 0;
      // the groups in the order of their first places
      const uint32_t starts = __reduce_or_sync(0xFFFFFFFFu, first ? 1u << at : 0u);
      if (e >= 0) {
        const int index = __popc(starts & (0xFFFFFFFFu >> (31 - at))) - 1;
        g.list[at] = static_cast<uint16_t>(lane);
        member[at] = pack_member(index, rank % group);
        if (first) {
          g.expert[index] = static_cast<uint16_t>(e);
          g.begin[index] = static_cast<uint16_t>(at);
          g.size[index] = static_cast<uint16_t>(min(__popc(same) - rank, group));
        }
      }
      if (lane == 0) *g.count = __popc(starts);
    }
    __syncthreads();
    return;
  }
  constexpr int kRuns = (kMoeMaxTokens * kMoeMaxTopK + 32 * W - 1) / (32 * W);  // of 32, a warp
  // [W][experts]: a warp's pairs of an expert, then the place of the first of
  // them; and an expert's first place and first group
  uint16_t *counts = reinterpret_cast<uint16_t *>(scratch);
  uint16_t *first_place = counts + W * experts, *first_group = first_place + experts;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int chunks = (pairs + 31) / 32, per_warp = (chunks + W - 1) / W;
  for (int i = threadIdx.x; i < W * experts; i += W * 32) counts[i] = 0;
  int expert[kRuns], rank[kRuns];
#pragma unroll
  for (int c = 0; c < kRuns; ++c) {
    const int p = (warp * per_warp + c) * 32 + lane;
    expert[c] = c < per_warp && p < pairs && in_bounds(p, 1, pairs, status) ? ids[p] : -1;
    if (expert[c] < 0 || expert[c] >= experts) expert[c] = -1;
    rank[c] = 0;
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < kRuns; ++c) {
    if (c >= per_warp) break;
    const uint32_t same = __match_any_sync(0xFFFFFFFFu, expert[c]);
    const int before = __popc(same & ((1u << lane) - 1u));
    if (expert[c] >= 0) rank[c] = counts[warp * experts + expert[c]] + before;
    __syncwarp();
    if (expert[c] >= 0 && before == 0)
      counts[warp * experts + expert[c]] += static_cast<uint16_t>(__popc(same));
    __syncwarp();
  }
  __syncthreads();
  if (warp == 0) {
    uint32_t place0 = 0, group0 = 0;
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
      const uint32_t at = place0 + (sum & 0xFFFFu) - n, first = group0 + (sum >> 16) - q;
      if (e < experts) {
        first_place[e] = static_cast<uint16_t>(at);
        first_group[e] = static_cast<uint16_t>(first);
        uint32_t base = at;
        for (int w = 0; w < W; ++w) {
          const uint32_t c = counts[w * experts + e];
          counts[w * experts + e] = static_cast<uint16_t>(base);
          base += c;
        }
      }
      for (uint32_t j = 0; j < q; ++j) {
        g.expert[first + j] = static_cast<uint16_t>(e);
        g.begin[first + j] = static_cast<uint16_t>(at + j * group);
        g.size[first + j] = static_cast<uint16_t>(min(n - j * group, static_cast<uint32_t>(group)));
      }
      const uint32_t last = __shfl_sync(0xFFFFFFFFu, sum, 31);
      place0 += last & 0xFFFFu;
      group0 += last >> 16;
    }
    if (lane == 0) *g.count = static_cast<int>(group0);
  }
  __syncthreads();
#pragma unroll
  for (int c = 0; c < kRuns; ++c) {
    const int p = (warp * per_warp + c) * 32 + lane;
    if (c >= per_warp || p >= pairs) continue;
    const int e = expert[c];
    const int at = e >= 0 ? counts[warp * experts + e] + rank[c] : 0xFFFF;
    place[p] = static_cast<uint16_t>(at);
    if (e >= 0) {
      g.list[at] = static_cast<uint16_t>(p);
      const int i = at - first_place[e];
      member[at] = pack_member(first_group[e] + i / group, i % group);
    }
  }
  __syncthreads();
}

}  // namespace mx
