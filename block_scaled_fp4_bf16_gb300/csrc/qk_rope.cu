// RMS norm of each query and key head and the rotation by position, and its gradients.
//
// Forward: s = mean(x^2), r = (s + eps)^-1/2, n = x r w; a pair (a, b) of channels with
// angle phi becomes (a cos - b sin, b cos + a sin).  Backward: with g the pair's gradient
// turned back, dw = sum g x r, dx = r (g w - x r mean(g w x r)).
//
// Both read each element once and write it once.  A group of LANES lanes takes a head, 16
// channels a lane (two 16-byte loads), so that the mean is a few shuffles, and a lane holds
// both channels of its eight pairs in either order of the channels; a warp takes 32 / LANES
// heads at a time and goes through the heads of a token with the sines and cosines in
// registers: they are computed once for a token and slice of its heads, not once a head.
// 8192 tokens of 72 x 128: 56 us, 0.80 of the time that a plain copy's rate gives (a variant of
// the kernel that only copies takes 50 to 56 us).  Gradients of 4096 x 40 x 128: 34 us, 0.56 of
// it, 4 of them for the second launch, the rest latency with 16 warps an SM (registers).
#include <type_traits>

#include "decode.h"
#include "mx_device.cuh"

namespace mx {
namespace {

constexpr int kWarps = 8;

// f / 2 pi modulo 1, in units of 2^-64: the phase of a position is then one 64-bit
// product, exact modulo a turn.
__device__ __forceinline__ uint64_t turns_of(float f) {
  constexpr uint64_t kInv2Pi = 0x28BE60DB9391054Aull;  // 2^64 / 2 pi
  const uint32_t b = __float_as_uint(f);
  const int be = static_cast<int>((b >> 23) & 255u);
  const uint64_t m = (b & 0x7FFFFFu) | (be ? 0x800000u : 0u);
  const int e = (be ? be : 1) - 150;  // |f| = m 2^e
  const uint64_t lo = m * kInv2Pi, hi = __umul64hi(m, kInv2Pi);
  uint64_t t;
  if (e >= 0)
    t = e < 64 ? lo << e : 0;
  else if (e > -64)
    t = (lo >> -e) | (hi << (64 + e));
  else
    t = e > -128 ? hi >> (-e - 64) : 0;
  return (b >> 31) ? 0 - t : t;
}

// The 16 channels of lane j of a head: two chunks of 8 that begin at these channels.  The
// lane's pairs are 8 j .. 8 j + 7: (chunk 0, chunk 1) element by element, or neighbours.
struct Chunks {
  int at[2];
  bool in, turns;
};

__device__ __forceinline__ Chunks chunks_of(int j, const RopeArgs &a) {
  Chunks c;
  c.in = 16 * j < a.head_dim;
  c.turns = 16 * j < a.rotary_dim;
  if (c.turns && !a.interleaved)
    c.at[0] = 8 * j, c.at[1] = 8 * j + a.rotary_dim / 2;
  else
    c.at[0] = 16 * j, c.at[1] = 16 * j + 8;
  return c;
}

__device__ __forceinline__ void unpack(const uint4 &q, float *v) {
  const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    v[2 * i] = __uint_as_float(w[i] << 16);
    v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
  }
}

__device__ __forceinline__ uint4 pack(const float *v) {
  uint32_t w[4];
#pragma unroll
  for (int i = 0; i < 4; ++i)
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w[i]) : "f"(v[2 * i + 1]), "f"(v[2 * i]));
  return make_uint4(w[0], w[1], w[2], w[3]);
}

// A part's weight in shared memory, in the lanes' order: lane j's 16 channels, four at a time
// (0 for a lane without channels: its terms go into its head's sums).
struct Weights {
  float4 of[4][16];  // [four][lane j]
};
__device__ __forceinline__ void load_weights(Weights &w, const uint16_t *weight, const RopeArgs &a) {
  for (int i = threadIdx.x; i < 64 && weight != nullptr; i += kWarps * 32) {
    const int j = i >> 2, four = i & 3;
    const Chunks c = chunks_of(j, a);
    const int at = c.at[four >> 1] + 4 * (four & 1);
    float v[4] = {};
    if (c.in && in_bounds(at, 4, a.head_dim, a.status))
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = __uint_as_float(static_cast<uint32_t>(weight[at + e]) << 16);
    w.of[four][j] = make_float4(v[0], v[1], v[2], v[3]);
  }
}
__device__ __forceinline__ void weights_of(float *w, const Weights &s, int j) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float4 v = s.of[i][j];
    w[4 * i] = v.x, w[4 * i + 1] = v.y, w[4 * i + 2] = v.z, w[4 * i + 3] = v.w;
  }
}

// A lane's 16 channels of a row that begins at element `row` (zeros if !in).
struct Row {
  uint4 q[2];
};
__device__ __forceinline__ Row load_row(const uint16_t *p, int64_t row, const Chunks &c, bool in,
                                        int64_t extent, uint32_t *status) {
  Row r;
#pragma unroll
  for (int i = 0; i < 2; ++i)
    r.q[i] = in && in_bounds(row + c.at[i], 8, extent, status)
                 ? *reinterpret_cast<const uint4 *>(p + row + c.at[i])
                 : make_uint4(0, 0, 0, 0);
  return r;
}

__device__ __forceinline__ void store_row(uint16_t *p, int64_t row, const Chunks &c, bool in,
                                          const float *v, int64_t extent, uint32_t *status) {
#pragma unroll
  for (int i = 0; i < 2; ++i)
    if (in && in_bounds(row + c.at[i], 8, extent, status))
      *reinterpret_cast<uint4 *>(p + row + c.at[i]) = pack(v + 8 * i);
}

template <int LANES>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int m = LANES / 2; m > 0; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
  return v;
}

// The frequencies of all pairs as turns, in shared memory (in registers they would cost a
// quarter of the warps).
__device__ __forceinline__ void load_turns(uint64_t *turns, const RopeArgs &a) {
  for (int i = threadIdx.x; i < a.rotary_dim / 2; i += kWarps * 32) turns[i] = turns_of(a.inv_freq[i]);
}

// Sine and cosine of the lane's eight pairs at a position.
struct Angles {
  float sin[8], cos[8];
};
__device__ __forceinline__ void angles_of(Angles &t, const uint64_t *turns, int position) {
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    // (the upper 32 bits as a signed fraction of a turn: half turns in [-1, 1))
    const uint64_t phase = turns[i] * static_cast<uint64_t>(static_cast<int64_t>(position));
    const float half = static_cast<float>(static_cast<int32_t>(phase >> 32)) * 0x1p-31f;
    sincospif(half, &t.sin[i], &t.cos[i]);
  }
}

// Turns the lane's pairs, by the angle (SIGN 1) or back (-1).
template <int SIGN>
__device__ __forceinline__ void turn(float *v, const Angles &t, bool interleaved) {
  auto pair = [&](float &x, float &y, int i) {
    const float a = x, b = y, s = SIGN * t.sin[i];
    x = a * t.cos[i] - b * s;
    y = b * t.cos[i] + a * s;
  };
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 8; ++i) pair(v[2 * i], v[2 * i + 1], i);
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) pair(v[i], v[8 + i], i);
  }
}

// A warp's items: (token, slice of the groups of heads), in the order of the tokens.
struct Share {
  int groups[2];  // of queries and keys, 32 / LANES heads each
  int slices[2], per_slice[2];
};
struct Item {
  int64_t token;
  int first, last;  // groups
};
__device__ __forceinline__ Item item_of(int64_t i, int slices, int per_slice, int groups) {
  Item t;
  if (slices == 1) {
    t = Item{i, 0, groups};
  } else {  // (there are slices only where tokens are few)
    const int n = static_cast<int>(i), token = n / slices, first = (n - token * slices) * per_slice;
    t = Item{token, first, min(first + per_slice, groups)};
  }
  return t;
}

// The reciprocal norm of a head, from its lane's 16 channels.
template <int LANES>
__device__ __forceinline__ float reciprocal_norm(const float *v, const RopeArgs &a, float per_dim) {
  float sum = 0.0f;
#pragma unroll
  for (int e = 0; e < 16; ++e) sum += v[e] * v[e];
  return rsqrtf(head_sum<LANES>(sum) * per_dim + a.eps);
}

// Queries and keys count as one row of heads: groups of the queries', then of the keys'.
template <int LANES>
__global__ void __launch_bounds__(kWarps * 32, 2)
    rope_kernel(const __grid_constant__ RopeArgs a, const __grid_constant__ Share share) {
  constexpr int kHeads = 32 / LANES, kBatch = 2;
  __shared__ uint64_t turns[kRopeMaxDim / 2];
  __shared__ Weights weights[2];
  griddep_launch_dependents();
  griddep_wait();
  load_turns(turns, a);
  load_weights(weights[0], a.part[0].weight, a);
  load_weights(weights[1], a.part[1].weight, a);
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, j = lane % LANES;
  const Chunks c = chunks_of(j, a);
  const float per_dim = 1.0f / static_cast<float>(a.head_dim);
  const int64_t items = a.tokens * share.slices[0], stride = static_cast<int64_t>(gridDim.x) * kWarps;
  for (int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + warp; i < items; i += stride) {
    const Item item = item_of(i, share.slices[0], share.per_slice[0], share.groups[0] + share.groups[1]);
    Angles t;
    bool turned = false;
    // groups first .. last - 1 of a part (K: queries or keys, so that its fields are constants)
    auto part = [&](auto which, int first, int last) {
      constexpr int K = decltype(which)::value;
      if (first >= last) return;
      const Heads &p = a.part[K];
      const int64_t cols = static_cast<int64_t>(p.heads) * a.head_dim;
      const int step = kHeads * a.head_dim, own = lane / LANES * a.head_dim;
      const int64_t x_at = item.token * p.ld + own, y_at = item.token * p.ld_y + own;
      Row x[2][kBatch];  // a batch, and the next one on its way
      auto load = [&](Row(&to)[kBatch], int g0) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b)
          to[b] = load_row(p.x, x_at + static_cast<int64_t>(g0 + b) * step, c,
                           c.in && g0 + b < last && (g0 + b) * kHeads + lane / LANES < p.heads,
                           (a.tokens - 1) * p.ld + cols, a.status);
      };
      auto turn_batch = [&](const Row(&of)[kBatch], int g0) {
#pragma unroll
        for (int b = 0; b < kBatch; ++b) {
          if (g0 + b >= last) break;
          float v[16];
          unpack(of[b].q[0], v);
          unpack(of[b].q[1], v + 8);
          if (p.weight != nullptr) {
            const float r = reciprocal_norm<LANES>(v, a, per_dim);
            float w[16];
            weights_of(w, weights[K], j);
#pragma unroll
            for (int e = 0; e < 16; ++e) v[e] = v[e] * r * w[e];
          }
          if (c.turns) turn<1>(v, t, a.interleaved);
          store_row(p.y, y_at + static_cast<int64_t>(g0 + b) * step, c,
                    c.in && (g0 + b) * kHeads + lane / LANES < p.heads, v, (a.tokens - 1) * p.ld_y + cols, a.status);
        }
      };
      load(x[0], first);
      if (!turned) {  // (while the first heads are on their way)
        turned = true;
        if (c.turns && in_bounds(item.token, 1, a.tokens, a.status)) angles_of(t, turns + 8 * j, a.positions[item.token]);
      }
      for (int g0 = first; g0 < last; g0 += 2 * kBatch) {
        if (g0 + kBatch < last) load(x[1], g0 + kBatch);
        turn_batch(x[0], g0);
        if (g0 + kBatch >= last) break;
        if (g0 + 2 * kBatch < last) load(x[0], g0 + 2 * kBatch);
        turn_batch(x[1], g0 + kBatch);
      }
    };
    part(std::integral_constant<int, 0>(), item.first, min(item.last, share.groups[0]));
    part(std::integral_constant<int, 1>(), max(item.first - share.groups[0], 0), item.last - share.groups[0]);
  }
}

// The gradients of the inputs, and each CTA's sums of those of the weights: of the queries,
// then of the keys (one part's sums in registers at a time).  The order of the sums follows
// from the sizes and the number of SMs alone: a warp's tokens in order, then the lanes, then
// the warps, then (backward_sum_kernel) the CTAs.
template <int LANES>
__global__ void __launch_bounds__(kWarps * 32, 2)
    rope_backward_kernel(const __grid_constant__ RopeArgs a, const __grid_constant__ Share share) {
  constexpr int kHeads = 32 / LANES;
  __shared__ uint64_t turns[kRopeMaxDim / 2];
  __shared__ Weights weights[2];
  __shared__ float sums[kWarps][kRopeMaxDim];
  griddep_launch_dependents();
  griddep_wait();
  load_turns(turns, a);
  load_weights(weights[0], a.part[0].weight, a);
  load_weights(weights[1], a.part[1].weight, a);
  __syncthreads();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, j = lane % LANES;
  const Chunks c = chunks_of(j, a);
  const float per_dim = 1.0f / static_cast<float>(a.head_dim);
  auto part = [&](auto which) {
    constexpr int k = decltype(which)::value;
    const Heads &p = a.part[k];
    const int64_t cols = static_cast<int64_t>(p.heads) * a.head_dim, stride = static_cast<int64_t>(gridDim.x) * kWarps;
    const int64_t items = p.heads > 0 ? a.tokens * share.slices[k] : 0;
    float dw[16] = {};
    for (int64_t i = static_cast<int64_t>(blockIdx.x) * kWarps + warp; i < items; i += stride) {
      const Item item = item_of(i, share.slices[k], share.per_slice[k], share.groups[k]);
      const int step = kHeads * a.head_dim, own = lane / LANES * a.head_dim;
      const int64_t x_at = item.token * p.ld + own, dy_at = item.token * p.ld_dy + own, y_at = item.token * p.ld_y + own;
      Angles t;
      Row x[2], dy[2];  // of a group, and of the next one, on its way
      auto load = [&](int to, int g) {
        const bool in = c.in && g * kHeads + lane / LANES < p.heads;
        const int64_t at = static_cast<int64_t>(g) * step;
        // (without a norm the inputs are not read)
        x[to] = load_row(p.x, x_at + at, c, in && p.weight != nullptr, (a.tokens - 1) * p.ld + cols, a.status);
        dy[to] = load_row(p.dy, dy_at + at, c, in, (a.tokens - 1) * p.ld_dy + cols, a.status);
      };
      auto back = [&](int of, int g) {
        const bool in = c.in && g * kHeads + lane / LANES < p.heads;
        float v[16];
        unpack(dy[of].q[0], v);
        unpack(dy[of].q[1], v + 8);
        if (c.turns) turn<-1>(v, t, a.interleaved);
        if (p.weight != nullptr) {
          float n[16], w[16];
          unpack(x[of].q[0], n);
          unpack(x[of].q[1], n + 8);
          const float r = reciprocal_norm<LANES>(n, a, per_dim);
          weights_of(w, weights[k], j);
          float dot = 0.0f;
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            n[e] = in ? n[e] * r : 0.0f;  // (others' x is 0, but r may be infinite)
            dw[e] += v[e] * n[e];
            v[e] *= w[e];
            dot += v[e] * n[e];
          }
          dot = head_sum<LANES>(dot) * per_dim;
#pragma unroll
          for (int e = 0; e < 16; ++e) v[e] = r * (v[e] - n[e] * dot);
        }
        store_row(p.y, y_at + static_cast<int64_t>(g) * step, c, in, v, (a.tokens - 1) * p.ld_y + cols, a.status);
      };
      if (item.first >= item.last) continue;
      load(0, item.first);
      if (c.turns && in_bounds(item.token, 1, a.tokens, a.status)) angles_of(t, turns + 8 * j, a.positions[item.token]);
      for (int g = item.first; g < item.last; g += 2) {
        if (g + 1 < item.last) load(1, g + 1);
        back(0, g);
        if (g + 1 >= item.last) break;
        if (g + 2 < item.last) load(0, g + 2);
        back(1, g + 1);
      }
    }
    if (a.partials == nullptr) return;
    __syncthreads();  // (the queries' sums are read)
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      float s = dw[e];
#pragma unroll
      for (int m = 16; m >= LANES; m >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, m);
      if (lane < LANES && c.in) sums[warp][c.at[e >> 3] + (e & 7)] = s;
    }
    __syncthreads();
    for (int d = threadIdx.x; d < a.head_dim; d += kWarps * 32) {
      float s = sums[0][d];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) s += sums[w][d];
      a.partials[(static_cast<int64_t>(blockIdx.x) * 2 + k) * a.head_dim + d] = s;
    }
  };
  part(std::integral_constant<int, 0>());
  part(std::integral_constant<int, 1>());
}

// dweight[d] = the CTAs' sums, in their order within each of 32 warps (so that all are read at
// once): a CTA takes 32 columns of the 2 head_dim.
constexpr int kSumWarps = 32;
__global__ void __launch_bounds__(kSumWarps * 32)
    backward_sum_kernel(const __grid_constant__ RopeArgs a, int ctas) {
  __shared__ float sums[kSumWarps][32];
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int i = blockIdx.x * 32 + lane;
  float s = 0.0f;
  if (i < 2 * a.head_dim) {
#pragma unroll
    for (int k = 0; k < kRopeBackCtas / kSumWarps; ++k) {
      const int p = k * kSumWarps + warp;
      if (p < ctas) s += a.partials[static_cast<int64_t>(p) * 2 * a.head_dim + i];
    }
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || i >= 2 * a.head_dim) return;
#pragma unroll
  for (int w = 1; w < kSumWarps; ++w) s += sums[w][lane];
  const int k = i >= a.head_dim;
  float *out = a.part[k].dweight;
  if (out != nullptr) out[i - k * a.head_dim] = s;
}
static_assert(kRopeBackCtas % kSumWarps == 0, "all partials are summed");

int lanes_of(int head_dim) {
  int lanes = 1;
  while (16 * lanes < head_dim) lanes *= 2;
  return lanes;
}

// Slices of a token's groups of heads: those with which the busiest warp has the least to do,
// an item's angles counted as one group (8192 tokens of 18 groups on 3648 warps: whole tokens
// leave most warps with two and some with three).
void slice(int64_t tokens, int groups, int64_t warps, int *slices, int *per_slice) {
  *slices = 1;
  *per_slice = groups;
  int64_t least = INT64_MAX;
  for (int p = groups; p >= 1; --p) {
    const int n = (groups + p - 1) / p;
    if (n > 1 && tokens * n >= (int64_t(1) << 31)) break;  // (the kernel divides 32-bit numbers)
    const int64_t cost = (tokens * n + warps - 1) / warps * (p + 1);
    if (cost < least) least = cost, *slices = n, *per_slice = p;
  }
}

Share share_of(const RopeArgs &a, int lanes, int64_t warps, bool together) {
  const int heads = 32 / lanes;
  Share s;
  for (int k = 0; k < 2; ++k) s.groups[k] = (a.part[k].heads + heads - 1) / heads;
  for (int k = 0; k < 2; ++k)
    slice(a.tokens, together ? s.groups[0] + s.groups[1] : s.groups[k], warps, &s.slices[k], &s.per_slice[k]);
  return s;
}

template <int LANES>
cudaError_t forward(const RopeArgs &a, cudaStream_t s) {
  const int64_t most = static_cast<int64_t>(a.num_sms) * 2;
  const Share share = share_of(a, LANES, most * kWarps, true);
  const int64_t ctas = (a.tokens * share.slices[0] + kWarps - 1) / kWarps;
  return launch_pdl(rope_kernel<LANES>, dim3(static_cast<unsigned>(ctas < most ? ctas : most)),
                    dim3(kWarps * 32), 0, s, a, share);
}

template <int LANES>
cudaError_t backward(const RopeArgs &a, cudaStream_t s) {
  int64_t most = static_cast<int64_t>(a.num_sms) * 2;
  if (most > kRopeBackCtas) most = kRopeBackCtas;
  const Share share = share_of(a, LANES, most * kWarps, false);
  const int64_t slices = share.slices[0] > share.slices[1] ? share.slices[0] : share.slices[1];
  int64_t ctas = (a.tokens * slices + kWarps - 1) / kWarps;
  ctas = ctas < 1 ? 1 : ctas < most ? ctas : most;
  const cudaError_t e = launch_pdl(rope_backward_kernel<LANES>, dim3(static_cast<unsigned>(ctas)),
                                   dim3(kWarps * 32), 0, s, a, share);
  if (e != cudaSuccess || a.partials == nullptr) return e;
  return launch_pdl(backward_sum_kernel, dim3((2 * a.head_dim + 31) / 32), dim3(kSumWarps * 32), 0, s, a,
                    static_cast<int>(ctas));
}

}  // namespace

cudaError_t launch_qk_rope(const RopeArgs &a, cudaStream_t s) {
  switch (lanes_of(a.head_dim)) {
    case 1: return forward<1>(a, s);
    case 2: return forward<2>(a, s);
    case 4: return forward<4>(a, s);
    case 8: return forward<8>(a, s);
    default: return forward<16>(a, s);
  }
}

cudaError_t launch_qk_rope_backward(const RopeArgs &a, cudaStream_t s) {
  switch (lanes_of(a.head_dim)) {
    case 1: return backward<1>(a, s);
    case 2: return backward<2>(a, s);
    case 4: return backward<4>(a, s);
    case 8: return backward<8>(a, s);
    default: return backward<16>(a, s);
  }
}

}  // namespace mx
