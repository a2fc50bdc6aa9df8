// RMS norm of each query and key head and the rotation by position, and its gradients.
//
// Forward: s = mean(x^2), r = (s + eps)^-1/2, n = x r w; a pair (a, b) of channels with
// angle phi becomes (a cos - b sin, b cos + a sin).  Backward: with g the pair's gradient
// turned back, dw = sum g x r, dx = r (g w - x r mean(g w x r)).
//
// Both read each element once and write it once.  A group of LANES lanes takes a head, 16
// channels a lane (two 16-byte pieces), so that the mean is a few shuffles, and a lane holds both
// channels of its eight pairs in either order of the channels; a warp takes 32 / LANES heads at a
// time and goes through the heads of a token with the sines and cosines in registers: they are
// computed once for a token and slice of its heads, not once a head.  The rows come through a
// ring of shared memory, so that a warp's next heads, of the next token too, are on their way.
//
// The bytes bound it, but instructions come close behind: two channels to an instruction, and
// the angles shared out over a warp's heads.  8192 tokens of 72 x 128: 49 us, 0.93 of the time
// that a plain copy's rate gives (one channel to an instruction 51.5; all angles in every lane 54.5;
// pieces of 16 channels for the channels that do not turn, half sectors each, 60; a third CTA
// on an SM 54).  Gradients of 4096 x 40 x 128: 27 us, 0.70 of it (16384: 0.93), 4 of them for the second
// launch, the rest uneven shares.
#include <type_traits>

#include "async_copy.cuh"
#include "decode.h"

namespace mx {
namespace {

constexpr int kWarps = 8;
constexpr int kCtas = 2;  // of an SM

// f / 2 pi modulo 1, to the nearest unit of 2^-64: the phase of a position is then one 64-bit
// product, off by at most 2^-34 of a turn (2^31 half units).  1 / 2 pi has 128 bits, of which a
// frequency of 2^16 takes 80; 64 were right for frequencies up to 1 (2^-18 of a turn at 2^16).
__device__ __forceinline__ uint64_t turns_of(float f) {
  constexpr uint64_t kHigh = 0x28BE60DB9391054Aull, kLow = 0x7F09D5F47D4D3770ull;  // 2^128 / 2 pi
  const uint32_t b = __float_as_uint(f);
  const int be = static_cast<int>((b >> 23) & 255u);
  const uint64_t m = (b & 0x7FFFFFu) | (be ? 0x800000u : 0u);
  const int e = (be ? be : 1) - 150;  // |f| = m 2^e
  // m / 2 pi in units of 2^-128
  const uint64_t p0 = m * kLow, carry = __umul64hi(m, kLow), p1 = m * kHigh + carry;
  const uint64_t p2 = __umul64hi(m, kHigh) + (p1 < carry ? 1 : 0);
  uint64_t t, half;  // times 2^e in units of 2^-64, and the next bit
  if (e >= 0) {  // (frequencies of 2^23 and more)
    t = e == 0 ? p1 : e < 64 ? p1 << e | p0 >> (64 - e) : 0;
    half = e < 64 ? p0 << e >> 63 : 0;
  } else if (e > -64) {
    t = p1 >> -e | p2 << (64 + e);
    half = p1 >> (-e - 1) & 1;
  } else {
    t = e > -128 ? p2 >> (-e - 64) : 0;
    half = e == -64 ? p1 >> 63 : e > -128 ? p2 >> (-e - 65) & 1 : 0;
  }
  t += half;
  return (b >> 31) ? 0 - t : t;
}

// The 16 channels of lane j of a head: two chunks of 8 that begin at these channels, from the
// first and the second half of the turning (or the other) ones, so that lanes side by side read
// and write whole sectors.
struct Chunks {
  int at[2];
  bool in, turns;
};

__device__ __forceinline__ Chunks chunks_of(int j, const RopeArgs &a) {
  Chunks c;
  c.in = 16 * j < a.head_dim;
  c.turns = 16 * j < a.rotary_dim;
  const int from = c.turns ? 0 : a.rotary_dim, half = (c.turns ? a.rotary_dim : a.head_dim - a.rotary_dim) / 2;
  c.at[0] = from + 8 * j - from / 2;
  c.at[1] = c.at[0] + half;
  return c;
}

// The lane's eight pairs: their first and their second channels, two pairs to a float2 (for
// instructions that take two).  Pair e is (e of chunk 0, e of chunk 1); interleaved
// (2 i, 2 i + 1) of chunk e % 2, i = e / 2.
struct Pairs {
  float2 x[4], y[4];
};
__device__ __forceinline__ int channel_of(const Chunks &c, bool interleaved, int e, int second) {
  return interleaved ? c.at[e & 1] + (e & 6) + second : c.at[second] + e;
}
__device__ __forceinline__ float2 widen(uint32_t w) {
  return make_float2(__uint_as_float(w << 16), __uint_as_float(w & 0xFFFF0000u));
}
__device__ __forceinline__ void unpack(const uint4 &chunk0, const uint4 &chunk1, bool interleaved, Pairs &v) {
  uint32_t w[4] = {chunk0.x, chunk0.y, chunk0.z, chunk0.w}, u[4] = {chunk1.x, chunk1.y, chunk1.z, chunk1.w};
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t x = __byte_perm(w[i], u[i], 0x5410);
      u[i] = __byte_perm(w[i], u[i], 0x7632);
      w[i] = x;
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) v.x[i] = widen(w[i]), v.y[i] = widen(u[i]);
}
__device__ __forceinline__ uint32_t narrow(const float2 &v) {
  uint32_t w;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(w) : "f"(v.y), "f"(v.x));
  return w;
}
__device__ __forceinline__ void pack(const Pairs &v, bool interleaved, uint4 &chunk0, uint4 &chunk1) {
  uint32_t w[4], u[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) w[i] = narrow(v.x[i]), u[i] = narrow(v.y[i]);
  if (interleaved) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t x = __byte_perm(w[i], u[i], 0x5410);
      u[i] = __byte_perm(w[i], u[i], 0x7632);
      w[i] = x;
    }
  }
  chunk0 = make_uint4(w[0], w[1], w[2], w[3]);
  chunk1 = make_uint4(u[0], u[1], u[2], u[3]);
}

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 minus(const float2 &v) { return make_float2(-v.x, -v.y); }

// A part's weight in shared memory, as the lanes' Pairs (0 for a lane without channels: its terms
// go into its head's sums).
struct Weights {
  float4 of[4][16];  // [four][lane j]
};
__device__ __forceinline__ void load_weights(Weights &w, const uint16_t *weight, const RopeArgs &a) {
  for (int i = threadIdx.x; i < 64 && weight != nullptr; i += kWarps * 32) {
    const int j = i >> 2, four = i & 3;
    const Chunks c = chunks_of(j, a);
    float v[4] = {};
#pragma unroll
    for (int e = 0; e < 4; ++e) {
      const int at = channel_of(c, a.interleaved, 4 * (four & 1) + e, four >> 1);
      if (c.in && in_bounds(at, 1, a.head_dim, a.status)) v[e] = __uint_as_float(static_cast<uint32_t>(weight[at]) << 16);
    }
    w.of[four][j] = make_float4(v[0], v[1], v[2], v[3]);
  }
}
__device__ __forceinline__ void weights_of(Pairs &w, const Weights &s, int j) {
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const float4 x = s.of[i][j], y = s.of[2 + i][j];
    w.x[2 * i] = make_float2(x.x, x.y), w.x[2 * i + 1] = make_float2(x.z, x.w);
    w.y[2 * i] = make_float2(y.x, y.y), w.y[2 * i + 1] = make_float2(y.z, y.w);
  }
}

// Writes the lane's chunks of a head, the first at element `at`.
__device__ __forceinline__ void store(uint16_t *p, int64_t at, const Chunks &c, bool in, const Pairs &v, bool interleaved,
                                      int64_t extent, uint32_t *status) {
  uint4 q[2];
  pack(v, interleaved, q[0], q[1]);
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const int64_t to = at + (i ? c.at[1] - c.at[0] : 0);
    if (in && in_bounds(to, 8, extent, status)) *reinterpret_cast<uint4 *>(p + to) = q[i];
  }
}

template <int LANES>
__device__ __forceinline__ float head_sum(float v) {
#pragma unroll
  for (int m = LANES / 2; m > 0; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
  return v;
}

// The frequencies of all pairs as turns, in shared memory (in registers they would cost a
// quarter of the warps), in the lanes' order: eight of a lane.
__device__ __forceinline__ void load_turns(uint64_t *turns, const RopeArgs &a) {
  for (int i = threadIdx.x; i < a.rotary_dim / 2; i += kWarps * 32) {
    const int j = i >> 3, e = i & 7, pair = a.interleaved ? 4 * j + (e >> 1) + (e & 1) * (a.rotary_dim / 4) : i;
    turns[i] = in_bounds(pair, 1, a.rotary_dim / 2, a.status) ? turns_of(a.inv_freq[pair]) : 0;
  }
}

// Sine and cosine of the lane's eight pairs at a position.  The lanes with the same channels of
// a warp's heads each compute a share of them.
struct Angles {
  float2 sin[4], cos[4];
};
template <int LANES>
__device__ __forceinline__ void angles_of(Angles &t, const uint64_t *turns, int position, int lane) {
  constexpr int kHeads = 32 / LANES, kOwn = kHeads >= 8 ? 1 : 8 / kHeads;
  const int first = lane / LANES * kOwn & 7;
  float sin[kOwn], cos[kOwn];
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    // (the upper 32 bits, to the nearest, as a signed fraction of a turn: half turns in [-1, 1))
    const uint64_t phase = turns[8 * (lane % LANES) + first + i] * static_cast<uint64_t>(static_cast<int64_t>(position));
    const float half = static_cast<float>(static_cast<int32_t>((phase + 0x80000000ull) >> 32)) * 0x1p-31f;
    sincospif(half, &sin[i], &cos[i]);
  }
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const int from = i / kOwn * LANES + lane % LANES;
    const float s = __shfl_sync(0xFFFFFFFFu, sin[i % kOwn], from), c = __shfl_sync(0xFFFFFFFFu, cos[i % kOwn], from);
    if (i & 1)
      t.sin[i >> 1].y = s, t.cos[i >> 1].y = c;
    else
      t.sin[i >> 1].x = s, t.cos[i >> 1].x = c;
  }
}

// Turns the lane's pairs, by the angle (SIGN 1) or back (-1).
template <int SIGN>
__device__ __forceinline__ void turn(Pairs &v, const Angles &t) {
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 x = v.x[i], y = v.y[i], s = SIGN > 0 ? t.sin[i] : minus(t.sin[i]);
    v.x[i] = fma_f32x2(x, t.cos[i], mul_f32x2(minus(y), s));
    v.y[i] = fma_f32x2(y, t.cos[i], mul_f32x2(x, s));
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
  } else {  // (there are slices only where 32 bits hold their number)
    const int n = static_cast<int>(i), token = n / slices, first = (n - token * slices) * per_slice;
    t = Item{token, first, min(first + per_slice, groups)};
  }
  return t;
}

// The reciprocal norm of a head, from its lane's 16 channels.
template <int LANES>
__device__ __forceinline__ float reciprocal_norm(const Pairs &v, const RopeArgs &a, float per_dim) {
  float2 sum = both(0.0f);
#pragma unroll
  for (int i = 0; i < 4; ++i) sum = fma_f32x2(v.y[i], v.y[i], fma_f32x2(v.x[i], v.x[i], sum));
  return rsqrtf(head_sum<LANES>(sum.x + sum.y) * per_dim + a.eps);
}

// A warp's way through its items, group by group.
struct Cursor {
  int64_t i;
  Item item;
  int g;
  bool more;
};
__device__ __forceinline__ Cursor cursor_at(int64_t i, int64_t items, int slices, int per_slice, int groups) {
  Cursor c;
  c.i = i;
  c.more = i < items;
  c.item = c.more ? item_of(i, slices, per_slice, groups) : Item{0, 0, 0};
  c.g = c.item.first;
  return c;
}
__device__ __forceinline__ void step_on(Cursor &c, int64_t stride, int64_t items, int slices, int per_slice, int groups) {
  if (++c.g == c.item.last) c = cursor_at(c.i + stride, items, slices, per_slice, groups);
}

// A warp's ring in shared memory: groups on their way, each lane's pieces for itself (a lane reads
// only what it copied, so that nothing but its own copies is waited for).
constexpr int kPiece = 512;  // 16 bytes of every lane
template <int PIECES, int STAGES>
struct Ring {
  static constexpr int kStage = PIECES * kPiece + 128;  // and the token's position, for every lane
  static constexpr int kBytes = STAGES * kStage;
};
constexpr int kForwardStages = 4, kBackwardStages = 3;
using ForwardRing = Ring<2, kForwardStages>;
using BackwardRing = Ring<4, kBackwardStages>;

// Queries and keys count as one row of heads: groups of the queries', then of the keys'.
template <int LANES>
__global__ void __launch_bounds__(kWarps * 32, kCtas)
    rope_kernel(const __grid_constant__ RopeArgs a, const __grid_constant__ Share share) {
  constexpr int kHeads = 32 / LANES;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint64_t turns[kRopeMaxDim / 2];  // (lanes without pairs read any)
  __shared__ Weights weights[2];
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, j = lane % LANES, sub = lane / LANES;
  const Chunks c = chunks_of(j, a);
  const float per_dim = 1.0f / static_cast<float>(a.head_dim);
  const int slices = share.slices[0], per_slice = share.per_slice[0], queries = share.groups[0];
  const int groups = queries + share.groups[1];
  const int64_t items = a.tokens * slices, stride = static_cast<int64_t>(gridDim.x) * kWarps;
  const uint32_t ring = smem_u32(smem) + warp * ForwardRing::kBytes;
  Cursor at = cursor_at(static_cast<int64_t>(warp) * gridDim.x + blockIdx.x, items, slices, per_slice, groups), ahead = at;
  const int step = kHeads * a.head_dim, own = sub * a.head_dim;
  auto copy_next = [&](int stage) {
    if (ahead.more) {
      const int k = ahead.g >= queries, group = ahead.g - (k ? queries : 0);
      const Heads &p = a.part[k];
      const bool in = c.in && group * kHeads + sub < p.heads;
      const int64_t x_at = ahead.item.token * p.ld + (group * step + own);
      const int64_t extent = (a.tokens - 1) * p.ld + static_cast<int64_t>(p.heads) * a.head_dim;
      const uint32_t to = ring + stage * ForwardRing::kStage + lane * 16;
#pragma unroll
      for (int i = 0; i < 2; ++i)
        cp_async16(to + i * kPiece, p.x + x_at + (in ? c.at[i] : 0), in && in_bounds(x_at + c.at[i], 8, extent, a.status));
      if (ahead.g == ahead.item.first && in_bounds(ahead.item.token, 1, a.tokens, a.status))
        cp_async4(ring + stage * ForwardRing::kStage + 2 * kPiece + lane * 4, a.positions + ahead.item.token);
      step_on(ahead, stride, items, slices, per_slice, groups);
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < kForwardStages - 1; ++i) copy_next(i);
  load_turns(turns, a);
  load_weights(weights[0], a.part[0].weight, a);
  load_weights(weights[1], a.part[1].weight, a);
  __syncthreads();
  Angles t;
  int stage = 0;
  while (at.more) {
    cp_async_wait<kForwardStages - 2>();
    const uint32_t from = ring + stage * ForwardRing::kStage;
    Pairs v;
    unpack(lds128(from + lane * 16), lds128(from + kPiece + lane * 16), a.interleaved, v);
    if (at.g == at.item.first && a.rotary_dim > 0)
      angles_of<LANES>(t, turns, static_cast<int>(lds32(from + 2 * kPiece + lane * 4)), lane);
    copy_next(stage == 0 ? kForwardStages - 1 : stage - 1);
    stage = stage + 1 == kForwardStages ? 0 : stage + 1;
    const int k = at.g >= queries, group = at.g - (k ? queries : 0);
    const Heads &p = a.part[k];
    if (p.weight != nullptr) {
      const float r = reciprocal_norm<LANES>(v, a, per_dim);
      Pairs w;
      weights_of(w, weights[k], j);
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v.x[i] = mul_f32x2(mul_f32x2(v.x[i], both(r)), w.x[i]);
        v.y[i] = mul_f32x2(mul_f32x2(v.y[i], both(r)), w.y[i]);
      }
    }
    if (c.turns) turn<1>(v, t);
    store(p.y, at.item.token * p.ld_y + (group * step + own + c.at[0]), c, c.in && group * kHeads + sub < p.heads, v,
          a.interleaved, (a.tokens - 1) * p.ld_y + static_cast<int64_t>(p.heads) * a.head_dim, a.status);
    step_on(at, stride, items, slices, per_slice, groups);
  }
}

// The gradients of the inputs, and each CTA's sums of those of the weights: of the queries,
// then of the keys (one part's sums in registers at a time).  The order of the sums follows
// from the sizes and the number of SMs alone: a warp's tokens in order, then the lanes, then
// the warps, then (backward_sum_kernel) the CTAs.  They are binary32: shared out so, a chain of additions is
// as long as a warp's tokens, of which there are thousands of times fewer than of all.
template <int LANES>
__global__ void __launch_bounds__(kWarps * 32, kCtas)
    rope_backward_kernel(const __grid_constant__ RopeArgs a, const __grid_constant__ Share share) {
  constexpr int kHeads = 32 / LANES;
  extern __shared__ __align__(16) uint8_t smem[];
  __shared__ uint64_t turns[kRopeMaxDim / 2];  // (lanes without pairs read any)
  __shared__ Weights weights[2];
  __shared__ float sums[kWarps][kRopeMaxDim];
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, j = lane % LANES, sub = lane / LANES;
  const Chunks c = chunks_of(j, a);
  const float per_dim = 1.0f / static_cast<float>(a.head_dim);
  const int64_t stride = static_cast<int64_t>(gridDim.x) * kWarps;
  const uint32_t ring = smem_u32(smem) + warp * BackwardRing::kBytes;
  const int step = kHeads * a.head_dim, own = sub * a.head_dim;
  Cursor at{}, ahead{};
  auto items_of = [&](int k) { return a.part[k].heads > 0 ? a.tokens * share.slices[k] : 0; };
  auto copy_next = [&](auto which, int stage) {
    constexpr int k = decltype(which)::value;
    const Heads &p = a.part[k];
    if (ahead.more) {
      const int64_t cols = static_cast<int64_t>(p.heads) * a.head_dim;
      const bool in = c.in && ahead.g * kHeads + sub < p.heads;
      const int64_t x_at = ahead.item.token * p.ld + (ahead.g * step + own);
      const int64_t dy_at = ahead.item.token * p.ld_dy + (ahead.g * step + own);
      const uint32_t to = ring + stage * BackwardRing::kStage + lane * 16;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const int d = in ? c.at[i] : 0;
        if (p.weight != nullptr)  // (without a norm the inputs are not read)
          cp_async16(to + i * kPiece, p.x + x_at + d, in && in_bounds(x_at + d, 8, (a.tokens - 1) * p.ld + cols, a.status));
        cp_async16(to + (2 + i) * kPiece, p.dy + dy_at + d,
                   in && in_bounds(dy_at + d, 8, (a.tokens - 1) * p.ld_dy + cols, a.status));
      }
      if (ahead.g == ahead.item.first && in_bounds(ahead.item.token, 1, a.tokens, a.status))
        cp_async4(ring + stage * BackwardRing::kStage + 4 * kPiece + lane * 4, a.positions + ahead.item.token);
      step_on(ahead, stride, items_of(k), share.slices[k], share.per_slice[k], share.groups[k]);
    }
    cp_async_commit();
  };
  // (the workers with one more item of the queries' are the last ones of the keys', and spread over
  // the CTAs)
  auto begin = [&](auto which) {
    constexpr int k = decltype(which)::value;
    const int64_t worker = static_cast<int64_t>(warp) * gridDim.x + blockIdx.x;
    at = cursor_at(k == 0 ? worker : stride - 1 - worker, items_of(k), share.slices[k], share.per_slice[k],
                   share.groups[k]);
    ahead = at;
#pragma unroll
    for (int i = 0; i < kBackwardStages - 1; ++i) copy_next(which, i);
  };
  Pairs dw;
  auto part = [&](auto which) {
    constexpr int k = decltype(which)::value;
    const Heads &p = a.part[k];
    const int64_t cols = static_cast<int64_t>(p.heads) * a.head_dim;
#pragma unroll
    for (int i = 0; i < 4; ++i) dw.x[i] = dw.y[i] = both(0.0f);
    Angles t;
    int stage = 0;
    while (at.more) {
      cp_async_wait<kBackwardStages - 2>();
      const uint32_t from = ring + stage * BackwardRing::kStage;
      Pairs v, n;
      unpack(lds128(from + 2 * kPiece + lane * 16), lds128(from + 3 * kPiece + lane * 16), a.interleaved, v);
      if (p.weight != nullptr) unpack(lds128(from + lane * 16), lds128(from + kPiece + lane * 16), a.interleaved, n);
      if (at.g == at.item.first && a.rotary_dim > 0)
        angles_of<LANES>(t, turns, static_cast<int>(lds32(from + 4 * kPiece + lane * 4)), lane);
      copy_next(which, stage == 0 ? kBackwardStages - 1 : stage - 1);
      stage = stage + 1 == kBackwardStages ? 0 : stage + 1;
      const bool in = c.in && at.g * kHeads + sub < p.heads;
      if (c.turns) turn<-1>(v, t);
      if (p.weight != nullptr) {
        // (others' x is 0, but r may be infinite)
        const float r = reciprocal_norm<LANES>(n, a, per_dim), own_r = in ? r : 0.0f;
        Pairs w;
        weights_of(w, weights[k], j);
        float2 dots = both(0.0f);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          n.x[i] = mul_f32x2(n.x[i], both(own_r));
          n.y[i] = mul_f32x2(n.y[i], both(own_r));
          dw.x[i] = fma_f32x2(v.x[i], n.x[i], dw.x[i]);
          dw.y[i] = fma_f32x2(v.y[i], n.y[i], dw.y[i]);
          v.x[i] = mul_f32x2(v.x[i], w.x[i]);
          v.y[i] = mul_f32x2(v.y[i], w.y[i]);
          dots = fma_f32x2(v.y[i], n.y[i], fma_f32x2(v.x[i], n.x[i], dots));
        }
        const float dot = -head_sum<LANES>(dots.x + dots.y) * per_dim;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v.x[i] = mul_f32x2(both(r), fma_f32x2(n.x[i], both(dot), v.x[i]));
          v.y[i] = mul_f32x2(both(r), fma_f32x2(n.y[i], both(dot), v.y[i]));
        }
      }
      store(p.y, at.item.token * p.ld_y + (at.g * step + own + c.at[0]), c, in, v, a.interleaved,
            (a.tokens - 1) * p.ld_y + cols, a.status);
      step_on(at, stride, items_of(k), share.slices[k], share.per_slice[k], share.groups[k]);
    }
  };
  auto add_up = [&](int k) {
    if (a.partials == nullptr) return;
    __syncthreads();  // (the queries' sums are read)
#pragma unroll
    for (int e = 0; e < 16; ++e) {
      const float2 &d = (e & 8 ? dw.y : dw.x)[(e & 7) >> 1];
      float s = e & 1 ? d.y : d.x;
#pragma unroll
      for (int m = 16; m >= LANES; m >>= 1) s += __shfl_xor_sync(0xFFFFFFFFu, s, m);
      if (lane < LANES && c.in) sums[warp][channel_of(c, a.interleaved, e & 7, e >> 3)] = s;
    }
    __syncthreads();
    for (int d = threadIdx.x; d < a.head_dim; d += kWarps * 32) {
      float s = sums[0][d];
#pragma unroll
      for (int w = 1; w < kWarps; ++w) s += sums[w][d];
      const int64_t to = (static_cast<int64_t>(blockIdx.x) * 2 + k) * a.head_dim + d;
      if (in_bounds(to, 1, kRopeBackCtas * 2 * a.head_dim, a.status)) a.partials[to] = s;
    }
  };
  const std::integral_constant<int, 0> queries;
  const std::integral_constant<int, 1> keys;
  begin(queries);
  load_turns(turns, a);
  load_weights(weights[0], a.part[0].weight, a);
  load_weights(weights[1], a.part[1].weight, a);
  __syncthreads();
  part(queries);
  cp_async_wait<0>();
  begin(keys);  // (on their way while the queries' sums are added up)
  add_up(0);
  part(keys);
  add_up(1);
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
      const int64_t at = static_cast<int64_t>(p) * 2 * a.head_dim + i;
      if (p < ctas && in_bounds(at, 1, kRopeBackCtas * 2 * a.head_dim, a.status)) s += a.partials[at];
    }
  }
  sums[warp][lane] = s;
  __syncthreads();
  if (warp != 0 || i >= 2 * a.head_dim) return;
#pragma unroll
  for (int w = 1; w < kSumWarps; ++w) s += sums[w][lane];
  const int k = i >= a.head_dim;
  float *out = a.part[k].dweight;
  if (out != nullptr && in_bounds(i - k * a.head_dim, 1, a.head_dim, a.status)) out[i - k * a.head_dim] = s;
}
static_assert(kRopeBackCtas % kSumWarps == 0, "all partials are summed");

int lanes_of(int head_dim) {
  int lanes = 1;
  while (16 * lanes < head_dim) lanes *= 2;
  return lanes;
}

Share share_of(const RopeArgs &a, int lanes, int64_t warps, bool together) {
  const int heads = 32 / lanes;
  Share s;
  for (int k = 0; k < 2; ++k) s.groups[k] = (a.part[k].heads + heads - 1) / heads;
  for (int k = 0; k < 2; ++k)
    rope_slices(a.tokens, together ? s.groups[0] + s.groups[1] : s.groups[k], warps, &s.slices[k], &s.per_slice[k]);
  return s;
}

cudaError_t allow_smem(const void *func, int bytes) {
  if (kernel_setup_get(func, nullptr)) return cudaSuccess;
  const cudaError_t e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
  if (e == cudaSuccess) kernel_setup_put(func, 0);
  return e;
}

template <int LANES>
cudaError_t forward(const RopeArgs &a, cudaStream_t s) {
  const int64_t most = static_cast<int64_t>(a.num_sms) * kCtas;
  const Share share = share_of(a, LANES, most * kWarps, true);
  const int64_t ctas = (a.tokens * share.slices[0] + kWarps - 1) / kWarps;
  constexpr int kSmem = kWarps * ForwardRing::kBytes;
  const cudaError_t e = allow_smem(reinterpret_cast<const void *>(rope_kernel<LANES>), kSmem);
  if (e != cudaSuccess) return e;
  return launch_pdl(rope_kernel<LANES>, dim3(static_cast<unsigned>(ctas < most ? ctas : most)),
                    dim3(kWarps * 32), kSmem, s, a, share);
}

template <int LANES>
cudaError_t backward(const RopeArgs &a, cudaStream_t s) {
  int64_t most = static_cast<int64_t>(a.num_sms) * kCtas;
  if (most > kRopeBackCtas) most = kRopeBackCtas;
  const Share share = share_of(a, LANES, most * kWarps, false);
  const int64_t slices = share.slices[0] > share.slices[1] ? share.slices[0] : share.slices[1];
  int64_t ctas = (a.tokens * slices + kWarps - 1) / kWarps;
  ctas = ctas < 1 ? 1 : ctas < most ? ctas : most;
  constexpr int kSmem = kWarps * BackwardRing::kBytes;
  cudaError_t e = allow_smem(reinterpret_cast<const void *>(rope_backward_kernel<LANES>), kSmem);
  if (e == cudaSuccess)
    e = launch_pdl(rope_backward_kernel<LANES>, dim3(static_cast<unsigned>(ctas)), dim3(kWarps * 32), kSmem, s, a, share);
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
