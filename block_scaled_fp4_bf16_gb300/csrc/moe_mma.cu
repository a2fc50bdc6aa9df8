// The experts' products on the FP4 tensor cores, activations as sums of FP4.
//
// The weights' bytes bound these products, so no instruction should touch a
// weight: codes and scales go from memory to the block-scaled FP4 product as
// they lie.  For that the activations have to be FP4 too, without losing their
// digits: a value is written as a sum of eight E2M1 digits,
//     x = 2^e (q_0 + 2^-2 q_1 + 2^-5 q_2 + ... + 2^-20 q_7),   e for its block,
// each digit the rounding of what the ones before it left (what is left after
// q_0 is at most 1 of 6, after every other at most 1/2 of 4, so eight digits
// reach 2^-21 of the block's scale: a BF16 value is exact unless its last bit
// lies below that).  The digits of a token are eight rows of the product's
// narrow operand, and the epilogue adds their eight sums in binary32.  The FP4
// rate makes the eightfold product cheaper than converting the weights: M = 128,
// N = 32 (four tokens), K = 64 a step.
//
// split_kernel makes the digits (an "image": for a row and 256 elements of K the
// eight rows of 128 bytes as the product reads them, 128-byte swizzle included,
// and their scales), expert_mma_kernel streams weights and images.  The images'
// rows are the (token, slot) pairs sorted by expert, so that a group's lie
// together and come with two copies a stage.
#include <cuda_fp16.h>

#include "moe_groups.cuh"

namespace mx {
namespace {

constexpr int kDigits = 8;
constexpr int kImageK = 256;                   // elements of K of a stage
constexpr int kImageCodes = kDigits * 128;     // bytes of codes
// Bytes of a group's scales: a scale tile of 128 rows (16 pairs' digits) and four
// blocks, two (MXFP4) or four (NVFP4) of them a stage.
template <int FMT>
constexpr int kImageScales = (FMT == 0 ? 2 : 4) * 512;
static_assert(kMoeGroupMax * kDigits == 128, "a group's digits fill a scale tile");
// Weight of digit p: 2^-kShift[p].
__host__ __device__ constexpr int digit_shift(int p) { return p == 0 ? 0 : 3 * p - 1; }

struct SplitParams {
  const void *x;        // x: BF16 rows; h: the partial sums [parts][2][pairs][k]
  int64_t ld, extent;   // row stride, elements from x's base (bounds-checked build)
  int parts, gelu;      // h
  int k, stages;
  const int32_t *ids;   // [pairs]
  int pairs, experts;
  int top_k, group;     // pairs of a group at most
  uint8_t *codes;       // [stages][pairs][kImageCodes], rows by place
  uint8_t *scales;      // [stages][groups][kImageScales]
  float *factors;       // NVFP4: [pairs], the power of two of a place
  char *plan;           // Groups and the places' members (written for x, read for h)
  uint32_t *status;
};

constexpr int kSplitWarps = 8;

// Largest e with |v| <= 6 * 2^e for |v| <= top, as small as it can be; top > 0.
__device__ __forceinline__ int block_exponent(float top) {
  const uint32_t u = __float_as_uint(top);
  if (u < 0x00800000u) return -127;  // subnormal: 2^-126 at most
  const int e = static_cast<int>(u >> 23) - 127;
  return (u & 0x007FFFFFu) > 0x00400000u ? e - 1 : e - 2;
}

// 2^e for -149 <= e <= 127.
__device__ __forceinline__ float pow2(int e) {
  return e >= -126 ? __uint_as_float(static_cast<uint32_t>(e + 127) << 23)
                   : __uint_as_float(1u << (e + 149));
}

// v += eight floats.
__device__ __forceinline__ void add8(const SplitParams &p, int64_t off, float (&v)[8]) {
  if (!in_bounds(off, 8, p.extent, p.status)) return;
  const float4 *src = reinterpret_cast<const float4 *>(static_cast<const float *>(p.x) + off);
  const float4 a = src[0], b = src[1];
  v[0] += a.x, v[1] += a.y, v[2] += a.z, v[3] += a.w;
  v[4] += b.x, v[5] += b.y, v[6] += b.z, v[7] += b.w;
}

// Eight consecutive elements of row r of x, or of h = act(gate) up, from `at`
// (zeros past k).
template <typename XT>
__device__ __forceinline__ void load8(const SplitParams &p, int r, int at, float (&v)[8]) {
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = 0.0f;
  if (at >= p.k) return;
  if constexpr (sizeof(XT) == 2) {
    const int64_t off = r * p.ld + at;
    if (!in_bounds(off, 8, p.extent, p.status)) return;
    const uint4 q = *reinterpret_cast<const uint4 *>(static_cast<const XT *>(p.x) + off);
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      v[2 * i] = __uint_as_float(w[i] << 16);
      v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
  } else {
    float u[8] = {};
    for (int s = 0; s < p.parts; ++s) {
      add8(p, (static_cast<int64_t>(2 * s) * p.pairs + r) * p.ld + at, v);
      add8(p, (static_cast<int64_t>(2 * s + 1) * p.pairs + r) * p.ld + at, u);
    }
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
      const float2 a = p.gelu ? gelu_f32x2(make_float2(v[i], v[i + 1]))
                              : make_float2(v[i] / (1.0f + expf(-v[i])),
                                            v[i + 1] / (1.0f + expf(-v[i + 1])));
      v[i] = a.x * u[i];
      v[i + 1] = a.y * u[i + 1];
    }
  }
}

// Row blockIdx.y (x: a token, which goes to the places of its pairs; h: a place),
// stages blockIdx.x * kSplitWarps ..: a warp makes the image of one stage, eight
// elements a lane.  MXFP4: UE8M0 scales for 32 (four lanes), digit p
// with the scale 2^(e - shift p); NVFP4: E4M3 for 16 (two lanes), a power of two
// relative to the row's factor, the digits' weights left to the reader.  A block
// that holds an infinity or NaN gets the scale NaN.
template <int FMT, typename XT>
__global__ void __launch_bounds__(kSplitWarps * 32) split_kernel(const SplitParams p) {
  __shared__ float tops[kSplitWarps];
  constexpr int kPairs = kMoeMaxTokens * kMoeMaxTopK;
  constexpr bool kGather = sizeof(XT) == 2;  // x: tokens to places
  __shared__ __align__(16) char groups[kGather ? Groups::bytes(kPairs) : 16];
  __shared__ __align__(16) char scratch[kGather ? 2 * (kSplitWarps + 2) * kMoeMaxExperts : 16];
  __shared__ uint16_t places[kGather ? kPairs : 1], members[kGather ? kPairs : 1];
  griddep_launch_dependents();
  griddep_wait();
  const int r = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint16_t *plan_members = reinterpret_cast<uint16_t *>(p.plan + Groups::bytes(p.pairs));
  if constexpr (kGather) {
    make_groups<kSplitWarps>(Groups::at(groups, p.pairs), places, members, scratch, p.ids, p.pairs,
                             p.experts, p.group, p.status);
    if (blockIdx.x == 0 && r == 0) {
      for (int i = threadIdx.x; i < Groups::bytes(p.pairs) / 4; i += kSplitWarps * 32)
        reinterpret_cast<uint32_t *>(p.plan)[i] = reinterpret_cast<const uint32_t *>(groups)[i];
      for (int i = threadIdx.x; i < p.pairs; i += kSplitWarps * 32) plan_members[i] = members[i];
    }
  } else {
    // the places behind the last group's are empty
    const Groups g = Groups::at(p.plan, p.pairs);
    const int n = *g.count;
    if (n == 0 || r >= g.begin[n - 1] + g.size[n - 1]) return;
  }
  const int stage = blockIdx.x * kSplitWarps + warp;
  float v[8];
  load8<XT>(p, r, stage * kImageK + lane * 8, v);
  int row_e = 0;  // NVFP4: exponent of the row's factor
  if constexpr (FMT == 1) {
    float top = 0.0f;  // of the row's finite elements
    const auto raise = [&](const float (&u)[8]) {
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float a = fabsf(u[i]);
        if (a < __uint_as_float(0x7F800000u)) top = fmaxf(top, a);
      }
    };
    raise(v);
    for (int s = warp; s < p.stages; s += kSplitWarps) {
      if (s == stage) continue;
      float u[8];
      load8<XT>(p, r, s * kImageK + lane * 8, u);
      raise(u);
    }
    top = __uint_as_float(__reduce_max_sync(0xFFFFFFFFu, __float_as_uint(top)));
    if (lane == 0) tops[warp] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < kSplitWarps; ++w) top = fmaxf(top, tops[w]);
    // the largest block's scale becomes 2^8, the largest power of two of E4M3
    row_e = max(block_exponent(top) - 8, -118);
    if (blockIdx.x == 0) {
      if constexpr (kGather) {
        if (threadIdx.x < static_cast<unsigned>(p.top_k)) {
          const int at = places[r * p.top_k + threadIdx.x];
          if (at != 0xFFFF) p.factors[at] = pow2(row_e);
        }
      } else if (threadIdx.x == 0) {
        p.factors[r] = pow2(row_e);
      }
    }
  }
  if (stage >= p.stages) return;
  float top = 0.0f;
  uint32_t odd = 0;  // an infinity or NaN here
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    top = fmaxf(top, fabsf(v[i]));
    odd |= (__float_as_uint(v[i]) & 0x7F800000u) == 0x7F800000u;
  }
#pragma unroll
  for (int m = 1; m < (FMT == 0 ? 4 : 2); m <<= 1) {
    top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, m));
    odd |= __shfl_xor_sync(0xFFFFFFFFu, odd, m);
  }
  int e = block_exponent(top);
  uint32_t byte;
  if constexpr (FMT == 0) {
    e = max(e, -127);
    byte = odd ? 255u : static_cast<uint32_t>(e + 127);
  } else {
    const int j = min(max(e - row_e, -9), 8);  // 2^-9 is E4M3's least
    e = row_e + j;
    byte = odd ? 0x7Fu : j >= -6 ? static_cast<uint32_t>(j + 7) << 3 : 1u << (j + 9);
  }
  // the places of this row
  const int copies = kGather ? p.top_k : 1;
  const auto place = [&](int j) { return kGather ? static_cast<int>(places[r * p.top_k + j]) : r; };
  // v 2^-e, in two steps where one power of two would not be a normal number
  const float f0 = pow2(min(-e, 100)), f1 = pow2(-e - min(-e, 100));
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = odd ? 0.0f : v[i] * f0 * f1;
#pragma unroll
  for (int d = 0; d < kDigits; ++d) {
    uint32_t w = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint32_t c = cvt_e2m1x2(v[2 * i], v[2 * i + 1]);
      uint32_t h;
      asm("{\n .reg .b8 t;\n cvt.u8.u32 t, %1;\n cvt.rn.f16x2.e2m1x2 %0, t;\n}\n" : "=r"(h) : "r"(c));
      const float2 q = __half22float2(*reinterpret_cast<const __half2 *>(&h));
      const float up = d == 0 ? 4.0f : 8.0f;
      v[2 * i] = (v[2 * i] - q.x) * up;
      v[2 * i + 1] = (v[2 * i + 1] - q.y) * up;
      w |= c << (8 * i);
    }
    if (FMT == 0 && digit_shift(d) > e + 127) w = 0;  // no scale that small
    // row d of the 8 x 128 byte tile, 16-byte chunk lane / 4, swizzled
    const int at = d * 128 + (((lane >> 2) ^ d) << 4) + (lane & 3) * 4;
    for (int j = 0; j < copies; ++j) {
      const int to = place(j);
      if (to != 0xFFFF)
        *reinterpret_cast<uint32_t *>(
            p.codes + (static_cast<int64_t>(stage) * p.pairs + to) * kImageCodes + at) = w;
    }
  }
  // scale words of four blocks, for each digit's row
  constexpr int kWords = FMT == 0 ? 2 : 4;
  uint32_t words[kWords] = {};
#pragma unroll
  for (int b = 0; b < 4 * kWords; ++b)
    words[b / 4] |= __shfl_sync(0xFFFFFFFFu, byte, b * (8 / kWords)) << (8 * (b % 4));
  if (lane < kDigits) {
#pragma unroll
    for (int i = 0; i < kWords; ++i) {
      uint32_t w = words[i];
      if constexpr (FMT == 0) {
        // 255 stays NaN; a digit whose scale would lie below 2^-127 is 0
        const uint32_t nan = __vcmpeq4(w, 0xFFFFFFFFu);
        w = __vsubus4(w, (lane == 0 ? 0u : 3u * lane - 1u) * 0x01010101u) | nan;
      }
      for (int j = 0; j < copies; ++j) {
        const int to = place(j);
        if (to == 0xFFFF) continue;
        // digit rows of a group in the order of a scale tile: row c at c % 32, word c / 32
        const int member = kGather ? members[to] : plan_members[to];
        const int m = member % kMoeGroupMax;
        *reinterpret_cast<uint32_t *>(
            p.scales +
            (static_cast<int64_t>(stage) * p.pairs + member / kMoeGroupMax) * kImageScales<FMT> +
            i * 512 + ((m & 3) * kDigits + lane) * 16 + (m >> 2) * 4) = w;
      }
    }
  }
}

// ---------------------------------------------------------------- the product

constexpr int kMmaWarps = 6;  // copies, product, four of the epilogue
constexpr int kMmaThreads = kMmaWarps * 32;
constexpr int kMaxSlots = 16;
constexpr int kMmaSmem = 227 * 1024;

struct MmaParams {
  MoeArgs a;
  const uint8_t *image, *image_scales;
  const float *factors;
  int stages;     // of 256 along K
  int tiles;      // 128-row tiles of an expert
  int parts;      // ranges of K, each an item with sums of its own
  int slots;      // stages in flight
  int bufs;       // accumulators (1 or 2)
  int b_off, sfa_off, sfb_off, bar_off, groups_at;  // shared memory (the weights at 0)
};

// UP: gate and up rows, h's partial sums as output; else rows of `hidden`, z's.
// An item is 128 rows (of each matrix) times a group's pairs over one range of
// K; a CTA walks consecutive items, group-major.  A product reads its 128 weight
// rows from shared memory in about 100 clocks however few columns it has
// (measured: 64-row tiles take as long as 128-row ones), so the tiles are whole and a
// call with few items divides K instead.
//
// Shared memory: a ring of stages: weights (128 rows x 128 bytes of each matrix),
// images (a kilobyte a pair), scale tiles of the weights and of the group.
// Tensor memory: accumulators [bufs][SEGS][NB][32 columns], then a set of
// scale columns for each stage in flight, four columns for each scale tile.
template <int FMT, bool UP, int NB>
__global__ void __launch_bounds__(kMmaThreads, 1)
    expert_mma_kernel(const __grid_constant__ CUtensorMap map0,
                      const __grid_constant__ CUtensorMap map1, const __grid_constant__ MmaParams p) {
  constexpr int kSegs = UP ? 2 : 1;
  constexpr int kAtoms = FMT == 0 ? 2 : 4;       // scale tiles (4 blocks) of a stage
  constexpr int kSfa = kAtoms * 512;             // bytes, of one matrix
  constexpr int kSfaCols = kAtoms * 4;
  constexpr int kSfb = kImageScales<FMT>;
  constexpr int kTile = 128 * 128;               // bytes of a stage's weights, of one matrix
  extern __shared__ __align__(1024) char smem[];
  const MoeArgs &a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  constexpr int kGroup = 4 * NB;  // tokens of a group at most
  const int slots = p.slots;
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + p.bar_off);
  uint64_t *empty = full + slots;
  uint64_t *acc_full = empty + slots;   // [2]
  uint64_t *acc_empty = acc_full + 2;   // [2]
  uint64_t *done = acc_empty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
  volatile uint32_t *abort = tmem_slot + 1;
  if (smem_u32(smem) & 1023u) {  // the 128-byte swizzle needs 1024-byte aligned tiles
    if (threadIdx.x == 0) atomicOr(a.status, kStatusTimeout);
    return;
  }
  if (threadIdx.x == 0) {
    for (int s = 0; s < slots; ++s) {
      mbar_init(smem_u32(&full[s]), 1);
      mbar_init(smem_u32(&empty[s]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&acc_full[i]), 1);
      mbar_init(smem_u32(&acc_empty[i]), 4);
    }
    mbar_init(smem_u32(done), 1);
    *abort = 0u;
    fence_barrier_init();
    prefetch_tmap(&map0);
    if (UP) prefetch_tmap(&map1);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;
  griddep_launch_dependents();
  griddep_wait();
  const int pairs = a.tokens * a.top_k;
  for (int i = threadIdx.x; i < Groups::bytes(pairs) / 16; i += kMmaThreads)
    reinterpret_cast<uint4 *>(smem + p.groups_at)[i] = reinterpret_cast<const uint4 *>(a.plan)[i];
  __syncthreads();
  const Groups g = Groups::at(smem + p.groups_at, pairs);
  const int64_t items = static_cast<int64_t>(*g.count) * p.tiles * p.parts;
  const int begin = static_cast<int>(items * blockIdx.x / gridDim.x);
  const int end = static_cast<int>(items * (blockIdx.x + 1) / gridDim.x);
  const int rows = UP ? a.inter : a.hidden, k = UP ? a.hidden : a.inter;
  const int katoms = (k / (FMT == 0 ? 32 : 16) + 3) >> 2;  // scale tiles along K
  const int group_items = p.tiles * p.parts;
  // an item's group, row tile and range of K
  struct Item {
    int grp, tile, part, st0, st1;
  };
  const auto item_at = [&](int item) {
    Item i;
    i.grp = item / group_items;
    const int r = item - i.grp * group_items;
    i.tile = r / p.parts;
    i.part = r - i.tile * p.parts;
    i.st0 = p.stages * i.part / p.parts;
    i.st1 = p.stages * (i.part + 1) / p.parts;
    return i;
  };
  constexpr int acc_cols = kSegs * NB * 32;
  const uint32_t sf_tmem = tmem + p.bufs * acc_cols;
  constexpr int sf_cols = (kSegs + 1) * kSfaCols;

  if (warp == 0) {
    // ------------------------------------------------------------ copies
    uint32_t it = 0, s = 0, ph = 0;
    bool ok = true;
    for (int item = begin; item < end && ok; ++item) {
      const Item im = item_at(item);
      const int grp = im.grp, e = g.expert[grp], n = g.size[grp];
      const int row0 = im.tile * 128;
      const int64_t scale_off =
          (static_cast<int64_t>(e) * p.tiles + im.tile) * static_cast<int64_t>(katoms) * 512;
      const uint8_t *sf0 = (UP ? a.gate.scales : a.down.scales) + scale_off;
      const uint8_t *sf1 = UP ? a.up.scales + scale_off : nullptr;
      const int64_t place = g.begin[grp];
      for (int st = im.st0; st < im.st1; ++st, ++it) {
        if (!mbar_wait_warp(smem_u32(&empty[s]), ph ^ 1u, abort, a.status)) {
          ok = false;
          break;
        }
        const uint32_t fb = smem_u32(&full[s]);
        const uint32_t sf_bytes = static_cast<uint32_t>(min(kAtoms, katoms - st * kAtoms)) * 512u;
        if (elect_one()) {
          mbar_arrive_expect_tx(fb, kSegs * (kTile + sf_bytes) + n * kImageCodes + kSfb);
          const uint32_t w = smem_u32(smem) + s * kSegs * kTile;
          const uint32_t sf = smem_u32(smem + p.sfa_off) + s * kSegs * kSfa;
          tma_load_2d(w, &map0, st * 128, e * rows + row0, fb);
          bulk_load(sf, sf0 + static_cast<int64_t>(st) * kSfa, sf_bytes, fb);
          if constexpr (UP) {
            tma_load_2d(w + kTile, &map1, st * 128, e * rows + row0, fb);
            bulk_load(sf + kSfa, sf1 + static_cast<int64_t>(st) * kSfa, sf_bytes, fb);
          }
          const int64_t at = static_cast<int64_t>(st) * pairs;
          bulk_load(smem_u32(smem + p.b_off) + s * kGroup * kImageCodes,
                    p.image + (at + place) * kImageCodes, n * kImageCodes, fb);
          bulk_load(smem_u32(smem + p.sfb_off) + s * kSfb, p.image_scales + (at + grp) * kSfb, kSfb,
                    fb);
        }
        __syncwarp();
        if (++s == static_cast<uint32_t>(slots)) s = 0, ph ^= 1u;
      }
    }
    // no copy may land after the CTA has left
    const uint32_t inflight = it < static_cast<uint32_t>(slots) ? it : static_cast<uint32_t>(slots);
    for (uint32_t j = it - inflight; j < it; ++j)
      mbar_drain(smem_u32(&full[j % slots]), (j / slots) & 1u);
  } else if (warp == 1) {
    // ------------------------------------------------------------ product
    uint32_t s = 0, ph = 0, buf = 0, bph = 0;
    bool ok = true;
    // One thread issues every product, so a product has to cost it few
    // instructions: the loops are unrolled and descriptors stepped by constants.
    const uint32_t w_ring = smem_u32(smem), b_ring = smem_u32(smem + p.b_off);
    const uint32_t sfa_ring = smem_u32(smem + p.sfa_off), sfb_ring = smem_u32(smem + p.sfb_off);
    for (int item = begin; item < end && ok; ++item) {
      const Item im = item_at(item);
      const int grp = im.grp;
      // columns: the digits of the group, to a multiple of 16
      const uint32_t columns = static_cast<uint32_t>(g.size[grp] * kDigits + 15) & ~15u;
      const uint32_t idesc0 = mma_idesc<FMT>(128, columns, 0);
      const uint32_t idesc2 = mma_idesc<FMT>(128, columns, 2);
      ok = mbar_wait_warp(smem_u32(&acc_empty[buf]), bph ^ 1u, abort, a.status);
      if (!ok) break;
      tc_fence_after();
      const uint32_t acc = tmem + buf * acc_cols;
      for (int st = im.st0; st < im.st1; ++st) {
        if (!mbar_wait_warp(smem_u32(&full[s]), ph, abort, a.status)) {
          ok = false;
          break;
        }
        tc_fence_after();
        if (elect_one()) {
          const uint32_t sfa_t = sf_tmem + s * sf_cols, sfb_t = sfa_t + kSegs * kSfaCols;
          const uint64_t sfa = smem_desc_scale_block(sfa_ring + s * kSegs * kSfa);
          const uint64_t sfb = smem_desc_scale_block(sfb_ring + s * kSfb);
          const int atoms = min(kAtoms, katoms - st * kAtoms);
          const int steps = min(4, (k - st * kImageK + 63) >> 6);  // of 64 inside K
#pragma unroll
          for (int j = 0; j < kAtoms; ++j)
            tc_cp_32x128b_warpx4(sfb_t + j * 4, sfb + ((j * 512) >> 4));
#pragma unroll
          for (int m = 0; m < kSegs; ++m) {
#pragma unroll
            for (int i = 0; i < kAtoms; ++i) {
              if (i < atoms)
                tc_cp_32x128b_warpx4(sfa_t + m * kSfaCols + i * 4,
                                     sfa + ((m * kSfa + i * 512) >> 4));
            }
          }
          const uint64_t wd = smem_desc_sw128_kmajor(w_ring + s * kSegs * kTile);
          const uint64_t bd = smem_desc_sw128_kmajor(b_ring + s * kGroup * 1024);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            if (kk < steps) {
              const int word = FMT == 0 ? kk >> 1 : kk;
              const uint32_t idesc = FMT == 0 && (kk & 1) ? idesc2 : idesc0;
#pragma unroll
              for (int m = 0; m < kSegs; ++m)
                tc_mma_block_scaled<FMT>(acc + m * NB * 32, wd + m * (kTile >> 4) + 2 * kk,
                                         bd + 2 * kk, idesc, sfa_t + m * kSfaCols + word * 4,
                                         sfb_t + word * 4, kk > 0 || st > im.st0 ? 1u : 0u);
            }
          }
          tc_commit(smem_u32(&empty[s]));
          if (st == im.st1 - 1) tc_commit(smem_u32(&acc_full[buf]));
        }
        __syncwarp();
        if (++s == static_cast<uint32_t>(slots)) s = 0, ph ^= 1u;
      }
      if (++buf == static_cast<uint32_t>(p.bufs)) buf = 0, bph ^= 1u;
    }
    // every product issued has finished before the tensor memory goes
    if (elect_one()) tc_commit(smem_u32(done));
    __syncwarp();
    mbar_drain(smem_u32(done), 0u);
  } else {
    // ------------------------------------------------------------ epilogue
    const int q = warp & 3;  // this warp's lane quarter
    uint32_t buf = 0, bph = 0;
    const int64_t out_extent = static_cast<int64_t>(p.parts) * kSegs * pairs * rows;
    for (int item = begin; item < end; ++item) {
      const Item im = item_at(item);
      const int grp = im.grp, e = g.expert[grp], n = g.size[grp];
      const int row = im.tile * 128 + q * 32 + lane;
      const float alpha0 = FMT == 1 ? (UP ? a.gate.ts : a.down.ts)[e] : 1.0f;
      const float alpha1 = FMT == 1 && UP ? a.up.ts[e] : 1.0f;
      if (!mbar_wait_warp(smem_u32(&acc_full[buf]), bph, abort, a.status)) break;
      tc_fence_after();
      const uint32_t acc = tmem + buf * acc_cols + (static_cast<uint32_t>(q * 32) << 16);
      for (int i = 0; i < (n + 3) / 4; ++i) {
        float sum[kSegs][4];
#pragma unroll
        for (int m = 0; m < kSegs; ++m) {
          uint32_t r[32];
          tc_ld_32x32b_x32(acc + (m * NB + i) * 32, r);
          tc_wait_ld();
          // the digits' sums, the least first
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float t = 0.0f;
#pragma unroll
            for (int d = kDigits - 1; d >= 0; --d) {
              const float v = __uint_as_float(r[j * 8 + d]);
              if constexpr (FMT == 0)
                t = __fadd_rn(t, v);
              else
                t = __fmaf_rn(v, 1.0f / static_cast<float>(1 << digit_shift(d)), t);
            }
            sum[m][j] = t;
          }
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const int c = i * 4 + j;
          if (c >= n || row >= rows) continue;
          const int place = g.begin[grp] + c, pair = g.list[place];
          const float f = FMT == 1 ? p.factors[place] : 1.0f;
#pragma unroll
          for (int m = 0; m < kSegs; ++m) {
            const float v = FMT == 1 ? sum[m][j] * f * (m == 0 ? alpha0 : alpha1) : sum[m][j];
            const int64_t o = (static_cast<int64_t>(im.part * kSegs + m) * pairs +
                               (UP ? place : pair)) * rows + row;
            if (in_bounds(o, 1, out_extent, a.status)) (UP ? a.h : a.z)[o] = v;
          }
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&acc_empty[buf]));
      if (++buf == static_cast<uint32_t>(p.bufs)) buf = 0, bph ^= 1u;
    }
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// Pairs of a group: the product takes them together, in quarters of 32 columns.
int group_size(const MoeArgs &a) { return a.tokens <= 4 ? 4 : a.tokens <= 8 ? 8 : 16; }

// The images in the workspace: codes of x, scales of x, codes of h, scales of h.
struct Images {
  uint8_t *codes, *scales;
};
Images images(const MoeArgs &a, bool of_h) {
  const int64_t pairs = static_cast<int64_t>(a.tokens) * a.top_k;
  uint8_t *at = a.image + (of_h ? moe_image_bytes(pairs, a.hidden) : 0);
  const int64_t stages = ((of_h ? a.inter : a.hidden) + kImageK - 1) / kImageK;
  return Images{at, at + pairs * stages * kImageCodes};
}

template <int FMT, typename XT>
cudaError_t launch_split(const MoeArgs &a, const void *x, int64_t ld, int rows, int k, Images out,
                         float *factors, cudaStream_t s) {
  SplitParams p{};
  p.x = x;
  p.ld = ld;
  p.extent = sizeof(XT) == 2 ? (rows - 1) * ld + k
                             : static_cast<int64_t>(a.up_parts) * 2 * rows * k;
  p.parts = a.up_parts;
  p.gelu = a.gelu;
  p.k = k;
  p.stages = (k + kImageK - 1) / kImageK;
  p.ids = a.ids;
  p.pairs = a.tokens * a.top_k;
  p.experts = a.experts;
  p.top_k = a.top_k;
  p.group = group_size(a);
  p.plan = a.plan;
  p.codes = out.codes;
  p.scales = out.scales;
  p.factors = factors;
  p.status = a.status;
  return launch_pdl(split_kernel<FMT, XT>, dim3((p.stages + kSplitWarps - 1) / kSplitWarps, rows),
                    dim3(kSplitWarps * 32), 0, s, p);
}

template <int FMT, bool UP, int NB>
cudaError_t launch_mma(const MoeArgs &a, Images image, const float *factors, cudaStream_t s) {
  constexpr int kSegs = UP ? 2 : 1, kAtoms = FMT == 0 ? 2 : 4;
  const auto kernel = expert_mma_kernel<FMT, UP, NB>;
  const void *func = reinterpret_cast<const void *>(kernel);
  if (!kernel_setup_get(func, nullptr)) {
    const cudaError_t e =
        cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, kMmaSmem);
    if (e != cudaSuccess) return e;
    kernel_setup_put(func, 0);
  }
  const int rows = UP ? a.inter : a.hidden, k = UP ? a.hidden : a.inter;
  const int pairs = a.tokens * a.top_k;
  MmaParams p{};
  p.a = a;
  p.image = image.codes;
  p.image_scales = image.scales;
  p.factors = factors;
  p.stages = (k + kImageK - 1) / kImageK;
  constexpr int kGroup = 4 * NB;
  p.tiles = (rows + 127) / 128;
  p.parts = UP ? a.up_parts : a.down_parts;
  constexpr int kTile = 128 * 128;
  constexpr int per_slot =
      kSegs * (kTile + kAtoms * 512) + kGroup * kImageCodes + kImageScales<FMT>;
  const int fixed = 512 + Groups::bytes(pairs);
  constexpr int sf_cols = (kSegs + 1) * kAtoms * 4, acc = kSegs * NB * 32;
  int slots = (kMmaSmem - fixed) / per_slot;
  slots = slots < kMaxSlots ? slots : kMaxSlots;
  p.bufs = 2 * acc + 4 * sf_cols <= 512 ? 2 : 1;
  const int tmem_slots = (512 - p.bufs * acc) / sf_cols;
  p.slots = slots < tmem_slots ? slots : tmem_slots;
  if (p.slots < 2) return cudaErrorInvalidValue;
  p.b_off = p.slots * kSegs * kTile;
  p.sfa_off = p.b_off + p.slots * kGroup * 1024;
  p.sfb_off = p.sfa_off + p.slots * kSegs * kAtoms * 512;
  p.bar_off = p.sfb_off + p.slots * kImageScales<FMT>;
  p.groups_at = (p.bar_off + 8 * (2 * p.slots + 5) + 16 + 15) / 16 * 16;
  const int smem = p.groups_at + Groups::bytes(pairs);
  if (smem > kMmaSmem) return cudaErrorInvalidValue;
  CUtensorMap map0, map1;
  const int64_t stacked = static_cast<int64_t>(a.experts) * rows;
  if (!encode_codes_window_map(&map0, UP ? a.gate.codes : a.down.codes, stacked, k, 128) ||
      !encode_codes_window_map(&map1, UP ? a.up.codes : a.down.codes, stacked, k, 128))
    return cudaErrorInvalidValue;
  const int most = a.experts < pairs ? a.experts : pairs;  // experts with a pair
  const int64_t items = static_cast<int64_t>(most + pairs / kGroup) * p.tiles * p.parts;
  const int grid = items < a.num_sms ? static_cast<int>(items) : a.num_sms;
  return launch_pdl(kernel, dim3(grid), dim3(kMmaThreads), smem, s, map0, map1, p);
}

template <int FMT, bool UP>
cudaError_t launch_product(const MoeArgs &a, Images image, const float *factors, cudaStream_t s) {
  if (a.tokens <= 4) return launch_mma<FMT, UP, 1>(a, image, factors, s);
  if (a.tokens <= 8) return launch_mma<FMT, UP, 2>(a, image, factors, s);
  return launch_mma<FMT, UP, 4>(a, image, factors, s);
}

template <int FMT>
cudaError_t launch_all(const MoeArgs &a, cudaStream_t s) {
  const int pairs = a.tokens * a.top_k;
  const Images x = images(a, false), h = images(a, true);
  cudaError_t e =
      launch_split<FMT, uint16_t>(a, a.x, a.ld_x, a.tokens, a.hidden, x, a.factors, s);
  if (e == cudaSuccess) e = launch_product<FMT, true>(a, x, a.factors, s);
  if (e == cudaSuccess)
    e = launch_split<FMT, float>(a, a.h, a.inter, pairs, a.inter, h, a.factors + pairs, s);
  if (e == cudaSuccess) e = launch_product<FMT, false>(a, h, a.factors + pairs, s);
  return e;
}

}  // namespace

size_t moe_image_bytes(int64_t rows, int64_t k) {
  return static_cast<size_t>(rows) * static_cast<size_t>((k + kImageK - 1) / kImageK) *
         (kImageCodes + kImageScales<1>);  // a group's scales for each row: there are no more groups
}

// Ranges of K of a product of `rows` rows for `pairs` pairs: so many that a call
// with few pairs has an item for every SM or nearly (at least 4 stages each), and no
// more than moe_max_parts(pairs).
int moe_parts(int64_t pairs, int64_t experts, int64_t rows, int64_t k, int num_sms) {
  const int64_t most = experts < pairs ? experts : pairs;
  const int64_t items = most * ((rows + 127) / 128), stages = (k + kImageK - 1) / kImageK;
  int parts = 1;
  while (2 * parts <= moe_max_parts(pairs) && items * parts * 4 <= num_sms * 3 &&
         stages >= 8 * parts)
    parts *= 2;
  return parts;
}

size_t moe_plan_bytes(int64_t pairs) {
  return static_cast<size_t>(Groups::bytes(static_cast<int>(pairs))) + static_cast<size_t>(pairs) * 2;
}

cudaError_t launch_expert_products(const MoeArgs &a, cudaStream_t s) {
  return a.fmt == 0 ? launch_all<0>(a, s) : launch_all<1>(a, s);
}

}  // namespace mx
