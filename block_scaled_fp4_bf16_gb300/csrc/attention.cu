// Attention of a few query tokens of each sequence over a paged cache of E4M3 codes.
//
//   s_t = scale * 2^(ek) q . kcode_t,   out = sum_t softmax(s)_t 2^(ev) vcode_t
//
// The cache's bytes bound it: each is read once for the 8 (query token, head) rows that share
// a key head (16 of 64 channels).  More rows make more tiles, which read the cache again, some six
// tenths of it from memory and the rest from L2 (16 x 2 x 8192 of 64/8 heads: 238 MB from memory for a
// cache of some 145).  Keys, and values transposed, are the 16-row side of FP16 products (16 x 8 x 16,
// binary32 sums) and the rows its 8 columns, so that the conversion of codes, which costs more than the
// products, is done once for all rows of a tile and few rows waste little (the rows on the 16-row side: 165
// us for 64 x up to 8192 tokens of 64/8 heads, where this took 94; now 101 over 568 MB that L2 has nothing
// of, which take 85 at a copy's rate).
// E4M3 is exact in FP16; q enters under a power of two of its row, a weight as the sum of two FP16
// numbers, each a product of its own: as one number its 11 bits showed in the BF16 outputs (0.0005 from
// binary32's, where two leave 0.0002 and less; 64 x up to 8192 of 128 channels 100 us with one, 101 with two, of
// 64 channels 59 and 62, two tiles of those 91 and 98).
//
// Every warp is a worker of its own: the blocks of 32 tokens of all (row tile, sequence,
// key head) together are shared out evenly and in order over the workers, so that uneven
// lengths and few sequences fill the GPU alike.  A worker streams its blocks through its own
// ring of shared memory (cp.async, no barrier wider than the warp) and keeps queries, sums
// and the softmax's state in registers.  A row has two running maxima, as powers of two rounded up:
// `top` of its logits, to which its sum of weights is relative, and `gap` of logit - top + value
// scale, with which the FP16 weights are relative to the largest contribution to the output, however
// far the blocks' scales lie apart.  Both are whole numbers, so that what a new maximum takes off the
// sums is a power of two and exact; the second is one of differences, which binary32 has for logits
// of any size (a maximum of logit + value scale would lose the scale from 2^24 on).
// What a worker leaves unfinished goes to the workspace or, at its end, in its ring; its CTA joins the
// parts of its workers, and a second, small launch those of the CTAs, in their order (all by the second
// launch: 1 x 131072 of 32/4 heads 82 us, so 32, of which the cache takes 20, what precedes the first
// block 4, and the joins 8).
//
// Layouts: the order of channels in a product is free, so lane (g, t) = (lane / 4, lane % 4)
// takes 16 consecutive bytes of keys g and g + 8 as four k-steps, and the queries are laid out
// to match; the order of the output's channels is free as well, so a lane takes 16 consecutive
// channels of its two tokens' values and owns 16 consecutive channels of two rows' output.
// 16-byte pieces of a row are exchanged by the row's number (exclusive or), which leaves every
// load free of conflicts.
#include <cuda_fp16.h>

#include "async_copy.cuh"
#include "kv_cache.cuh"

namespace mx {
namespace {

constexpr int kMaxSms = 160;
constexpr int64_t kMostBlocks = int64_t(1) << 31;  // of all sequences
template <int DIM>
constexpr int kJoinThreads = DIM == 256 ? 256 : 128;
constexpr float kLift = 14.0f;  // FP16 weights are up to 2^14 (in two numbers: to 2^-22, at least to 2^-25)

constexpr int kLeastExponent = -255;  // of a row's factor: under any keys' scale its logits are 0 to binary32

// NT: columns of the products in eights, the rows of a tile.
template <int DIM, int NT>
struct Shape {
  static constexpr int kRows = 8 * NT;
  // (registers: DIM / 4 * NT sums and half as many of queries a lane)
  static constexpr int kWarps = DIM == 64 ? (NT == 1 ? 16 : 12) : DIM == 128 ? 12 : 6;
  static constexpr int kStages = DIM == 64 ? (NT == 1 ? 3 : 4) : 2;
  static constexpr int kBlockBytes = 2 * kCacheBlock * DIM;  // keys, values
  static constexpr int kRing = kBlockBytes * kStages;
  static constexpr int kSteps = DIM / 16;    // k-steps of q . k
  static constexpr int kChunks = DIM / 64;   // 16-byte pieces of a key that a lane reads
  static constexpr int kRun = DIM == 64 ? 8 : 16;  // channels of a value that a lane reads at once
  static constexpr int kRuns = DIM / 8 / kRun;
};

// A (tile, sequence, head) that a CTA begins and others go on with: the last of them (-1: none).
struct Split {
  int last_cta, tile, b, h;
};

// What the two launches share.
struct Plan {
  Split *splits;         // of each CTA
  float *parts;          // one for each worker (part_floats): of what another began and it ended
  float *cta_parts;      // two for each CTA
  int tiles, rows, group;  // rows: of all tiles of a (sequence, key head)
  int part_rows;           // rows of a part
  int workers, ctas;
  int blocks_per_page;
};

// Numbers of a part: sums [rows][dim], then each row's two maxima and its weight.
__host__ __device__ constexpr int64_t part_floats(int64_t rows, int dim) {
  return rows * dim + (3 * rows + 3) / 4 * 4;
}

// Shares of `total` blocks: worker p has [begin(p), begin(p + 1)).
struct Shares {
  int64_t q, r;
  __device__ Shares(int64_t total, int workers) : q(total / workers), r(total % workers) {}
  __device__ int64_t begin(int64_t p) const { return p * q + (p < r ? p : r); }
  __device__ int64_t owner(int64_t f) const {
    return f < r * (q + 1) ? f / (q + 1) : r + (f - r * (q + 1)) / q;
  }
};

// The first token that any query of a sequence of this length sees.
__device__ __forceinline__ int first_seen(const AttentionArgs &a, int length) {
  if (a.window == 0) return 0;
  const int64_t t = length - a.q_tokens - a.window + 1;
  return t > 0 ? static_cast<int>(t) : 0;
}
__device__ __forceinline__ int blocks_of(const AttentionArgs &a, int length) {
  return static_cast<int>((static_cast<int64_t>(length) + kCacheBlock - 1) / kCacheBlock) -
         first_seen(a, length) / kCacheBlock;
}
__device__ __forceinline__ int length_of(const AttentionArgs &a, int b) {
  return static_cast<int>(cache_length(a.c, b));  // (lengths are 32-bit numbers)
}

// Where 16-byte piece `chunk` of row `row` lies in a block's shared memory.
template <int DIM>
__device__ __forceinline__ uint32_t place(int row, int chunk) {
  if constexpr (DIM == 64) {  // two rows to 128 bytes
    const int line = row >> 1;
    return line * 128 + ((((row & 1) * 4 + chunk) ^ ((line * 2) & 7)) * 16);
  } else {
    return row * DIM + ((chunk ^ (row & 7)) * 16);
  }
}

// Four E4M3 codes as two pairs of FP16.
__device__ __forceinline__ void half4_of(uint32_t codes, uint32_t &lo, uint32_t &hi) {
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.rn.f16x2.e4m3x2 %0, l;\n cvt.rn.f16x2.e4m3x2 %1, h;\n}\n"
      : "=r"(lo), "=r"(hi)
      : "r"(codes));
}

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The transpose of an 8 x 8 matrix of FP16, two of a row in a lane.
__device__ __forceinline__ uint32_t transpose8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

__device__ __forceinline__ float exp2_approx(float x) {
  float y;
  asm("ex2.approx.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

__device__ __forceinline__ uint32_t half2_bits(float lo, float hi) {
  uint32_t h;
  asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(hi), "f"(lo));
  return h;
}

__device__ __forceinline__ float2 half2_values(uint32_t h) {
  float2 v;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, h;\n}\n" : "=f"(v.x), "=f"(v.y) : "r"(h));
  return v;
}

__device__ __forceinline__ uint32_t bf16x2_bits(float lo, float hi) {
  uint32_t h;
  asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(h) : "f"(hi), "f"(lo));
  return h;
}

// 0x80 in each byte that is a NaN code.
__device__ __forceinline__ uint32_t nan_codes(uint32_t codes) {
  return ((codes & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
}

// `top` and `gap` of a row without a logit yet: finite, so that -inf less one of them is -inf.
constexpr float kNone = -0x1.fffffep127f;

// Sequence, key head, tile and block of a place in the order of all blocks.
struct Place {
  int b, h, tile;
  int block, blocks;  // of the sequence: from its first seen one
};

__device__ __forceinline__ Place place_of(int64_t f, const uint32_t *first, const CacheArgs &c) {
  Place p;
  const int64_t per_tile = static_cast<int64_t>(first[c.sequences]) * c.heads;
  p.tile = static_cast<int>(f / per_tile);
  f -= p.tile * per_tile;
  int lo = 0, hi = c.sequences;  // the last b with first[b] * heads <= f (it has blocks of its own)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (static_cast<int64_t>(first[mid]) * c.heads <= f)
      lo = mid;
    else
      hi = mid;
  }
  p.b = lo;
  p.blocks = static_cast<int>(first[lo + 1] - first[lo]);
  f -= static_cast<int64_t>(first[lo]) * c.heads;
  p.h = static_cast<int>(f / p.blocks);
  p.block = static_cast<int>(f - static_cast<int64_t>(p.h) * p.blocks);
  return p;
}

// The next place; true if it is in another (tile, sequence, head).
__device__ __forceinline__ bool advance(Place &p, const uint32_t *first, const CacheArgs &c) {
  if (++p.block < p.blocks) return false;
  p.block = 0;
  if (++p.h < c.heads) return true;
  p.h = 0;
  do {
    if (++p.b == c.sequences) p.b = 0, ++p.tile;
    p.blocks = static_cast<int>(first[p.b + 1] - first[p.b]);
  } while (p.blocks == 0);
  return true;
}

// The power of two that brings a row's largest (as binary32 bits) to 2^14 .. 2^15 (a subnormal one
// below that) is 2^-shift.
__device__ __forceinline__ int query_shift(uint32_t largest) {
  const int e = static_cast<int>(largest >> 23);
  return largest == 0 || e == 255 ? 0 : max(e, 1) - 127 - 14;
}

// What turns a row's sums into its output: two factors, which together may leave binary32's
// range where the result does not.
struct Factors {
  float by_weight, by_scale;
};
__device__ __forceinline__ Factors factors_of(float gap, float weight) {
  return Factors{weight == 0.0f ? 0.0f : exp2f(-kLift) / weight, exp2f(gap)};
}

// Writes four channels of a finished row, and its log-sum-exp with the first.
__device__ __forceinline__ void finish(const AttentionArgs &a, const Plan &plan, int b, int h, int row, int d, int dim,
                                       const float (&v)[4], const Factors &f, float top, float weight) {
  const int64_t o_row = static_cast<int64_t>(b) * a.q_tokens + row / plan.group;
  const int64_t head = static_cast<int64_t>(h) * plan.group + row % plan.group;
  const int64_t to = o_row * a.ld_out + head * dim + d;
  const int64_t extent = (static_cast<int64_t>(a.c.sequences) * a.q_tokens - 1) * a.ld_out +
                         static_cast<int64_t>(a.q_heads) * dim;
  if (in_bounds(to, 4, extent, a.c.status))
    *reinterpret_cast<uint2 *>(a.out + to) =
        make_uint2(bf16x2_bits(v[0] * f.by_weight * f.by_scale, v[1] * f.by_weight * f.by_scale),
                   bf16x2_bits(v[2] * f.by_weight * f.by_scale, v[3] * f.by_weight * f.by_scale));
  const int64_t lse_at = o_row * a.q_heads + head;
  if (a.lse != nullptr && d == 0 && in_bounds(lse_at, 1, static_cast<int64_t>(a.c.sequences) * a.q_tokens * a.q_heads, a.c.status))
    a.lse[lse_at] = weight == 0.0f ? -INFINITY : (top + log2f(weight)) * 0.6931471805599453f;
}

// A part: sums [rows][dim]; each row's two maxima and its weight, `rows` apart.
struct Part {
  float *sums, *state;
  int rows;
};
// Part `index` of `count` in the workspace.
__device__ __forceinline__ Part part_at(float *parts, int64_t index, int64_t count, int rows, int dim, uint32_t *status) {
  float *const p = parts + index * part_floats(rows, dim);
  return Part{p, p + static_cast<int64_t>(rows) * dim, in_bounds(index, 1, count, status) ? rows : 0};
}

// The sum of the parts part(0) .. part(n - 1) of a row, four channels from d on.
struct Joined {
  float v[4], top, gap, weight;
};
template <typename PartOf>
__device__ __forceinline__ Joined join(int n, const PartOf &part, int row, int d, int dim, uint32_t *status) {
  Joined j{{0.0f, 0.0f, 0.0f, 0.0f}, kNone, kNone, 0.0f};
#pragma unroll 4
  for (int i = 0; i < n; ++i) {
    const Part p = part(i);
    if (!in_bounds(row, 1, p.rows, status)) continue;
    const float top = p.state[row], gap = p.state[p.rows + row], weight = p.state[2 * p.rows + row];
    const float4 v = *reinterpret_cast<const float4 *>(p.sums + row * dim + d);
    const float now = fmaxf(j.top, top);
    j.weight = j.weight * exp2_approx(j.top - now) + weight * exp2_approx(top - now);
    const float gap_j = j.gap + (j.top - now), gap_p = gap + (top - now), now_gap = fmaxf(fmaxf(gap_j, gap_p), kNone);
    const float keep = exp2_approx(gap_j - now_gap), add = exp2_approx(gap_p - now_gap);
    j.v[0] = j.v[0] * keep + v.x * add;
    j.v[1] = j.v[1] * keep + v.y * add;
    j.v[2] = j.v[2] * keep + v.z * add;
    j.v[3] = j.v[3] * keep + v.w * add;
    j.top = now;
    j.gap = now_gap;
  }
  return j;
}

__device__ __forceinline__ void put_part(const Part &p, int row, int d, int dim, const Joined &j, uint32_t *status) {
  if (!in_bounds(row, 1, p.rows, status)) return;
  *reinterpret_cast<float4 *>(p.sums + row * dim + d) = make_float4(j.v[0], j.v[1], j.v[2], j.v[3]);
  if (d == 0) {
    p.state[row] = j.top;
    p.state[p.rows + row] = j.gap;
    p.state[2 * p.rows + row] = j.weight;
  }
}

// A worker's parts: 0 goes on with a (tile, sequence, head) that another began, 1 begins one.
struct PartInfo {
  int valid, ends;  // ends: the (tile, sequence, head) does
  int tile, b, h, blocks;
  Part part;        // in the worker's shared memory (the last one of its share) or the workspace
};
// Parts of one (tile, sequence, head) by neighbouring workers of a CTA.
struct Chain {
  int warp, count;      // the first worker, the number of workers
  int begins, ends;
  int tile, b, h, blocks;
};

template <int DIM, int NT>
__global__ void __launch_bounds__(Shape<DIM, NT>::kWarps * 32, 1)
    attention_kernel(const __grid_constant__ AttentionArgs a, const __grid_constant__ Plan plan) {
  using S = Shape<DIM, NT>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t warp_sum[S::kWarps];
  __shared__ PartInfo infos[S::kWarps][2];
  __shared__ Chain chains[S::kWarps + 1];
  __shared__ int n_chains;
  __shared__ float states[S::kWarps][3 * S::kRows];
  griddep_launch_dependents();
  griddep_wait();
  const CacheArgs &c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  uint32_t *const first = reinterpret_cast<uint32_t *>(smem + S::kWarps * S::kRing);

  // blocks before each sequence
  {
    int64_t before = 0;
    for (int b0 = 0; b0 < c.sequences; b0 += S::kWarps * 32) {
      const int b = b0 + threadIdx.x;
      const int64_t n = b < c.sequences ? blocks_of(a, length_of(a, b)) : 0;
      int64_t sum = n;
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const int64_t up = __shfl_up_sync(0xFFFFFFFFu, sum, m);
        if (lane >= m) sum += up;
      }
      if (lane == 31) warp_sum[warp] = sum;
      __syncthreads();
      int64_t all = 0;
      for (int w = 0; w < S::kWarps; ++w) {
        if (w < warp) sum += warp_sum[w];
        all += warp_sum[w];
      }
      if (b < c.sequences) first[b] = static_cast<uint32_t>(before + sum - n);
      before += all;
      __syncthreads();
    }
    const bool seen = before <= kMostBlocks;  // (uniform; else nothing is)
    if (threadIdx.x == 0) {
      first[c.sequences] = seen ? static_cast<uint32_t>(before) : 0;
      if (!seen) atomicOr(c.status, kStatusIndexBit);
    }
    if (!seen)  // (each thread's own words of above)
      for (int b = threadIdx.x; b < c.sequences; b += S::kWarps * 32) first[b] = 0;
    if (threadIdx.x < 2 * S::kWarps) infos[threadIdx.x >> 1][threadIdx.x & 1].valid = 0;
    __syncthreads();
  }
  // sequences without blocks: rows of 0
  for (int b = blockIdx.x; b < c.sequences; b += gridDim.x) {
    if (first[b] != first[b + 1]) continue;
    for (int i = threadIdx.x; i < c.heads * plan.rows * (DIM / 4); i += S::kWarps * 32) {
      const float zero[4] = {};
      const int row = i / (DIM / 4) % plan.rows, h = i / (DIM / 4) / plan.rows;
      finish(a, plan, b, h, row, i % (DIM / 4) * 4, DIM, zero, Factors{0.0f, 0.0f}, -INFINITY, 0.0f);
    }
  }
  const int64_t total = static_cast<int64_t>(first[c.sequences]) * c.heads * plan.tiles;
  const Shares shares(total, plan.workers);
  // What turns a sum into a logit is scale * log2(e) times powers of two of the row and the block's keys,
  // of which each may leave binary32's range where the logit does not: the scale is taken apart, and a
  // row's factor is kept as its bits, to which exponents are added.
  int scale_exp;
  const float part = frexpf(a.scale, &scale_exp);
  const uint32_t scale_bits = __float_as_uint((part == 0.0f ? 1.0f : part) * 1.4426950408889634f);
  if (part == 0.0f) scale_exp = kLeastExponent;
  const int worker = blockIdx.x * S::kWarps + warp;
  const int64_t begin = shares.begin(worker), end = shares.begin(worker + 1);

  if (begin < end) {
    const uint32_t ring = smem_u32(smem) + warp * S::kRing;
    const int64_t block_extent = c.pages * c.heads * static_cast<int64_t>(plan.blocks_per_page);

    // ---- copies, kStages - 1 blocks ahead.  next_*: the block to be copied next.
    Place next = place_of(begin, first, c);
    Place at = next;
    int64_t left = end - begin;  // blocks still to be copied
    int next_length = 0, next_start = 0, next_page_index = 0, next_in_page = 0, next_page = 0;
    auto load_page = [&] {
      const int64_t i = static_cast<int64_t>(next.b) * c.max_pages + next_page_index;
      next_page = in_bounds(i, 1, c.sequences * c.max_pages, c.status) ? c.table[i] : -1;
    };
    auto locate = [&] {
      next_length = length_of(a, next.b);
      next_start = first_seen(a, next_length);
      const int block = next_start / kCacheBlock + next.block;
      next_page_index = block / plan.blocks_per_page;
      next_in_page = block - next_page_index * plan.blocks_per_page;
      load_page();
    };
    locate();
    struct Ahead {
      bool held;        // on a page of the pool
      int key_scale, value_scale;
    };
    Ahead ahead[S::kStages];  // of the blocks in the ring
#pragma unroll
    for (int i = 0; i < S::kStages; ++i) ahead[i] = Ahead{false, 0, 0};
    // a lane's pieces of a row pair, quad or so: their places repeat every eight rows
    constexpr int kRowsAtOnce = 512 / DIM, kPieces = DIM / 16, kTurn = 8 / kRowsAtOnce > 0 ? 8 / kRowsAtOnce : 1;
    uint32_t to[kTurn];
#pragma unroll
    for (int i = 0; i < kTurn; ++i)
      to[i] = place<DIM>(i * kRowsAtOnce + lane / kPieces, lane % kPieces) - i * 512;
    auto copy_next = [&](int stage, Ahead &x) {
      if (left > 0) {
        x.held = next_page >= 0 && next_page < c.pages;
        if (!x.held && lane == 0) atomicOr(c.status, kStatusIndexBit);
        const int64_t block = x.held ? (static_cast<int64_t>(next_page) * c.heads + next.h) * plan.blocks_per_page + next_in_page : 0;
        const int t0 = (next_start / kCacheBlock + next.block) * kCacheBlock;
        const uint8_t *const from_k = c.codes[0] + block * (kCacheBlock * DIM) + lane * 16;
        const uint8_t *const from_v = c.codes[1] + block * (kCacheBlock * DIM) + lane * 16;
        const uint32_t dst = ring + stage * S::kBlockBytes;
        if (x.held && t0 >= next_start && t0 + kCacheBlock <= next_length && in_bounds(block, 1, block_extent, c.status)) {
#pragma unroll
          for (int i = 0; i < kCacheBlock * DIM / 512; ++i) {
            cp_async16(dst + to[i % kTurn] + i * 512, from_k + i * 512);
            cp_async16(dst + kCacheBlock * DIM + to[i % kTurn] + i * 512, from_v + i * 512);
          }
        } else {
          // rows that no query sees come as zeros: whatever lies there, NaN among it, stays out
#pragma unroll
          for (int i = 0; i < kCacheBlock * DIM / 512; ++i) {
            const int token = t0 + i * kRowsAtOnce + lane / kPieces;
            const bool in = x.held && token < next_length && token >= next_start && in_bounds(block, 1, block_extent, c.status);
            cp_async16(dst + to[i % kTurn] + i * 512, from_k + i * 512, in);
            cp_async16(dst + kCacheBlock * DIM + to[i % kTurn] + i * 512, from_v + i * 512, in);
          }
        }
        if (in_bounds(block, 1, block_extent, c.status)) {
          x.key_scale = c.scales[0][block];
          x.value_scale = c.scales[1][block];
        }
        if (--left > 0) {
          if (!advance(next, first, c)) {
            if (++next_in_page == plan.blocks_per_page) {
              next_in_page = 0;
              ++next_page_index;
              load_page();
            }
          } else {
            locate();
          }
        }
      }
      cp_async_commit();
    };
#pragma unroll
    for (int i = 0; i < S::kStages - 1; ++i) copy_next(i, ahead[i]);

    // ---- the blocks, one after the other
    float out[NT][DIM / 16][4];  // [..][..][2 e + r]: channels 2 i + e of the lane's, rows 2 t + r
    float top[NT][2], gap[NT][2], weight[NT][2];
    uint32_t factor[NT][2];      // of the rows' logits, as bits: scale, log2(e) and the row's power of two
    int exponent_low = 0, exponent_high = 0;  // of all rows' powers of two
    uint32_t query[NT][S::kSteps][2];
    int length = 0, start = 0;
    bool from_start = false, fresh = true;
    int stage = 0;
    for (int64_t f = begin; f < end; ++f) {
      if (fresh) {  // a new (tile, sequence, head): its queries
        fresh = false;
        exponent_low = exponent_high = 0;
        from_start = at.block == 0;
        length = length_of(a, at.b);
        start = first_seen(a, length);
#pragma unroll
        for (int nt = 0; nt < NT; ++nt) {
          const int row = at.tile * S::kRows + nt * 8 + g;
          const int64_t q_row = static_cast<int64_t>(at.b) * a.q_tokens + row / plan.group;
          const int64_t q_at = q_row * a.ld_q + (static_cast<int64_t>(at.h) * plan.group + row % plan.group) * DIM;
          const int64_t extent = (static_cast<int64_t>(c.sequences) * a.q_tokens - 1) * a.ld_q +
                                 static_cast<int64_t>(a.q_heads) * DIM;
          uint4 raw[S::kChunks][2];
          uint32_t largest = 0;
#pragma unroll
          for (int i = 0; i < S::kChunks; ++i) {
            const int chunk = DIM == 64 ? t : 8 * (i >> 1) + 2 * t + (i & 1);
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const int64_t e = q_at + chunk * 16 + k * 8;
              raw[i][k] = row < plan.rows && in_bounds(e, 8, extent, c.status)
                              ? *reinterpret_cast<const uint4 *>(a.q + e)
                              : make_uint4(0, 0, 0, 0);
              const uint32_t w[4] = {raw[i][k].x, raw[i][k].y, raw[i][k].z, raw[i][k].w};
#pragma unroll
              for (int u = 0; u < 4; ++u) largest = max(largest, max((w[u] & 0x7FFFu) << 16, w[u] & 0x7FFF0000u));
            }
          }
          largest = max(largest, __shfl_xor_sync(0xFFFFFFFFu, largest, 1));
          largest = max(largest, __shfl_xor_sync(0xFFFFFFFFu, largest, 2));
          const int shift = query_shift(largest);
          const float f1 = exp2_int(-shift / 2), f2 = exp2_int(-shift - -shift / 2);
          const int exponent = max(scale_exp + shift, kLeastExponent);
          exponent_low = min(exponent_low, __reduce_min_sync(0xFFFFFFFFu, exponent));
          exponent_high = max(exponent_high, __reduce_max_sync(0xFFFFFFFFu, exponent));
          const uint32_t mine = scale_bits + (static_cast<uint32_t>(exponent) << 23);
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            factor[nt][r] = __shfl_sync(0xFFFFFFFFu, mine, (2 * t + r) * 4);
            top[nt][r] = gap[nt][r] = kNone;
            weight[nt][r] = 0.0f;
          }
#pragma unroll
          for (int i = 0; i < S::kChunks; ++i)
#pragma unroll
            for (int u = 0; u < 4; ++u) {
              const uint4 &v = raw[i][u >> 1];
              const uint32_t w0 = (u & 1) ? v.z : v.x, w1 = (u & 1) ? v.w : v.y;
              const uint32_t h0 = half2_bits(__uint_as_float(w0 << 16) * f1 * f2, __uint_as_float(w0 & 0xFFFF0000u) * f1 * f2);
              const uint32_t h1 = half2_bits(__uint_as_float(w1 << 16) * f1 * f2, __uint_as_float(w1 & 0xFFFF0000u) * f1 * f2);
              query[nt][i * 4 + u][0] = h0;
              query[nt][i * 4 + u][1] = h1;
            }
#pragma unroll
          for (int i = 0; i < DIM / 16; ++i)
#pragma unroll
            for (int k = 0; k < 4; ++k) out[nt][i][k] = 0.0f;
        }
      }

      cp_async_wait<S::kStages - 2>();
      __syncwarp();  // the lanes' copies are there for all, and the stage before this one is read
      const Ahead here = ahead[0];
#pragma unroll
      for (int i = 0; i + 1 < S::kStages; ++i) ahead[i] = ahead[i + 1];
      copy_next(stage == 0 ? S::kStages - 1 : stage - 1, ahead[S::kStages - 2]);
      const uint32_t keys = ring + stage * S::kBlockBytes, values = keys + kCacheBlock * DIM;

      // logits: s[nt][j][2 e + r] of token 16 j + 8 e + g and row 2 t + r of eight
      float s[NT][2][4] = {};
#pragma unroll
      for (int i = 0; i < S::kChunks; ++i) {
        const int chunk = DIM == 64 ? t : 8 * (i >> 1) + 2 * t + (i & 1);
        uint4 k[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) k[j] = lds128(keys + place<DIM>(8 * j + g, chunk));
#pragma unroll
        for (int u = 0; u < 4; ++u) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint4 &k0 = k[2 * j], &k1 = k[2 * j + 1];
            uint32_t a0, a1, a2, a3;
            half4_of(u == 0 ? k0.x : u == 1 ? k0.y : u == 2 ? k0.z : k0.w, a0, a2);
            half4_of(u == 0 ? k1.x : u == 1 ? k1.y : u == 2 ? k1.z : k1.w, a1, a3);
#pragma unroll
            for (int nt = 0; nt < NT; ++nt) mma_f16(s[nt][j], a0, a1, a2, a3, query[nt][i * 4 + u][0], query[nt][i * 4 + u][1]);
          }
        }
      }

      const int t0 = (start / kCacheBlock + at.block) * kCacheBlock;
      const int position = length - a.q_tokens;  // of the first query
      // do all rows see all of the block?
      const bool whole = here.held && t0 + kCacheBlock - 1 <= position &&
                         (a.window == 0 || static_cast<int64_t>(t0) >= length - a.window);
      const int key_exp = here.key_scale - 127;
      const float value_exp = static_cast<float>(here.value_scale - 127);
      float most[NT][2];
      if (key_exp + exponent_low >= -125 && key_exp + exponent_high <= 126) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float f = __uint_as_float(factor[nt][r] + (static_cast<uint32_t>(key_exp) << 23));
#pragma unroll
            for (int i = 0; i < 4; ++i) s[nt][i >> 1][2 * (i & 1) + r] *= f;
          }
      } else {  // in two steps of finite factors (0 stays 0)
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int e = (static_cast<int>(factor[nt][r] - scale_bits) >> 23) + key_exp;
            const float f1 = exp2_int(min(max(e / 2, -126), 126)), f2 = exp2_int(min(max(e - e / 2, -126), 126));
#pragma unroll
            for (int i = 0; i < 4; ++i) s[nt][i >> 1][2 * (i & 1) + r] *= __uint_as_float(scale_bits) * f1;
#pragma unroll
            for (int i = 0; i < 4; ++i) s[nt][i >> 1][2 * (i & 1) + r] *= f2;
          }
      }
      if (!whole) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const int p = position + (at.tile * S::kRows + nt * 8 + 2 * t + r) / plan.group;
            const int64_t low = a.window == 0 ? 0 : p - a.window + 1;
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int token = t0 + 8 * i + g;
              if (!(here.held && token <= p && token < length && token >= low))
                s[nt][i >> 1][2 * (i & 1) + r] = -INFINITY;
            }
          }
      }
      bool grows = false;
#pragma unroll
      for (int nt = 0; nt < NT; ++nt)
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          float m = fmaxf(fmaxf(s[nt][0][r], s[nt][0][2 + r]), fmaxf(s[nt][1][r], s[nt][1][2 + r]));
          m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 4));
          m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 8));
          m = fmaxf(m, __shfl_xor_sync(0xFFFFFFFFu, m, 16));
          most[nt][r] = m;
          grows |= m > top[nt][r] || m - top[nt][r] > gap[nt][r] - value_exp;
        }
      if (__any_sync(0xFFFFFFFFu, grows)) {
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            const float now = fmaxf(top[nt][r], ceilf(most[nt][r])), down = top[nt][r] - now;
            const float kept = gap[nt][r] + down;
            const float now_gap = fmaxf(fmaxf(kept, ceilf(most[nt][r] - now) + value_exp), kNone);
            weight[nt][r] *= exp2_approx(down);
            const float keep = exp2_approx(kept - now_gap);
            top[nt][r] = now;
            gap[nt][r] = now_gap;
#pragma unroll
            for (int i = 0; i < DIM / 16; ++i) {
              out[nt][i][r] *= keep;
              out[nt][i][2 + r] *= keep;
            }
          }
      }
      // weights: in binary32 for their sum, as two FP16 numbers relative to the largest contribution
      uint32_t p[NT][4], p_low[NT][4];
#pragma unroll
      for (int nt = 0; nt < NT; ++nt) {
        float w[2][4];
#pragma unroll
        for (int r = 0; r < 2; ++r) {
          const float lift = value_exp + kLift - gap[nt][r];
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float l = s[nt][i >> 1][2 * (i & 1) + r] - top[nt][r];
            weight[nt][r] += exp2_approx(l);
            w[r][i] = exp2_approx(l + lift);
          }
        }
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t high = half2_bits(w[0][i], w[1][i]);
          const float2 back = half2_values(high);
          p[nt][i] = transpose8(high);
          p_low[nt][i] = transpose8(half2_bits(w[0][i] - back.x, w[1][i] - back.y));
        }
      }

#pragma unroll
      for (int run = 0; run < S::kRuns; ++run) {
        // the lane's tokens 16 j + 2 t, + 1 and + 8, + 9
        constexpr int kWords = S::kRun / 4;
        uint32_t v[2][4][kWords];
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k) {
            const int row = 16 * j + 2 * t + (k & 1) + 8 * (k >> 1);
            if constexpr (DIM == 64) {
              const uint2 x = lds64(values + place<DIM>(row, g >> 1) + (g & 1) * 8);
              v[j][k][0] = x.x, v[j][k][1] = x.y;
            } else {
              const uint4 x = lds128(values + place<DIM>(row, 8 * run + g));
              v[j][k][0] = x.x, v[j][k][1] = x.y, v[j][k][2] = x.z, v[j][k][3] = x.w;
            }
          }
        if (!whole) {
          // A NaN is for the rows that see it only: they get it by themselves, the product a
          // zero (0 * NaN would bring it to all).
          uint32_t nan = 0;
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int w = 0; w < kWords; ++w) nan |= nan_codes(v[j][k][w]);
          if (__any_sync(0xFFFFFFFFu, nan != 0)) {
            for (int row = 0; row < kCacheBlock; ++row) {
              const int token = t0 + row;
#pragma unroll
              for (int e = 0; e < S::kRun; ++e) {  // the lane's channels of the output
                const int col = g * S::kRun + e;
                uint32_t code;
                const uint32_t addr = values + place<DIM>(row, 8 * run + col / 16) + col % 16;
                asm volatile("ld.shared.u8 %0, [%1];" : "=r"(code) : "r"(addr));
                if ((code & 0x7Fu) != 0x7Fu) continue;
#pragma unroll
                for (int nt = 0; nt < NT; ++nt)
#pragma unroll
                  for (int r = 0; r < 2; ++r) {
                    const int q = position + (at.tile * S::kRows + nt * 8 + 2 * t + r) / plan.group;
                    const int64_t low = a.window == 0 ? 0 : q - a.window + 1;
                    if (here.held && token <= q && token < length && token >= low)
                      out[nt][(run * S::kRun + e) / 2][2 * (e & 1) + r] = NAN;
                  }
              }
            }
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int k = 0; k < 4; ++k)
#pragma unroll
                for (int w = 0; w < kWords; ++w) v[j][k][w] &= ~((nan_codes(v[j][k][w]) >> 7) * 0xFFu);
          }
        }
#pragma unroll
        for (int w = 0; w < kWords; ++w) {
          // the same channel of two neighbouring tokens, for four channels
          uint32_t b[4][2][2];  // [channel][j][tokens 2 t, + 1 / + 8, + 9]
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const uint32_t lo = __byte_perm(v[j][2 * k][w], v[j][2 * k + 1][w], 0x5140);
              const uint32_t hi = __byte_perm(v[j][2 * k][w], v[j][2 * k + 1][w], 0x7362);
              half4_of(lo, b[0][j][k], b[1][j][k]);
              half4_of(hi, b[2][j][k], b[3][j][k]);
            }
#pragma unroll
          for (int e = 0; e < 4; e += 2)
#pragma unroll
            for (int j = 0; j < 2; ++j)
#pragma unroll
              for (int nt = 0; nt < NT; ++nt) {
                float(&sums)[4] = out[nt][(run * S::kRun + 4 * w + e) / 2];
                mma_f16(sums, b[e][j][0], b[e + 1][j][0], b[e][j][1], b[e + 1][j][1], p[nt][2 * j], p[nt][2 * j + 1]);
                mma_f16(sums, b[e][j][0], b[e + 1][j][0], b[e][j][1], b[e + 1][j][1], p_low[nt][2 * j], p_low[nt][2 * j + 1]);
              }
        }
      }
      stage = stage + 1 == S::kStages ? 0 : stage + 1;

      // ---- the end of a (tile, sequence, head), or of the worker's share
      const bool last = at.block + 1 == at.blocks;
      if (last || f + 1 == end) {
        fresh = true;
        const bool whole_row = from_start && last;
        // (the last part of a share takes the place of the ring; an earlier one, which goes to memory, ends
        // what another worker began)
        const bool in_ring = f + 1 == end;
        Part part = part_at(plan.parts, worker, plan.workers, plan.part_rows, DIM, c.status);
        if (in_ring) {
          part = Part{reinterpret_cast<float *>(smem + warp * S::kRing), states[warp], S::kRows};
          cp_async_wait<0>();
          __syncwarp();
        }
        if (!whole_row && lane == 0)
          infos[warp][from_start] = PartInfo{1, last, at.tile, at.b, at.h, at.blocks, part};
#pragma unroll
        for (int nt = 0; nt < NT; ++nt)
#pragma unroll
          for (int r = 0; r < 2; ++r) {
            Joined j;
            j.weight = weight[nt][r];
            j.weight += __shfl_xor_sync(0xFFFFFFFFu, j.weight, 4);
            j.weight += __shfl_xor_sync(0xFFFFFFFFu, j.weight, 8);
            j.weight += __shfl_xor_sync(0xFFFFFFFFu, j.weight, 16);
            j.top = top[nt][r];
            j.gap = gap[nt][r];
            const int pr = nt * 8 + 2 * t + r, row = at.tile * S::kRows + pr;
            if (row >= plan.rows) continue;
            const Factors factors = factors_of(j.gap, j.weight);
#pragma unroll
            for (int run = 0; run < S::kRuns; ++run)
#pragma unroll
              for (int e = 0; e < S::kRun; e += 4) {
#pragma unroll
                for (int k = 0; k < 4; ++k) j.v[k] = out[nt][(run * S::kRun + e + k) / 2][2 * (k & 1) + r];
                const int d = run * 128 + g * S::kRun + e;
                if (whole_row)
                  finish(a, plan, at.b, at.h, row, d, DIM, j.v, factors, j.top, j.weight);
                else
                  put_part(part, pr, d, DIM, j, c.status);
              }
          }
      }
      if (f + 1 < end) advance(at, first, c);
    }
  }

  // ---- the workers' parts: chains of one (tile, sequence, head) by neighbouring workers
  __syncthreads();
  static_assert(S::kRing >= S::kRows * DIM * 4, "a part in the ring's place");
  if (warp == 0) {
    // lane w: the chain that worker w begins; a chain that goes on from the CTA before is w = 0's too
    const bool in = lane < S::kWarps;
    const PartInfo head = in ? infos[lane][0] : PartInfo{}, tail = in ? infos[lane][1] : PartInfo{};
    const uint32_t heads = __ballot_sync(0xFFFFFFFFu, in && head.valid), tails = __ballot_sync(0xFFFFFFFFu, in && tail.valid);
    const int goes_on = heads & 1u;
    // workers after w that go on with its chain: up to the first that begins one itself
    const auto after = [&](int w) {
      const int run = __ffs(static_cast<int>(~(heads >> (w + 1)))) - 1, tail_at = __ffs(static_cast<int>(tails >> (w + 1)));
      return tail_at > 0 && tail_at < run ? tail_at : run;
    };
    if (in && tail.valid) {
      const int n = after(lane);
      chains[goes_on + __popc(tails & ((1u << lane) - 1))] =
          Chain{lane, 1 + n, 1, n > 0 ? infos[lane + n][0].ends : 0, tail.tile, tail.b, tail.h, tail.blocks};
    }
    if (lane == 0 && goes_on) {
      // (if worker 0 has a tail, too, the next workers go on with that one)
      const int n = tail.valid ? 0 : after(0);
      chains[0] = Chain{0, 1 + n, 0, infos[n][0].ends, head.tile, head.b, head.h, head.blocks};
    }
    if (lane == 0) n_chains = goes_on + __popc(tails);
  }
  __syncthreads();
  if (threadIdx.x == S::kWarps * 32 - 1) {
    Split split{-1, 0, 0, 0};
    if (n_chains > 0 && chains[n_chains - 1].begins && !chains[n_chains - 1].ends) {
      const Chain &chain = chains[n_chains - 1];
      const int64_t f0 = chain.tile * (total / plan.tiles) + static_cast<int64_t>(first[chain.b]) * c.heads + static_cast<int64_t>(chain.h) * chain.blocks;
      split = Split{static_cast<int>(shares.owner(f0 + chain.blocks - 1) / S::kWarps), chain.tile, chain.b, chain.h};
    }
    if (in_bounds(blockIdx.x, 1, plan.ctas, c.status)) plan.splits[blockIdx.x] = split;
  }
  const int per_chain = plan.part_rows * (DIM / 4);
  for (int i = threadIdx.x; i < n_chains * per_chain; i += S::kWarps * 32) {
    const Chain &chain = chains[i / per_chain];
    const int pr = i % per_chain / (DIM / 4), d = i % (DIM / 4) * 4, row = chain.tile * S::kRows + pr;
    if (row >= plan.rows) continue;
    const auto part = [&](int k) { return infos[chain.warp + k][k == 0 && chain.begins].part; };
    const Joined j = join(chain.count, part, pr, d, DIM, c.status);
    if (chain.begins && chain.ends)
      finish(a, plan, chain.b, chain.h, row, d, DIM, j.v, factors_of(j.gap, j.weight), j.top, j.weight);
    else
      put_part(part_at(plan.cta_parts, static_cast<int64_t>(blockIdx.x) * 2 + chain.begins, 2 * plan.ctas, plan.part_rows, DIM, c.status),
               pr, d, DIM, j, c.status);
  }
}

// Joins the CTAs' parts of a row: CTA (x, y) row y of what CTA x of the launch before began and
// left unfinished.  Groups of a row's DIM / 4 threads take every so many-th part's sums; where
// that is more than one, each warp takes the parts' states first, so that all loads of a thread go out
// together (1 x 131072 of 32/4 heads 32.2 us with a state before each part's sums, so 31.1 then).
template <int DIM>
__global__ void __launch_bounds__(kJoinThreads<DIM>)
    join_kernel(const __grid_constant__ AttentionArgs a, const __grid_constant__ Plan plan, int tile_rows) {
  constexpr int kThreads = kJoinThreads<DIM>, kLanes = DIM / 4, kGroups = kThreads / kLanes, kAhead = 6;
  constexpr int kOwn = (kMaxSms + 31) / 32;  // states of a lane: each warp takes all of them for itself
  __shared__ __align__(16) float sums[kGroups][DIM];
  __shared__ float states[kGroups][3], factors[kThreads / 32][kOwn * 32];
  griddep_launch_dependents();
  griddep_wait();
  const int p0 = blockIdx.x, pr = blockIdx.y, warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const Split split = in_bounds(p0, 1, plan.ctas, a.c.status) ? plan.splits[p0] : Split{-1, 0, 0, 0};
  if (split.last_cta < 0) return;
  const int row = split.tile * tile_rows + pr;
  if (row >= plan.rows) return;
  const int group = threadIdx.x / kLanes, d = threadIdx.x % kLanes * 4;
  const int n = split.last_cta - p0 + 1;  // (at most as many as CTAs)
  // (the first CTA's part begins the row, the others' go on with it)
  const auto part = [&](int k) {
    return part_at(plan.cta_parts, static_cast<int64_t>(p0 + k) * 2 + (k == 0), 2 * plan.ctas, plan.part_rows, DIM, a.c.status);
  };
  if (n <= kGroups) {
    const Joined own = join(group < n, [&](int) { return part(group); }, pr, d, DIM, a.c.status);
    put_part(Part{sums[group], states[group], 1}, 0, d, DIM, own, a.c.status);
    __syncthreads();
    if (group != 0) return;
    const Joined j = join(n, [&](int k) { return Part{sums[k], states[k], 1}; }, 0, d, DIM, a.c.status);
    finish(a, plan, split.b, split.h, row, d, DIM, j.v, factors_of(j.gap, j.weight), j.top, j.weight);
    return;
  }
  const auto load = [&](int k) {
    if (k >= n) return make_float4(0.0f, 0.0f, 0.0f, 0.0f);
    const Part p = part(k);
    return in_bounds(pr, 1, p.rows, a.c.status) ? *reinterpret_cast<const float4 *>(p.sums + pr * DIM + d)
                                                : make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  };
  float4 x[kAhead];
#pragma unroll
  for (int i = 0; i < kAhead; ++i) x[i] = load(group + i * kGroups);
  float top[kOwn], gap[kOwn], weight[kOwn], all_top = kNone, all_gap = kNone, all_weight = 0.0f;
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    const int k = lane + i * 32;
    top[i] = gap[i] = kNone;
    weight[i] = 0.0f;
    if (k < n) {
      const Part p = part(k);
      if (!in_bounds(pr, 1, p.rows, a.c.status)) continue;
      top[i] = p.state[pr], gap[i] = p.state[p.rows + pr], weight[i] = p.state[2 * p.rows + pr];
    }
    all_top = fmaxf(all_top, top[i]);
  }
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) all_top = fmaxf(all_top, __shfl_xor_sync(0xFFFFFFFFu, all_top, m));
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    const float down = top[i] - all_top;
    gap[i] += down;
    all_gap = fmaxf(all_gap, gap[i]);
    all_weight += weight[i] * exp2_approx(down);
  }
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) all_gap = fmaxf(all_gap, __shfl_xor_sync(0xFFFFFFFFu, all_gap, m));
#pragma unroll
  for (int i = 0; i < kOwn; ++i) {
    if (i * 32 >= n) break;
    factors[warp][lane + i * 32] = exp2_approx(gap[i] - all_gap);
  }
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) all_weight += __shfl_xor_sync(0xFFFFFFFFu, all_weight, m);
  __syncwarp();
  float v[4] = {};
  const auto add = [&](int k, const float4 &y) {
    const float f = k < n ? factors[warp][k] : 0.0f;
    v[0] += y.x * f, v[1] += y.y * f, v[2] += y.z * f, v[3] += y.w * f;
  };
#pragma unroll
  for (int i = 0; i < kAhead; ++i) add(group + i * kGroups, x[i]);
  for (int k0 = group + kAhead * kGroups; k0 < n; k0 += kAhead * kGroups) {
#pragma unroll
    for (int i = 0; i < kAhead; ++i) x[i] = load(k0 + i * kGroups);
#pragma unroll
    for (int i = 0; i < kAhead; ++i) add(k0 + i * kGroups, x[i]);
  }
  *reinterpret_cast<float4 *>(&sums[group][d]) = make_float4(v[0], v[1], v[2], v[3]);
  __syncthreads();
  if (group != 0) return;
#pragma unroll
  for (int g = 1; g < kGroups; ++g) {
    const float4 y = *reinterpret_cast<const float4 *>(&sums[g][d]);
    v[0] += y.x, v[1] += y.y, v[2] += y.z, v[3] += y.w;
  }
  finish(a, plan, split.b, split.h, row, d, DIM, v, factors_of(all_gap, all_weight), all_top, all_weight);
}

constexpr size_t kSplitBytes = kMaxSms * sizeof(Split);
static_assert(kSplitBytes % 16 == 0, "alignment of the parts");

// The rows of a tile: 8, or 16 of 64 channels where there are more than 8.  A second tile reads
// the cache again, mostly from memory, but 16 rows take registers from as many warps (16 x 2 x 8192
// of 64/8 heads, in tiles of 8 / of 16 rows: 128 channels 52 / 65 us; 64 x 2 of 64 channels 109 / 98;
// 256 channels, before weights had two parts, 110 / 116).
int tile_rows_of(int64_t rows, int dim) { return rows <= 8 || dim > 64 ? 8 : 16; }
int64_t part_rows_of(int64_t rows, int dim) { return rows < tile_rows_of(rows, dim) ? rows : tile_rows_of(rows, dim); }

template <int DIM, int NT>
cudaError_t launch(const AttentionArgs &a, cudaStream_t s) {
  using S = Shape<DIM, NT>;
  Plan plan;
  plan.group = a.q_heads / a.c.heads;
  plan.rows = plan.group * a.q_tokens;
  plan.tiles = (plan.rows + S::kRows - 1) / S::kRows;
  plan.part_rows = static_cast<int>(part_rows_of(plan.rows, DIM));
  plan.blocks_per_page = a.c.page_tokens / kCacheBlock;
  const int ctas = a.num_sms < kMaxSms ? a.num_sms : kMaxSms;
  plan.workers = ctas * S::kWarps;
  plan.ctas = ctas;
  plan.splits = static_cast<Split *>(a.workspace);
  plan.cta_parts = reinterpret_cast<float *>(static_cast<uint8_t *>(a.workspace) + kSplitBytes);
  plan.parts = plan.cta_parts + 2 * ctas * part_floats(plan.part_rows, DIM);
  constexpr size_t kFixed = static_cast<size_t>(S::kWarps) * S::kRing;
  const size_t smem = kFixed + (static_cast<size_t>(a.c.sequences) + 1) * sizeof(uint32_t);
  const void *func = reinterpret_cast<const void *>(attention_kernel<DIM, NT>);
  if (!kernel_setup_get(func, nullptr)) {
    constexpr size_t kMost = kFixed + (kAttentionMaxSequences + 1) * sizeof(uint32_t);
    static_assert(kMost + 8192 <= 227 * 1024, "shared memory");
    const cudaError_t e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(kMost));
    if (e != cudaSuccess) return e;
    kernel_setup_put(func, 0);
  }
  const cudaError_t e = launch_pdl(attention_kernel<DIM, NT>, dim3(static_cast<unsigned>(ctas)), dim3(S::kWarps * 32),
                                   smem, s, a, plan);
  if (e != cudaSuccess) return e;
  return launch_pdl(join_kernel<DIM>, dim3(static_cast<unsigned>(ctas), plan.part_rows), dim3(kJoinThreads<DIM>), 0, s, a,
                    plan, S::kRows);
}

}  // namespace

size_t attention_workspace_bytes(int64_t rows, int head_dim) {
  const int warps = head_dim == 64    ? (tile_rows_of(rows, 64) == 8 ? Shape<64, 1>::kWarps : Shape<64, 2>::kWarps)
                    : head_dim == 128 ? Shape<128, 1>::kWarps
                                      : Shape<256, 1>::kWarps;
  const int64_t parts = kMaxSms * (2 + warps);  // of the CTAs and of their warps
  return kSplitBytes + static_cast<size_t>(parts * part_floats(part_rows_of(rows, head_dim), head_dim)) * sizeof(float);
}

cudaError_t launch_attention(const AttentionArgs &a, cudaStream_t s) {
  switch (a.c.head_dim) {
    case 64: {
      const int64_t rows = static_cast<int64_t>(a.q_heads / a.c.heads) * a.q_tokens;
      return tile_rows_of(rows, 64) == 8 ? launch<64, 1>(a, s) : launch<64, 2>(a, s);
    }
    case 128: return launch<128, 1>(a, s);
    default: return launch<256, 1>(a, s);
  }
}

}  // namespace mx
