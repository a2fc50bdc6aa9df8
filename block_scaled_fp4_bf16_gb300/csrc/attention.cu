// Attention of a few query tokens of each sequence over a paged cache of E4M3 codes.
//
//   s_t = scale * 2^(ek) q . kcode_t,   out = sum_t softmax(s)_t 2^(ev) vcode_t
//
// The cache's bytes bound it: each is read once for the up to 16 (query token, head) rows
// that share a key head, as the 16-row side of FP16 products (16 x 8 x 16, binary32 sums).
// E4M3 is exact in FP16; q enters under a power of two of its row.
//
// Every warp is a worker of its own: the blocks of 32 tokens of all (row tile, sequence,
// key head) together are shared out evenly and in order over the workers, so that uneven
// lengths and few sequences fill the GPU alike.  A worker streams its blocks through its own
// ring of shared memory (cp.async, no barrier wider than the warp) and keeps queries, sums
// and the softmax's running maximum in registers.  Weights of a block are taken relative to
// the block's own maximum and its sum joins the running one with one binary32 factor, which
// also carries the block's scale: no ratio between blocks' scales or weights is ever rounded
// to FP16.  What a worker leaves unfinished goes to the workspace; a second, small launch
// joins such parts in their order.
//
// Layouts: the order of channels in a product is free, so lane (g, c) = (lane / 4, lane % 4)
// takes 16 consecutive bytes of key g as four k-steps, and the queries are laid out to match;
// the order of columns is free as well, so a lane takes 16 consecutive channels of its two
// tokens' values and owns 32 consecutive channels of the output.  16-byte pieces of a row are
// exchanged by the row's number (exclusive or), which leaves every load free of conflicts.
#include <cuda_fp16.h>

#include "kv_cache.cuh"

namespace mx {
namespace {

constexpr int kTile = 16;  // rows of a product
constexpr int kMaxSms = 160;
constexpr int kJoinThreads = 128;

template <int DIM>
struct Shape {
  static constexpr int kWarps = DIM == 64 ? 16 : DIM == 128 ? 8 : 4;
  static constexpr int kStages = DIM == 256 ? 2 : 3;
  static constexpr int kRing = 2 * kCacheBlock * DIM * kStages;  // bytes of a warp: keys, values
  static constexpr int kSteps = DIM / 16;                        // k-steps of q . k
  static constexpr int kChunks = DIM / 64;                       // 16-byte pieces of a key a lane reads
  static constexpr int kRun = DIM == 64 ? 8 : 16;                // channels of a value a lane reads at once
  static constexpr int kRuns = DIM / 8 / kRun;
  static constexpr bool kQueriesInShared = DIM == 256;           // (registers: the sums take 128)
  static constexpr int kQueryBytes = kQueriesInShared ? kSteps * 512 : 0;
};

// What the two launches share: `first` holds the blocks before each sequence (one tile, one head).
struct Plan {
  int64_t *first;  // [sequences + 1]
  float *parts;    // two for each worker: sums [rows][DIM], maximum [rows], weight [rows]
  int tiles, rows, group;  // rows: of all tiles of a (sequence, key head)
  int part_rows;           // rows of a part
  int workers;
};

// Numbers of a part: 16-byte stores need its length in fours.
__host__ __device__ constexpr int64_t part_floats(int64_t rows, int dim) {
  return rows * dim + (2 * rows + 3) / 4 * 4;
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
__device__ __forceinline__ int64_t first_seen(const AttentionArgs &a, int64_t length) {
  if (a.window == 0) return 0;
  const int64_t t = length - a.q_tokens - a.window + 1;
  return t > 0 ? t : 0;
}
__device__ __forceinline__ int64_t blocks_of(const AttentionArgs &a, int64_t length) {
  return (length + kCacheBlock - 1) / kCacheBlock - first_seen(a, length) / kCacheBlock;
}

__device__ __forceinline__ void cp_async16(uint32_t dst, const void *src, bool in) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(in ? 16 : 0) : "memory");
}
__device__ __forceinline__ void cp_async_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void cp_async_wait() {
  asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

__device__ __forceinline__ uint4 lds128(uint32_t addr) {
  uint4 v;
  asm volatile("ld.shared.v4.u32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(addr));
  return v;
}
__device__ __forceinline__ uint2 lds64(uint32_t addr) {
  uint2 v;
  asm volatile("ld.shared.v2.u32 {%0, %1}, [%2];" : "=r"(v.x), "=r"(v.y) : "r"(addr));
  return v;
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

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
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

// Any NaN code among the four bytes?
__device__ __forceinline__ bool any_nan(uint32_t codes) {
  return (((codes & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u) != 0;
}

// Sequence, key head, tile and block of a place in the order of all blocks.
struct Place {
  int b, h, tile;
  int64_t block, blocks;  // of the sequence: from its first seen one
};

__device__ __forceinline__ Place place_of(int64_t f, const int64_t *first, const CacheArgs &c) {
  Place p;
  const int64_t per_tile = first[c.sequences] * c.heads;
  p.tile = static_cast<int>(f / per_tile);
  f %= per_tile;
  int lo = 0, hi = c.sequences;  // the last b with first[b] * heads <= f (and blocks of its own)
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] * c.heads <= f)
      lo = mid;
    else
      hi = mid;
  }
  p.b = lo;
  p.blocks = first[lo + 1] - first[lo];
  f -= first[lo] * c.heads;
  p.h = static_cast<int>(f / p.blocks);
  p.block = f % p.blocks;
  return p;
}

__device__ __forceinline__ void advance(Place &p, const int64_t *first, const CacheArgs &c) {
  if (++p.block < p.blocks) return;
  p.block = 0;
  if (++p.h < c.heads) return;
  p.h = 0;
  do {
    if (++p.b == c.sequences) p.b = 0, ++p.tile;
    p.blocks = first[p.b + 1] - first[p.b];
  } while (p.blocks == 0);
}

// One row's queries: a power of two 2^-shift brings its largest to 2^14 .. 2^15.
__device__ __forceinline__ int query_shift(uint32_t largest) {
  const int e = static_cast<int>(largest >> 23);
  return e == 0 || e == 255 ? 0 : e - 127 - 14;
}

template <int DIM>
__global__ void __launch_bounds__(Shape<DIM>::kWarps * 32, 1)
    attention_kernel(const __grid_constant__ AttentionArgs a, const __grid_constant__ Plan plan) {
  using S = Shape<DIM>;
  extern __shared__ __align__(128) uint8_t smem[];
  __shared__ int64_t warp_sum[S::kWarps];
  griddep_launch_dependents();
  griddep_wait();
  const CacheArgs &c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  int64_t *const first = reinterpret_cast<int64_t *>(smem + S::kWarps * (S::kRing + S::kQueryBytes));

  // blocks before each sequence
  {
    int64_t before = 0;
    for (int b0 = 0; b0 < c.sequences; b0 += S::kWarps * 32) {
      const int b = b0 + threadIdx.x;
      const int64_t n = b < c.sequences ? blocks_of(a, cache_length(c, b)) : 0;
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
      if (b < c.sequences) first[b] = before + sum - n;
      before += all;
      __syncthreads();
    }
    if (threadIdx.x == 0) first[c.sequences] = before;
    __syncthreads();
    if (blockIdx.x == 0)
      for (int b = threadIdx.x; b <= c.sequences; b += S::kWarps * 32) plan.first[b] = first[b];
  }
  const int64_t total = first[c.sequences] * c.heads * plan.tiles;
  const Shares shares(total, plan.workers);
  const int worker = blockIdx.x * S::kWarps + warp;
  const int64_t begin = shares.begin(worker), end = shares.begin(worker + 1);
  if (begin >= end) return;

  const uint32_t ring = smem_u32(smem) + warp * S::kRing;
  [[maybe_unused]] const uint32_t query_at = smem_u32(smem) + S::kWarps * S::kRing + warp * S::kQueryBytes;
  const int64_t code_extent = c.pages * c.heads * static_cast<int64_t>(c.page_tokens) * DIM;
  const int64_t scale_extent = c.pages * c.heads * static_cast<int64_t>(c.page_tokens / kCacheBlock);

  // ---- copies, kStages - 1 blocks ahead.  next_*: the block to be copied next.
  Place next = place_of(begin, first, c);
  int64_t next_at = begin;
  int64_t next_length = cache_length(c, next.b), next_start = first_seen(a, next_length);
  int64_t next_block = next_start / kCacheBlock + next.block;
  int64_t next_page = cache_page(c, next.b, next_block * kCacheBlock);
  int64_t base_of[S::kStages];  // first token's place in the pool of the blocks in the ring, -1: no page
#pragma unroll
  for (int i = 0; i < S::kStages; ++i) base_of[i] = -1;
  auto copy_next = [&](int stage, int64_t &base) {
    if (next_at < end) {
      const int64_t t0 = next_block * kCacheBlock;
      base = next_page < 0 ? -1 : (next_page * c.heads + next.h) * c.page_tokens + t0 % c.page_tokens;
      const int64_t from = base < 0 ? 0 : base * DIM;
      const uint32_t dst = ring + stage * (2 * kCacheBlock * DIM);
#pragma unroll
      for (int i = 0; i < kCacheBlock * DIM / 512; ++i) {
        const int u = i * 32 + lane, row = u / (DIM / 16), chunk = u % (DIM / 16);
        // rows that no query sees come as zeros: whatever lies there, NaN among it, stays out
        const bool in = base >= 0 && t0 + row < next_length && t0 + row >= next_start &&
                        in_bounds(from + u * 16, 16, code_extent, c.status);
        cp_async16(dst + place<DIM>(row, chunk), c.codes[0] + from + u * 16, in);
        cp_async16(dst + kCacheBlock * DIM + place<DIM>(row, chunk), c.codes[1] + from + u * 16, in);
      }
      if (++next_at < end) {
        const int b = next.b;
        advance(next, first, c);
        if (next.b != b) {
          next_length = cache_length(c, next.b);
          next_start = first_seen(a, next_length);
        }
        next_block = next_start / kCacheBlock + next.block;
        next_page = cache_page(c, next.b, next_block * kCacheBlock);
      }
    }
    cp_async_commit();
  };
#pragma unroll
  for (int i = 0; i < S::kStages - 1; ++i) copy_next(i, base_of[i]);

  // ---- the blocks, one after the other
  Place at = place_of(begin, first, c);
  float out[DIM / 8][4];
  float top[2], weight[2];       // running maximum (in powers of two) and sum, rows g and g + 8
  float factor[2];               // of a logit: scale, log2(e) and the row's power of two
  [[maybe_unused]] uint32_t query[S::kQueriesInShared ? 1 : S::kSteps][4];
  int64_t length = 0, start = 0;
  bool from_start = false, fresh = true;
  int stage = 0;
  for (int64_t f = begin; f < end; ++f) {
    if (fresh) {  // a new (tile, sequence, head): its queries
      fresh = false;
      from_start = at.block == 0;
      length = cache_length(c, at.b);
      start = first_seen(a, length);
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        top[r] = -INFINITY;
        weight[r] = 0.0f;
        const int row = at.tile * kTile + g + 8 * r;
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
        // (back in two steps, for the ends of binary32's range)
        factor[r] = a.scale * 1.4426950408889634f * exp2_int(shift / 2) * exp2_int(shift - shift / 2);
#pragma unroll
        for (int i = 0; i < S::kChunks; ++i)
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            const uint4 &v = raw[i][u >> 1];
            const uint32_t w0 = (u & 1) ? v.z : v.x, w1 = (u & 1) ? v.w : v.y;
            const uint32_t h0 = half2_bits(__uint_as_float(w0 << 16) * f1 * f2, __uint_as_float(w0 & 0xFFFF0000u) * f1 * f2);
            const uint32_t h1 = half2_bits(__uint_as_float(w1 << 16) * f1 * f2, __uint_as_float(w1 & 0xFFFF0000u) * f1 * f2);
            if constexpr (S::kQueriesInShared) {
              const uint32_t to = query_at + (i * 4 + u) * 512 + lane * 16 + r * 4;
              asm volatile("st.shared.u32 [%0], %1;" ::"r"(to), "r"(h0) : "memory");
              asm volatile("st.shared.u32 [%0], %1;" ::"r"(to + 8), "r"(h1) : "memory");
            } else {
              query[i * 4 + u][r] = h0;
              query[i * 4 + u][2 + r] = h1;
            }
          }
      }
#pragma unroll
      for (int i = 0; i < DIM / 8; ++i)
#pragma unroll
        for (int k = 0; k < 4; ++k) out[i][k] = 0.0f;
    }

    cp_async_wait<S::kStages - 2>();
    __syncwarp();  // the lanes' copies are there for all, and the stage before this one is read
    const int64_t base = base_of[0];
#pragma unroll
    for (int i = 0; i + 1 < S::kStages; ++i) base_of[i] = base_of[i + 1];
    const int free_stage = stage == 0 ? S::kStages - 1 : stage - 1;
    copy_next(free_stage, base_of[S::kStages - 2]);
    const bool held = base >= 0 && in_bounds(base / kCacheBlock, 1, scale_extent, c.status);
    const int key_exp = held ? c.scales[0][base / kCacheBlock] - 127 : 0;
    const int value_exp = held ? c.scales[1][base / kCacheBlock] - 127 : 0;
    const uint32_t keys = ring + stage * (2 * kCacheBlock * DIM), values = keys + kCacheBlock * DIM;

    // logits: s[j][0, 1] of row g and tokens 8 j + 2 t, + 1; s[j][2, 3] of row g + 8
    float s[4][4] = {};
#pragma unroll
    for (int i = 0; i < S::kChunks; ++i) {
      const int chunk = DIM == 64 ? t : 8 * (i >> 1) + 2 * t + (i & 1);
      uint4 k[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) k[j] = lds128(keys + place<DIM>(8 * j + g, chunk));
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        uint32_t q[4];
        if constexpr (S::kQueriesInShared) {
          const uint4 v = lds128(query_at + (i * 4 + u) * 512 + lane * 16);
          q[0] = v.x, q[1] = v.y, q[2] = v.z, q[3] = v.w;
        } else {
#pragma unroll
          for (int e = 0; e < 4; ++e) q[e] = query[i * 4 + u][e];
        }
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          uint32_t b0, b1;
          half4_of(u == 0 ? k[j].x : u == 1 ? k[j].y : u == 2 ? k[j].z : k[j].w, b0, b1);
          mma_f16(s[j], q, b0, b1);
        }
      }
    }

    const int64_t t0 = (start / kCacheBlock + at.block) * kCacheBlock;
    const int64_t here = length - a.q_tokens;  // position of the first query
    // do all rows see all of the block?
    const bool whole = held && t0 + kCacheBlock - 1 <= here &&
                       (a.window == 0 || t0 > here + a.q_tokens - 1 - a.window);
    uint32_t seen[2] = {0xFFu, 0xFFu};  // bit 2 j + k: the lane's token 8 j + 2 t + k
    if (!whole) {
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        const int row = at.tile * kTile + g + 8 * r;
        const int64_t p = here + row / plan.group;
        seen[r] = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const int64_t token = t0 + 8 * (i >> 1) + 2 * t + (i & 1);
          if (held && token <= p && token < length && (a.window == 0 || token > p - a.window)) seen[r] |= 1u << i;
        }
      }
    }
    // weights relative to the block's maximum, and the factors that join the block
    const float key_scale = exp2_int(key_exp), value_scale = exp2_int(value_exp);
    float keep[2], join[2];
    uint32_t p[4][2];
#pragma unroll
    for (int r = 0; r < 2; ++r) {
      float l[8], most = -INFINITY;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        l[i] = s[i >> 1][2 * r + (i & 1)] * factor[r] * key_scale;
        if (!whole && !(seen[r] >> i & 1)) l[i] = -INFINITY;
        most = fmaxf(most, l[i]);
      }
      most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
      most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
      const float ref = most == -INFINITY ? 0.0f : most;
      float sum = 0.0f;
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        l[i] = exp2_approx(l[i] - ref);
        sum += l[i];
      }
#pragma unroll
      for (int j = 0; j < 4; ++j) p[j][r] = half2_bits(l[2 * j], l[2 * j + 1]);
      const float now = fmaxf(top[r], most), now_ref = now == -INFINITY ? 0.0f : now;
      keep[r] = exp2_approx(top[r] - now_ref);
      join[r] = exp2_approx(most - now_ref);
      weight[r] = weight[r] * keep[r] + sum * join[r];
      join[r] *= value_scale;
      top[r] = now;
    }

#pragma unroll
    for (int run = 0; run < S::kRuns; ++run) {
      // the lane's tokens 16 j + 2 t, + 1 (b0) and + 8, + 9 (b1)
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
        // zero (0 * NaN would bring it to all).  With one query token no row differs.
        bool nan = false;
#pragma unroll
        for (int j = 0; j < 2; ++j)
#pragma unroll
          for (int k = 0; k < 4; ++k)
#pragma unroll
            for (int w = 0; w < kWords; ++w) nan |= any_nan(v[j][k][w]);
        if (__any_sync(0xFFFFFFFFu, nan)) {
          // the lane's values belong to columns g; its sums to columns 2 t, 2 t + 1 of rows g, g + 8
          for (int row = 0; row < kCacheBlock; ++row) {
            const int64_t token = t0 + row;
#pragma unroll
            for (int k = 0; k < 2; ++k)
              for (int e = 0; e < S::kRun; ++e) {
                const int col = (2 * t + k) * S::kRun + e;  // within the run
                uint32_t code;
                const uint32_t addr = values + place<DIM>(row, 8 * run + col / 16) + col % 16;
                asm volatile("ld.shared.u8 %0, [%1];" : "=r"(code) : "r"(addr));
                if ((code & 0x7Fu) != 0x7Fu) continue;
#pragma unroll
                for (int r = 0; r < 2; ++r) {
                  const int64_t pos = here + (at.tile * kTile + g + 8 * r) / plan.group;
                  if (held && token <= pos && token < length && (a.window == 0 || token > pos - a.window)) {
#pragma unroll
                    for (int x = 0; x < S::kRun; ++x)
                      if (x == e) out[run * S::kRun + x][2 * r + k] = NAN;
                  }
                }
              }
          }
#pragma unroll
          for (int j = 0; j < 2; ++j)
#pragma unroll
            for (int k = 0; k < 4; ++k)
#pragma unroll
              for (int w = 0; w < kWords; ++w) {
                const uint32_t high = ((v[j][k][w] & 0x7F7F7F7Fu) + 0x01010101u) & 0x80808080u;
                v[j][k][w] &= ~((high >> 7) * 0xFFu);
              }
        }
      }
#pragma unroll
      for (int w = 0; w < kWords; ++w) {
        // the same channel of two neighbouring tokens, for four channels
        uint32_t b[4][2][2];  // [channel][j][b0, b1]
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
        for (int e = 0; e < 4; ++e) {
          float part[4] = {};
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint32_t pa[4] = {p[2 * j][0], p[2 * j][1], p[2 * j + 1][0], p[2 * j + 1][1]};
            mma_f16(part, pa, b[e][j][0], b[e][j][1]);
          }
          float(&o)[4] = out[run * S::kRun + 4 * w + e];
          o[0] = o[0] * keep[0] + part[0] * join[0];
          o[1] = o[1] * keep[0] + part[1] * join[0];
          o[2] = o[2] * keep[1] + part[2] * join[1];
          o[3] = o[3] * keep[1] + part[3] * join[1];
        }
      }
    }
    stage = stage + 1 == S::kStages ? 0 : stage + 1;

    // ---- the end of a (tile, sequence, head), or of the worker's share
    const bool last = at.block + 1 == at.blocks;
    if (last || f + 1 == end) {
      fresh = true;
#pragma unroll
      for (int r = 0; r < 2; ++r) {
        float l = weight[r];
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 1);
        l += __shfl_xor_sync(0xFFFFFFFFu, l, 2);
        const int row = at.tile * kTile + g + 8 * r;
        if (row >= plan.rows) continue;
        if (from_start && last) {
          const int64_t o_row = static_cast<int64_t>(at.b) * a.q_tokens + row / plan.group;
          const int64_t head = static_cast<int64_t>(at.h) * plan.group + row % plan.group;
          const float inv = l == 0.0f ? 0.0f : 1.0f / l;
          const int64_t extent = (static_cast<int64_t>(c.sequences) * a.q_tokens - 1) * a.ld_out +
                                 static_cast<int64_t>(a.q_heads) * DIM;
#pragma unroll
          for (int run = 0; run < S::kRuns; ++run)
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int e = 0; e < S::kRun; e += 8) {
                uint32_t w[4];
#pragma unroll
                for (int u = 0; u < 4; ++u)
                  asm("cvt.rn.bf16x2.f32 %0, %1, %2;"
                      : "=r"(w[u])
                      : "f"(out[run * S::kRun + e + 2 * u + 1][2 * r + k] * inv),
                        "f"(out[run * S::kRun + e + 2 * u][2 * r + k] * inv));
                const int64_t to = o_row * a.ld_out + head * DIM + run * 128 + (2 * t + k) * S::kRun + e;
                if (in_bounds(to, 8, extent, c.status))
                  *reinterpret_cast<uint4 *>(a.out + to) = make_uint4(w[0], w[1], w[2], w[3]);
              }
          if (a.lse != nullptr && t == 0)
            a.lse[o_row * a.q_heads + head] = l == 0.0f ? -INFINITY : (top[r] + log2f(l)) * 0.6931471805599453f;
        } else {
          float *part = plan.parts + (static_cast<int64_t>(worker) * 2 + from_start) * part_floats(plan.part_rows, DIM);
          const int pr = g + 8 * r;
#pragma unroll
          for (int run = 0; run < S::kRuns; ++run)
#pragma unroll
            for (int k = 0; k < 2; ++k)
#pragma unroll
              for (int e = 0; e < S::kRun; e += 4)
                *reinterpret_cast<float4 *>(part + pr * DIM + run * 128 + (2 * t + k) * S::kRun + e) =
                    make_float4(out[run * S::kRun + e][2 * r + k], out[run * S::kRun + e + 1][2 * r + k],
                                out[run * S::kRun + e + 2][2 * r + k], out[run * S::kRun + e + 3][2 * r + k]);
          if (t == 0) {
            part[plan.part_rows * DIM + pr] = top[r];
            part[plan.part_rows * (DIM + 1) + pr] = l;
          }
        }
      }
    }
    if (f + 1 < end) advance(at, first, c);
  }
  cp_async_wait<0>();
}

// Joins the parts of one row of a (sequence, key head) that several workers share, in their
// order; a row of a sequence without blocks gets 0.
template <int DIM>
__global__ void __launch_bounds__(kJoinThreads)
    join_kernel(const __grid_constant__ AttentionArgs a, const __grid_constant__ Plan plan) {
  constexpr int kWarps = kJoinThreads / 32, kPer = DIM / 32;
  __shared__ float sums[kWarps][DIM];
  __shared__ float tops[kWarps], weights[kWarps];
  griddep_launch_dependents();
  griddep_wait();
  const CacheArgs &c = a.c;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int row = blockIdx.x % plan.rows, h = blockIdx.y, b = blockIdx.x / plan.rows;
  const int tile = row / kTile, pr = row % kTile;
  const int64_t o_row = static_cast<int64_t>(b) * a.q_tokens + row / plan.group;
  const int64_t head = static_cast<int64_t>(h) * plan.group + row % plan.group;
  const int64_t f0 = plan.first[b], blocks = plan.first[b + 1] - f0, per_tile = plan.first[c.sequences] * c.heads;
  int64_t p0 = 0, p1 = -1;
  int64_t begin = 0;
  if (blocks > 0) {
    const Shares shares(per_tile * plan.tiles, plan.workers);
    begin = tile * per_tile + f0 * c.heads + h * blocks;
    p0 = shares.owner(begin);
    p1 = shares.owner(begin + blocks - 1);
    if (p0 == p1) return;  // the worker has finished it
  }
  float sum[kPer] = {}, top = -INFINITY, weight = 0.0f;
  for (int64_t p = p0 + warp; p <= p1; p += kWarps) {
    // (the first worker's part begins the row, the others' go on with it)
    const float *part = plan.parts + (p * 2 + (p == p0)) * part_floats(plan.part_rows, DIM);
    const float m = part[plan.part_rows * DIM + pr], l = part[plan.part_rows * (DIM + 1) + pr];
    float v[kPer];
#pragma unroll
    for (int i = 0; i < kPer; ++i) v[i] = part[pr * DIM + i * 32 + lane];
    const float now = fmaxf(top, m), ref = now == -INFINITY ? 0.0f : now;
    const float keep = exp2f(top - ref), join = exp2f(m - ref);
    weight = weight * keep + l * join;
#pragma unroll
    for (int i = 0; i < kPer; ++i) sum[i] = sum[i] * keep + v[i] * join;
    top = now;
  }
#pragma unroll
  for (int i = 0; i < kPer; ++i) sums[warp][i * 32 + lane] = sum[i];
  if (lane == 0) tops[warp] = top, weights[warp] = weight;
  __syncthreads();
  float most = tops[0];
#pragma unroll
  for (int w = 1; w < kWarps; ++w) most = fmaxf(most, tops[w]);
  const float ref = most == -INFINITY ? 0.0f : most;
  float total = 0.0f, f[kWarps];
#pragma unroll
  for (int w = 0; w < kWarps; ++w) {
    f[w] = exp2f(tops[w] - ref);
    total += weights[w] * f[w];
  }
  const float inv = total == 0.0f ? 0.0f : 1.0f / total;
  const int64_t extent = (static_cast<int64_t>(c.sequences) * a.q_tokens - 1) * a.ld_out +
                         static_cast<int64_t>(a.q_heads) * DIM;
  for (int d = threadIdx.x * 2; d < DIM; d += kJoinThreads * 2) {
    float lo = 0.0f, hi = 0.0f;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) lo += sums[w][d] * f[w], hi += sums[w][d + 1] * f[w];
    uint32_t bits;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(bits) : "f"(hi * inv), "f"(lo * inv));
    const int64_t to = o_row * a.ld_out + head * DIM + d;
    if (in_bounds(to, 2, extent, c.status)) *reinterpret_cast<uint32_t *>(a.out + to) = bits;
  }
  if (a.lse != nullptr && threadIdx.x == 0)
    a.lse[o_row * a.q_heads + head] = total == 0.0f ? -INFINITY : (most + log2f(total)) * 0.6931471805599453f;
}

constexpr size_t round256(size_t n) { return (n + 255) / 256 * 256; }

template <int DIM>
size_t parts_bytes(int64_t rows) {
  const int64_t part_rows = rows < kTile ? rows : kTile;
  return static_cast<size_t>(kMaxSms) * Shape<DIM>::kWarps * 2 * static_cast<size_t>(part_floats(part_rows, DIM)) * sizeof(float);
}

template <int DIM>
cudaError_t launch(const AttentionArgs &a, cudaStream_t s) {
  using S = Shape<DIM>;
  Plan plan;
  plan.group = a.q_heads / a.c.heads;
  plan.rows = plan.group * a.q_tokens;
  plan.tiles = (plan.rows + kTile - 1) / kTile;
  plan.part_rows = plan.rows < kTile ? plan.rows : kTile;
  plan.first = static_cast<int64_t *>(a.workspace);
  plan.parts = reinterpret_cast<float *>(static_cast<uint8_t *>(a.workspace) +
                                         round256((static_cast<size_t>(a.c.sequences) + 1) * sizeof(int64_t)));
  const int ctas = a.num_sms < kMaxSms ? a.num_sms : kMaxSms;
  plan.workers = ctas * S::kWarps;
  const size_t smem = static_cast<size_t>(S::kWarps) * (S::kRing + S::kQueryBytes) +
                      (static_cast<size_t>(a.c.sequences) + 1) * sizeof(int64_t);
  const void *func = reinterpret_cast<const void *>(attention_kernel<DIM>);
  if (!kernel_setup_get(func, nullptr)) {
    const size_t most = static_cast<size_t>(S::kWarps) * (S::kRing + S::kQueryBytes) +
                        (kAttentionMaxSequences + 1) * sizeof(int64_t);
    const cudaError_t e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, static_cast<int>(most));
    if (e != cudaSuccess) return e;
    kernel_setup_put(func, 0);
  }
  const cudaError_t e = launch_pdl(attention_kernel<DIM>, dim3(static_cast<unsigned>(ctas)), dim3(S::kWarps * 32),
                                   smem, s, a, plan);
  if (e != cudaSuccess) return e;
  return launch_pdl(join_kernel<DIM>, dim3(static_cast<unsigned>(a.c.sequences) * plan.rows, a.c.heads),
                    dim3(kJoinThreads), 0, s, a, plan);
}

}  // namespace

size_t attention_workspace_bytes(int64_t sequences, int64_t rows, int head_dim) {
  const size_t first = round256((static_cast<size_t>(sequences) + 1) * sizeof(int64_t));
  switch (head_dim) {
    case 64: return first + parts_bytes<64>(rows);
    case 128: return first + parts_bytes<128>(rows);
    default: return first + parts_bytes<256>(rows);
  }
}

cudaError_t launch_attention(const AttentionArgs &a, cudaStream_t s) {
  switch (a.c.head_dim) {
    case 64: return launch<64>(a, s);
    case 128: return launch<128>(a, s);
    default: return launch<256>(a, s);
  }
}

}  // namespace mx
