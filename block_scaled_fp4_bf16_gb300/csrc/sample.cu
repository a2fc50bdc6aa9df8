// One token for each row of logits: temperature, top-k, top-p, min-p, one uniform number.
//
// What a row keeps is a prefix of its logits in descending order, so nothing is sorted: the
// threshold is a logit (and, among equal ones, an index), found by counting or by adding up
// weights on one side of it.  A thread-block cluster takes a row; each of its CTAs reads a
// contiguous slice once into shared memory, in which all further passes run.
//
// Borders are what can go wrong: with weights to binary32 the sums at a border of 10^5 tokens
// are off by more than the uniform numbers' spacing.  So a weight is computed to 2^-40 (pairs
// of binary32 numbers) and becomes a 64-bit integer in units of 2^-44: sums are then exact, in
// any order, and every comparison is one of integers.
#include "decode.h"
#include "mx_device.cuh"

namespace mx {
namespace {

constexpr int kWarps = 16, kThreads = kWarps * 32;
constexpr int kMaxCtas = 8;
constexpr int kUnit = 44;  // weights are in units of 2^-44
constexpr int kTable = 256;

// Order of logits as unsigned integers (no NaN among them).
__device__ __forceinline__ uint32_t logit_key(float v) {
  const uint32_t u = __float_as_uint(v == 0.0f ? 0.0f : v);  // (-0 equals 0)
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}
__device__ __forceinline__ float key_logit(uint32_t k) {
  return __uint_as_float((k & 0x80000000u) ? (k & 0x7FFFFFFFu) : ~k);
}

// 2^(j / 256), j < 256, as a sum of two binary32 numbers: the product of those powers
// 2^(1/2), 2^(1/4) .. 2^(1/256) that j has bits for, in units of 2^-63.
__device__ __forceinline__ float2 table_entry(int j) {
  constexpr uint64_t kRoot[8] = {0xB504F333F9DE6484ull, 0x9837F0518DB8A96Full, 0x8B95C1E3EA8BD6E7ull,
                                 0x85AAC367CC487B15ull, 0x82CD8698AC2BA1D7ull, 0x8164D1F3BC030773ull,
                                 0x80B1ED4FD999AB6Cull, 0x8058D7D2D5E5F6B1ull};
  uint64_t v = 1ull << 63;
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (j >> (7 - i) & 1) v = __umul64hi(v, kRoot[i]) << 1 | (v * kRoot[i] >> 63);
  const uint32_t hi = static_cast<uint32_t>(v >> 40);  // 24 bits: exact
  const int64_t lo = static_cast<int64_t>(v & ((1ull << 40) - 1));
  return make_float2(static_cast<float>(hi) * 0x1p-23f, static_cast<float>(lo) * 0x1p-63f);
}

// What turns a logit of the row into its weight: the largest logit, log2(e) / temperature as
// a sum of two numbers.
struct Scale {
  float top, hi, lo;
};

// round(2^44 exp((l - top) / temperature)), l <= top; 0 below 2^-45.
__device__ __forceinline__ uint64_t weight_of(float l, const Scale &c, const float2 *table) {
  if (l == c.top) return 1ull << kUnit;
  // l - top, exactly, as d + e
  const float d = l - c.top, b = d - l;
  const float e = (l - (d - b)) + (-c.top - b);
  const float p = d * c.hi;
  if (!(p > -46.0f)) return 0;
  const float pe = fmaf(d, c.hi, -p) + fmaf(d, c.lo, e * c.hi);
  // 2^(p + pe) = 2^(k / 256) 2^r
  const float kf = rintf(p * 256.0f);
  const int k = static_cast<int>(kf);
  const float r = fmaf(kf, -0x1p-8f, p);
  // y = r ln 2 as yh + yl, then e^y - 1 as q + ql
  const float yh = r * 0x1.62e43p-1f;
  const float yl = fmaf(r, 0x1.62e43p-1f, -yh) + fmaf(r, -0x1.05c61p-29f, pe * 0x1.62e43p-1f);
  const float ql = fmaf(yl, yh, yl) + yh * yh * fmaf(yh, fmaf(yh, 1.0f / 24.0f, 1.0f / 6.0f), 0.5f);
  const float qh = yh + ql, qe = ql - (qh - yh);
  // times the table's entry
  const float2 t = table[k & (kTable - 1)];
  const float m = t.x * qh;
  const float ml = fmaf(t.x, qh, -m) + fmaf(t.x, qe, fmaf(t.y, qh, t.y));
  const float s = t.x + m;
  const float sl = (m - (s - t.x)) + ml;  // the value is s + sl, s in [0.99, 2), |sl| < 2^-22
  const int64_t fixed = (static_cast<int64_t>(static_cast<int32_t>(s * 0x1p24f)) << 28) +
                        static_cast<int64_t>(__float2int_rn(sl * 0x1p52f));  // units of 2^-52
  const int shift = 52 - kUnit - (k >> 8);  // 8 .. 55
  return static_cast<uint64_t>((fixed + (1ll << (shift - 1))) >> shift);
}

// floor(f * n) for f in [0, 1) (the nearest inside, if it is outside) and n < 2^63.
__device__ __forceinline__ uint64_t part_of(float f, uint64_t n) {
  if (!(f > 0.0f)) return 0;
  if (f >= 1.0f) f = 0x1.fffffep-1f;
  const uint32_t b = __float_as_uint(f);
  const int e = max(static_cast<int>(b >> 23), 1);
  const uint64_t m = (b & 0x7FFFFFu) | ((b >> 23) ? 0x800000u : 0u);
  const int shift = 150 - e;  // f = m 2^-shift, shift >= 24
  const uint64_t lo = m * n, hi = __umul64hi(m, n);
  if (shift < 64) return lo >> shift | hi << (64 - shift);
  return shift < 128 ? hi >> (shift - 64) : 0;
}

struct Slots {
  uint64_t sum[2][kMaxCtas];
};

__device__ __forceinline__ void st_cluster_u64(uint32_t addr, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}

template <bool FP32>
__global__ void __launch_bounds__(kThreads)
    sample_kernel(const __grid_constant__ SampleArgs a, int ctas, int slice) {
  extern __shared__ uint32_t keys[];  // of this CTA's slice
  __shared__ float2 table[kTable];
  __shared__ Slots slots;
  __shared__ uint64_t warp_sums[2][kWarps];
  __shared__ Scale shared_scale;
  cluster_arrive_relaxed();
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank()), row = static_cast<int>(cluster_id_x());
  const int base = rank * slice, segment = slice / kWarps, from = warp * segment;
  const int64_t extent = static_cast<int64_t>(a.rows - 1) * a.ld + a.vocab;

  auto param = [&](const float *p, float off) {
    return p != nullptr && in_bounds(row, 1, a.rows, a.status) ? p[row] : off;
  };
  const float temperature = param(a.temperature, 1.0f), top_p = param(a.top_p, 1.0f);
  const float min_p = param(a.min_p, 0.0f), uniform = param(a.uniform, 0.0f);
  int top_k = a.top_k != nullptr && in_bounds(row, 1, a.rows, a.status) ? a.top_k[row] : 0;
  if (top_k <= 0 || top_k > a.vocab) top_k = a.vocab;

  if (threadIdx.x < kTable) table[threadIdx.x] = table_entry(threadIdx.x);
  // the slice; the largest logit, and the lowest index that has it
  uint64_t best = 0;
  bool nan = temperature != temperature || top_p != top_p || min_p != min_p || uniform != uniform;
  for (int i = from + lane; i < from + segment; i += 32) {
    const int at = base + i;
    if (at >= a.vocab) {
      keys[i] = 0;
      continue;
    }
    const int64_t e = row * a.ld + at;
    float v = 0.0f;
    if (in_bounds(e, 1, extent, a.status))
      v = FP32 ? static_cast<const float *>(a.logits)[e]
               : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(a.logits)[e]) << 16);
    nan |= v != v;
    const uint32_t k = logit_key(v);
    keys[i] = k;
    const uint64_t mine = static_cast<uint64_t>(k) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(at));
    best = mine > best ? mine : best;
  }
  if (nan) best = ~0ull;
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) {
    const uint64_t other = __shfl_xor_sync(0xFFFFFFFFu, best, m);
    best = other > best ? other : best;
  }
  if (lane == 0) warp_sums[0][warp] = best;
  cluster_wait();
  __syncthreads();

  // Every CTA's number to all of them, by turns in two sets of slots: a set is written again
  // only after the barrier that follows the reads of its last use.
  int turn = 0;
  auto share = [&](uint64_t v) {  // v: of thread 0
    if (threadIdx.x == 0)
      for (int r = 0; r < ctas; ++r)
        st_cluster_u64(mapa_shared(smem_u32(&slots.sum[turn][rank]), static_cast<uint32_t>(r)), v);
    cluster_sync();
    turn ^= 1;
    return turn ^ 1;
  };
  int sums_turn = 1;
  auto total_of = [&](uint64_t v) {  // the sum of v over the cluster's threads
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
    if (lane == 0) warp_sums[sums_turn][warp] = v;
    __syncthreads();
    uint64_t s = 0;
    if (threadIdx.x == 0)
      for (int w = 0; w < kWarps; ++w) s += warp_sums[sums_turn][w];
    sums_turn ^= 1;
    const int set = share(s);
    s = 0;
    for (int r = 0; r < ctas; ++r) s += slots.sum[set][r];
    return s;
  };

  {
    for (int w = 0; w < kWarps; ++w) best = warp_sums[0][w] > best ? warp_sums[0][w] : best;
    const int set = share(best);
    for (int r = 0; r < ctas; ++r) best = slots.sum[set][r] > best ? slots.sum[set][r] : best;
  }
  const uint32_t top_key = static_cast<uint32_t>(best >> 32);
  const float top = key_logit(top_key);
  const bool none = best == ~0ull || top == -INFINITY;
  if (none || temperature <= 0.0f) {
    if (rank == 0 && threadIdx.x == 0 && in_bounds(row, 1, a.rows, a.status)) {
      a.ids[row] = none ? -1 : static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(best));
      if (a.probability != nullptr) a.probability[row] = none ? 0.0f : 1.0f;
    }
    cluster_sync();  // (no CTA ends while another may still write to it)
    return;
  }
  if (threadIdx.x == 0) {
    const double c = 1.4426950408889634074 / static_cast<double>(fmaxf(temperature, 0x1p-100f));
    shared_scale.top = top;
    shared_scale.hi = static_cast<float>(c);
    shared_scale.lo = static_cast<float>(c - static_cast<double>(shared_scale.hi));
  }
  __syncthreads();
  const Scale scale = shared_scale;
  const uint32_t least = logit_key(-INFINITY);

  // kept: keys above `key`, and of those equal to it the ones up to index `last`
  struct Limit {
    uint32_t key;
    int last;
  };
  Limit limit{least, -1};
  auto kept = [&](uint32_t k, int i) { return k > limit.key || (k == limit.key && base + i <= limit.last); };
  auto weight = [&](uint32_t k) { return weight_of(key_logit(k), scale, table); };
  auto count_above = [&](uint32_t key) {
    uint64_t n = 0;
    for (int i = from + lane; i < from + segment; i += 32) n += keys[i] > key;
    return total_of(n);
  };
  auto mass_above = [&](uint32_t key) {
    uint64_t n = 0;
    for (int i = from + lane; i < from + segment; i += 32)
      if (keys[i] > key && kept(keys[i], i)) n += weight(keys[i]);
    return total_of(n);
  };
  // the index of the n-th of those equal to `key`
  auto nth_equal = [&](uint32_t key, uint64_t n) {
    int lo = -1, hi = a.vocab - 1;  // not enough up to lo, enough up to hi
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      uint64_t c = 0;
      for (int i = from + lane; i < from + segment; i += 32) c += keys[i] == key && base + i <= mid;
      if (total_of(c) >= n)
        hi = mid;
      else
        lo = mid;
    }
    return hi;
  };

  if (top_k < a.vocab) {
    // the largest key with fewer than top_k above it that is a logit's: the k-th logit
    uint32_t lo = least, hi = top_key;  // the k-th is in lo .. hi
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo) / 2;
      if (count_above(mid) >= static_cast<uint64_t>(top_k))
        lo = mid + 1;
      else
        hi = mid;
    }
    if (lo > least) {
      const uint64_t above = count_above(lo);
      limit.last = nth_equal(lo, static_cast<uint64_t>(top_k) - above);
      limit.key = lo;
    }
  }
  if (top_p < 1.0f) {
    const uint64_t all = mass_above(0);
    uint64_t want = part_of(top_p, all);  // the least whole number that is not below top_p * all
    // (exact but where top_p * all is whole: then one less would do)
    {
      const uint32_t b = __float_as_uint(top_p);
      const uint64_t m = (b & 0x7FFFFFu) | ((b >> 23) ? 0x800000u : 0u);
      const int shift = 150 - max(static_cast<int>(b >> 23), 1);
      const uint64_t lo = m * all;
      const bool whole = top_p <= 0.0f || (shift < 64 && (lo & ((1ull << shift) - 1)) == 0);
      if (!whole) ++want;
    }
    if (want < 1) want = 1;
    uint32_t lo = limit.key, hi = top_key;
    while (lo < hi) {
      const uint32_t mid = lo + (hi - lo) / 2;
      if (mass_above(mid) >= want)
        lo = mid + 1;
      else
        hi = mid;
    }
    const uint64_t above = mass_above(lo), each = weight(lo);
    if (each > 0 && above < want) {
      const uint64_t n = (want - above + each - 1) / each;
      const int last = nth_equal(lo, n);
      if (lo > limit.key || last < limit.last) limit.last = last;
      limit.key = lo;
    }
  }
  const uint64_t floor_weight =
      min_p > 0.0f ? static_cast<uint64_t>(ceil(fmin(static_cast<double>(min_p), 1.0) * static_cast<double>(1ull << kUnit)))
                   : 1;

  // the kept weights in the order of the indexes: warps' segments, then the one that has it
  uint64_t mine = 0;
  for (int i = from + lane; i < from + segment; i += 32)
    if (keys[i] > least && kept(keys[i], i)) {
      const uint64_t w = weight(keys[i]);
      if (w >= floor_weight) mine += w;
    }
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) mine += __shfl_xor_sync(0xFFFFFFFFu, mine, m);
  if (lane == 0) warp_sums[sums_turn][warp] = mine;
  __syncthreads();
  uint64_t sum = 0, before = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += warp_sums[sums_turn][w];
    sum += warp_sums[sums_turn][w];
  }
  const int set = share(sum);
  uint64_t all = 0;
  for (int r = 0; r < ctas; ++r) {
    if (r < rank) before += slots.sum[set][r];
    all += slots.sum[set][r];
  }
  const uint64_t target = part_of(uniform, all);  // the first place whose sum is above it
  if (before <= target && target < before + mine) {
    for (int i0 = from; i0 < from + segment; i0 += 32) {
      const int i = i0 + lane;
      uint64_t w = 0;
      if (keys[i] > least && kept(keys[i], i)) {
        w = weight(keys[i]);
        if (w < floor_weight) w = 0;
      }
      uint64_t upto = w;
#pragma unroll
      for (int m = 1; m < 32; m <<= 1) {
        const uint64_t up = __shfl_up_sync(0xFFFFFFFFu, upto, m);
        if (lane >= m) upto += up;
      }
      const uint32_t over = __ballot_sync(0xFFFFFFFFu, before + upto > target);
      if (over != 0) {
        if (lane == __ffs(over) - 1 && in_bounds(row, 1, a.rows, a.status)) {
          a.ids[row] = base + i;
          if (a.probability != nullptr)
            a.probability[row] = static_cast<float>(static_cast<double>(w) / static_cast<double>(all));
        }
        break;
      }
      before += __shfl_sync(0xFFFFFFFFu, upto, 31);
    }
  }
  cluster_sync();  // (no CTA ends while another may still write to it)
}

template <bool FP32>
cudaError_t launch(const SampleArgs &a, cudaStream_t s) {
  int ctas = 1;
  while (ctas < kMaxCtas && ctas * 4096 < a.vocab) ctas *= 2;
  const int per = (a.vocab + ctas - 1) / ctas;
  const int slice = (per + kThreads - 1) / kThreads * kThreads;
  const void *func = reinterpret_cast<const void *>(sample_kernel<FP32>);
  if (!kernel_setup_get(func, nullptr)) {
    const cudaError_t e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kSampleMaxVocab / kMaxCtas * static_cast<int>(sizeof(uint32_t)));
    if (e != cudaSuccess) return e;
    kernel_setup_put(func, 0);
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = ctas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(ctas) * static_cast<unsigned>(a.rows));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(slice) * sizeof(uint32_t);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, sample_kernel<FP32>, a, ctas, slice);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a, cudaStream_t s) {
  return a.fp32 ? launch<true>(a, s) : launch<false>(a, s);
}

}  // namespace mx
