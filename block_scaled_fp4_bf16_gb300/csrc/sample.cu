// One token for each row of logits: temperature, top-k, top-p, min-p, one uniform number.
//
// What a row keeps is a prefix of its logits in descending order, so nothing is sorted: the
// threshold is a logit (and, among equal ones, an index).  A thread-block cluster takes a
// row; each of its CTAs reads a contiguous slice once into shared memory, in which all
// further passes run.  A threshold takes three steps: counts (top-k) or weights (top-p) of
// bins of equal width in the exponent, the bin where the wanted sum is reached, and that
// bin's few logits, compared with one another by one CTA.
//
// Borders are what can go wrong: with weights to binary32 the sums at a border of 10^5 tokens
// are off by more than the uniform numbers' spacing.  So a weight is computed to 2^-40 and
// becomes a 64-bit integer in units of 2^-43: sums are then exact, in any order, and every
// comparison is one of integers.  The exponential goes by a table of 2^(j / 256) and a short
// polynomial (Tang, "Table-driven implementation of the exponential function in IEEE
// floating-point arithmetic", ACM TOMS 1989), in pairs of binary32 numbers whose parts come
// from error-free sums and products.
//
// A row is bound by the chain of its steps (a barrier of the cluster is 1 us) and by the forty
// operations of a weight, many rows by how many CTAs fit an SM (registers and the slice: two).
// 64 x 131072 with all kinds of rows: 53 us of which the logits' bytes take 5 (halving the range
// of keys for each threshold: 686 us); 1 x 32000 with top-k 11.7 us.
#include "decode.h"
#include "mx_device.cuh"

namespace mx {
namespace {

constexpr int kWarps = 16, kThreads = kWarps * 32;
constexpr int kMaxCtas = kSampleMaxCtas;
constexpr int kUnit = 43;  // weights are in units of 2^-43
constexpr int kTable = 256;
constexpr int kBins = 1024;    // the last one: all lower logits
// Powers of two that the other bins cover: first those where a threshold lies mostly (then few
// logits need an atomic addition), else all weights above 0.
constexpr float kSpan = 16.0f, kWholeSpan = 45.0f;
constexpr int kFew = 64;       // entries that are compared with one another at once
constexpr int kList = 1024;    // logits of a bin that one CTA takes
constexpr int kLimb = 15;      // bits of a weight that one 32-bit sum takes of a CTA's 2^15
constexpr int kLimbs = 3;

// Order of logits as unsigned integers (no NaN, no -0 among them).
__device__ __forceinline__ uint32_t logit_key(float v) {
  const uint32_t u = __float_as_uint(v);
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

__device__ __forceinline__ float2 both(float v) { return make_float2(v, v); }
__device__ __forceinline__ float2 add_f32x2(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 ra, rb, rd;\n mov.b64 ra, {%2, %3};\n mov.b64 rb, {%4, %5};\n"
      " add.rn.f32x2 rd, ra, rb;\n mov.b64 {%0, %1}, rd;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}
__device__ __forceinline__ float2 minus(float2 a, float2 b) {
  float2 d;
  asm("{\n .reg .b64 ra, rb, rd;\n mov.b64 ra, {%2, %3};\n mov.b64 rb, {%4, %5};\n"
      " sub.rn.f32x2 rd, ra, rb;\n mov.b64 {%0, %1}, rd;\n}\n"
      : "=f"(d.x), "=f"(d.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return d;
}

// A weight as two binary32 numbers whose bits count units: those of `high` above 4.0's units of
// 2^-21, those of `low` above kLowBase's units of 2^-43.  Sums of weights add the bits up.
struct Raw {
  float2 high, low;  // of two weights
};
constexpr uint32_t kHighBase = 0x40800000u, kLowBase = 0x35C00000u;  // 4.0, 1.5 * 2^-20
__device__ __forceinline__ uint64_t units_of(uint32_t high, uint32_t low) {
  return (static_cast<uint64_t>(high) << (kUnit - 21)) + static_cast<int64_t>(static_cast<int32_t>(low));
}
__device__ __forceinline__ uint64_t units_of(float high, float low) {
  return units_of(__float_as_uint(high) - kHighBase, __float_as_uint(low) - kLowBase);
}

// round(2^43 exp((l - top) / temperature)) of two logits l <= top (finite), 0 below 2^-44 and
// where !in.  Two at a time: a weight is some forty binary32 operations, which come in pairs.
__device__ __forceinline__ Raw weights_of(float2 l, const Scale &c, const float2 *table, const bool (&in)[2]) {
  // l - top, exactly, as d + e
  const float2 top = both(-c.top), b = minus(add_f32x2(l, top), l);
  float2 d = add_f32x2(l, top), e = add_f32x2(minus(l, minus(d, b)), minus(top, b));
  // -(l - top) / temperature in powers of two, and what its rounding leaves; a weight that is 0
  // goes on as 1, which is dropped at the end (no infinity or NaN on the way)
  float2 p = mul_f32x2(d, both(-c.hi));
  const bool some[2] = {in[0] && p.x < 46.0f, in[1] && p.y < 46.0f};
  d = make_float2(some[0] ? d.x : 0.0f, some[1] ? d.y : 0.0f);
  e = make_float2(some[0] ? e.x : 0.0f, some[1] ? e.y : 0.0f);
  p = make_float2(some[0] ? p.x : 0.0f, some[1] ? p.y : 0.0f);
  const float2 pe = fma_f32x2(d, both(c.lo), fma_f32x2(e, both(c.hi), fma_f32x2(d, both(c.hi), p)));
  // 2^(pe - p) = 2^(k / 256) 2^-r, k to the nearest: the sum with 1.5 * 2^23 ends in it (the
  // conversion instructions have an eighth of an addition's rate)
  const float2 kb = fma_f32x2(p, both(-256.0f), both(0x1.8p23f));
  const float2 r = fma_f32x2(add_f32x2(kb, both(-0x1.8p23f)), both(0x1p-8f), p);
  // y = pe ln 2 - r ln 2 as yh + yl, then e^y - 1 as qh + qe
  constexpr float kLn2 = 0x1.62e43p-1f, kLn2Low = -0x1.05c61p-29f;
  const float2 yh = mul_f32x2(r, both(-kLn2)), ny = mul_f32x2(r, both(kLn2));
  const float2 yl = fma_f32x2(pe, both(kLn2), fma_f32x2(r, both(-kLn2Low), fma_f32x2(r, both(-kLn2), ny)));
  const float2 c2 = fma_f32x2(ny, fma_f32x2(ny, both(1.0f / 24.0f), both(-1.0f / 6.0f)), both(0.5f));
  const float2 ql = fma_f32x2(yl, yh, fma_f32x2(mul_f32x2(ny, ny), c2, yl));
  const float2 qh = add_f32x2(yh, ql), qe = minus(ql, minus(qh, yh));
  // times the table's entry: s + sl, s in [0.99, 2.01), |sl| < 2^-22
  const uint32_t k0 = __float_as_uint(kb.x), k1 = __float_as_uint(kb.y);
  const float2 t0 = table[k0 & (kTable - 1)], t1 = table[k1 & (kTable - 1)];
  const float2 th = make_float2(t0.x, t1.x), tl = make_float2(t0.y, t1.y);
  const float2 m = mul_f32x2(th, qh), me = fma_f32x2(th, qh, mul_f32x2(m, both(-1.0f)));
  const float2 s = add_f32x2(th, m);
  const float2 sl = add_f32x2(minus(m, minus(s, th)), add_f32x2(fma_f32x2(th, qe, fma_f32x2(tl, qh, tl)), me));
  // times 2^(k / 256, rounded down)
  const float2 f = make_float2(some[0] ? __uint_as_float((k0 >> 8 << 23) + 0x3F800000u) : 0.0f,
                               some[1] ? __uint_as_float((k1 >> 8 << 23) + 0x3F800000u) : 0.0f);
  const float2 v = mul_f32x2(s, f), vl = mul_f32x2(sl, f);
  // in units of 2^-43: v + 4 is a multiple of 2^-21, what is left, below 2^-21 with vl, and
  // 1.5 * 2^-20 one of 2^-43
  Raw w;
  w.high = add_f32x2(v, both(4.0f));
  w.low = add_f32x2(add_f32x2(minus(v, add_f32x2(w.high, both(-4.0f))), vl), both(0x1.8p-20f));
  return w;
}

// The sum of a thread's weights: at most 64 (its part of a slice), so that 32 bits hold the
// sums of either part's units.
struct RawSum {
  uint32_t high = 0, low = 0, count = 0;
  __device__ void add(float h, float l) {
    high += __float_as_uint(h);
    low += __float_as_uint(l);
    ++count;
  }
  __device__ uint64_t total() const { return units_of(high - count * kHighBase, low - count * kLowBase); }
};

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

__device__ __forceinline__ void st_cluster_u64(uint32_t addr, uint64_t v) {
  asm volatile("st.shared::cluster.u64 [%0], %1;" ::"r"(addr), "l"(v) : "memory");
}
__device__ __forceinline__ uint32_t ld_cluster_u32(uint32_t addr) {
  uint32_t v;
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(addr) : "memory");
  return v;
}
__device__ __forceinline__ uint64_t warp_total(uint64_t v) {
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, m);
  return v;
}
__device__ __forceinline__ uint64_t warp_upto(uint64_t v, int lane) {  // the sum of the lanes up to this one
#pragma unroll
  for (int m = 1; m < 32; m <<= 1) {
    const uint64_t up = __shfl_up_sync(0xFFFFFFFFu, v, m);
    if (lane >= m) v += up;
  }
  return v;
}

// A logit and its index as one number, in the order of a row: greater logits, then lower
// indexes, are greater.
__device__ __forceinline__ uint64_t entry_of(float l, int index) {
  return static_cast<uint64_t>(logit_key(l)) << 32 | (0xFFFFFFFFu - static_cast<uint32_t>(index));
}

struct Shared {
  float2 table[kTable];
  uint32_t bins[1 + kLimbs][kBins];  // counts; weights in limbs of kLimb bits
  uint64_t list[kList];              // of the cluster's first CTA: (key, ~index)
  uint64_t slots[2][kMaxCtas];       // every CTA's number
  uint64_t sums[2][kWarps];
  uint64_t totals[kBins];            // of the cluster's bins
  uint64_t found[2];                 // what a search found
  uint32_t listed;                   // entries of a list
  int piece;
};

template <bool FP32>
__global__ void __launch_bounds__(kThreads, 2)
    sample_kernel(const __grid_constant__ SampleArgs a, int ctas, int slice, int sort_rows) {
  extern __shared__ __align__(16) float logits[];  // this CTA's slice
  __shared__ Shared sh;
  cluster_arrive_relaxed();
  griddep_launch_dependents();
  if (threadIdx.x < kTable) sh.table[threadIdx.x] = table_entry(threadIdx.x);
  for (int i = threadIdx.x; i < (1 + kLimbs) * kBins; i += kThreads) (&sh.bins[0][0])[i] = 0;
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int rank = static_cast<int>(cluster_ctarank());
  int row = static_cast<int>(cluster_id_x());
  if (sort_rows) {
    // Rows with top-p take twice as long as the others: where not all rows run at once, they
    // begin first.  This cluster's row is the one of its number in that order.
    const int i = threadIdx.x;
    const bool in = i < a.rows;
    const bool slow = in && in_bounds(i, 1, a.rows, a.status) && a.top_p[i] < 1.0f &&
                      (a.temperature == nullptr || a.temperature[i] > 0.0f);
    const uint32_t slows = __ballot_sync(0xFFFFFFFFu, slow), others = __ballot_sync(0xFFFFFFFFu, in && !slow);
    if (lane == 0) sh.sums[0][warp] = static_cast<uint64_t>(__popc(slows)) << 32 | static_cast<uint32_t>(__popc(others));
    __syncthreads();
    uint64_t before = 0, all = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sh.sums[0][w];
      all += sh.sums[0][w];
    }
    const uint32_t below = (1u << lane) - 1;
    const int place = slow ? static_cast<int>(before >> 32) + __popc(slows & below)
                           : static_cast<int>((all >> 32) + static_cast<uint32_t>(before)) + __popc(others & below);
    if (in && place == row) sh.piece = i;
    __syncthreads();
    row = sh.piece;
  }
  const int base = rank * slice, segment = slice / kWarps, from = warp * segment;
  const int64_t extent = static_cast<int64_t>(a.rows - 1) * a.ld + a.vocab;

  auto param = [&](const float *p, float off) {
    return p != nullptr && in_bounds(row, 1, a.rows, a.status) ? p[row] : off;
  };
  const float temperature = param(a.temperature, 1.0f), top_p = param(a.top_p, 1.0f);
  const float min_p = param(a.min_p, 0.0f), uniform = param(a.uniform, 0.0f);
  int top_k = a.top_k != nullptr && in_bounds(row, 1, a.rows, a.status) ? a.top_k[row] : 0;
  if (top_k <= 0 || top_k > a.vocab) top_k = a.vocab;

  // the slice, four logits a lane at a time; the largest, and the lowest index that has it
  float high = -INFINITY;
  int high_at = 0;
  bool nan = temperature != temperature || top_p != top_p || min_p != min_p || uniform != uniform;
  const bool fours = (static_cast<int64_t>(row) * a.ld) % 4 == 0;
#pragma unroll 4
  for (int i = from + lane * 4; i < from + segment; i += 128) {
    const int at = base + i;
    const int64_t e = row * a.ld + at;
    float v[4];
    if (fours && at + 4 <= a.vocab && in_bounds(e, 4, extent, a.status)) {
      if constexpr (FP32) {
        const float4 x = *reinterpret_cast<const float4 *>(static_cast<const float *>(a.logits) + e);
        v[0] = x.x, v[1] = x.y, v[2] = x.z, v[3] = x.w;
      } else {
        const uint2 x = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(a.logits) + e);
        v[0] = __uint_as_float(x.x << 16), v[1] = __uint_as_float(x.x & 0xFFFF0000u);
        v[2] = __uint_as_float(x.y << 16), v[3] = __uint_as_float(x.y & 0xFFFF0000u);
      }
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        v[j] = -INFINITY;
        if (at + j < a.vocab && in_bounds(e + j, 1, extent, a.status))
          v[j] = FP32 ? static_cast<const float *>(a.logits)[e + j]
                      : __uint_as_float(static_cast<uint32_t>(static_cast<const uint16_t *>(a.logits)[e + j]) << 16);
      }
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      nan |= v[j] != v[j];
      v[j] += 0.0f;  // (-0 equals 0)
      if (v[j] > high) high = v[j], high_at = at + j;  // (the lowest index of equal ones)
    }
    *reinterpret_cast<float4 *>(logits + i) = make_float4(v[0], v[1], v[2], v[3]);
  }
  uint64_t best = nan ? ~0ull : entry_of(high, high_at);
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) {
    const uint64_t other = __shfl_xor_sync(0xFFFFFFFFu, best, m);
    best = other > best ? other : best;
  }
  if (lane == 0) sh.sums[0][warp] = best;
  cluster_wait();
  __syncthreads();

  // Every CTA's number to all of them, by turns in two sets of slots: a set is written again
  // only after the barrier that follows the reads of its last use.
  int turn = 0;
  auto share = [&](uint64_t v) {  // v: of thread 0
    if (threadIdx.x < ctas) st_cluster_u64(mapa_shared(smem_u32(&sh.slots[turn][rank]), threadIdx.x), v);
    cluster_sync();
    turn ^= 1;
    return turn ^ 1;
  };
  {
    for (int w = 0; w < kWarps; ++w) best = sh.sums[0][w] > best ? sh.sums[0][w] : best;
    const int set = share(best);
    for (int r = 0; r < ctas; ++r) best = sh.slots[set][r] > best ? sh.slots[set][r] : best;
  }
  const float top = key_logit(static_cast<uint32_t>(best >> 32));
  const bool none = best == ~0ull || top == -INFINITY;
  if (none || temperature <= 0.0f || min_p > 1.0f) {  // (above 1 no weight reaches: the first alone is kept)
    if (rank == 0 && threadIdx.x == 0 && in_bounds(row, 1, a.rows, a.status)) {
      a.ids[row] = none ? -1 : static_cast<int32_t>(0xFFFFFFFFu - static_cast<uint32_t>(best));
      if (a.probability != nullptr) a.probability[row] = none ? 0.0f : 1.0f;
    }
    cluster_sync();  // (no CTA ends while another may still write to it)
    return;
  }
  Scale scale;
  scale.top = top;
  {
    // log2(e) / temperature as hi + lo
    const float t = fminf(fmaxf(temperature, 0x1p-100f), 0x1p100f);
    scale.hi = 0x1.715476p+0f / t;
    scale.lo = (fmaf(-scale.hi, t, 0x1.715476p+0f) + 0x1.4ae0cp-26f) / t;
  }

  // kept: logits above `limit`, and of those equal to it the ones up to index `last`
  float limit = -INFINITY;
  int limit_last = -1;
  auto kept = [&](float l, int i) { return l > limit || (l == limit && base + i <= limit_last); };
  const bool endless = top == INFINITY;  // (then those equal to it have all the weight)
  auto weight = [&](float l) -> uint64_t {
    if (endless) return l == top ? 1ull << kUnit : 0;
    const bool in[2] = {true, false};
    const Raw w = weights_of(both(l), scale, sh.table, in);
    return units_of(w.high.x, w.low.x);
  };
  // f(logit, place in the slice) for each of the warp's segment
  auto each = [&](auto &&f) {
#pragma unroll 2
    for (int i = from + lane * 4; i < from + segment; i += 128) {
      const float4 v = *reinterpret_cast<const float4 *>(logits + i);
      f(v.x, i), f(v.y, i + 1), f(v.z, i + 2), f(v.w, i + 3);
    }
  };
  // f(high, low, logit): the same with the weights (Raw) of those that are kept (0 for the others),
  // four computed side by side; a warp goes past four by 32 of which it keeps none.  (top finite)
  auto each_weight = [&](auto &&f) {
    for (int i = from + lane * 4; i < from + segment; i += 128) {
      const float4 x = *reinterpret_cast<const float4 *>(logits + i);
      const float v[4] = {x.x, x.y, x.z, x.w};
      bool in[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) in[j] = kept(v[j], i + j);
      if (!__any_sync(0xFFFFFFFFu, in[0] || in[1] || in[2] || in[3])) continue;
#pragma unroll
      for (int j = 0; j < 4; j += 2) {
        const bool pair[2] = {in[j], in[j + 1]};
        const Raw w = weights_of(make_float2(v[j], v[j + 1]), scale, sh.table, pair);
        f(w.high.x, w.low.x, v[j]);
        f(w.high.y, w.low.y, v[j + 1]);
      }
    }
  };

  // Bins of equal width in the exponent, in descending order of the logits (a logit's bin is a
  // monotonous function of it, in binary32 too).
  float per_bin = 0.0f;
  auto set_span = [&](float span) { per_bin = scale.hi * ((kBins - 1) / span); };
  const float narrow = scale.hi * ((kBins - 1) / kSpan);
  auto place_of = [&](float l) {
    const float x = l == top ? 0.0f : (top - l) * per_bin;
    return x < static_cast<float>(kBins - 1) ? x : static_cast<float>(kBins - 1);
  };
  // (to the nearest whole number: the sum with 2^23 ends in it)
  auto bin_of = [&](float l) { return __float_as_int(place_of(l) + 0x1p23f) - 0x4B000000; };
  // Logits below are in the last bin (with room for the roundings; others may be, too).
  auto far_end = [&] {
    const float width = static_cast<float>(kBins) / per_bin;
    return top - width - (fabsf(top) + width) * 0x1p-20f;
  };
  // the same within a range of bins (binary32 has 14 bits and more left there)
  auto bin_within = [&](float l, int from_bin, int to_bin) {
    const float x = (place_of(l) - static_cast<float>(from_bin) + 0.5f) *
                    (static_cast<float>(kBins - 1) / static_cast<float>(to_bin - from_bin + 1));
    return __float_as_int(x + 0x1p23f) - 0x4B000000;
  };
  auto clear_bins = [&] {
    __syncthreads();
    for (int i = threadIdx.x; i < (1 + kLimbs) * kBins; i += kThreads) (&sh.bins[0][0])[i] = 0;
    __syncthreads();
  };
  auto add_weight = [&](int bin, uint64_t w) {
#pragma unroll
    for (int l = 0; l < kLimbs; ++l) {
      const uint32_t limb = static_cast<uint32_t>(w >> (kLimb * l)) & ((1u << kLimb) - 1);
      if (limb != 0) atomicAdd(&sh.bins[1 + l][bin], limb);
    }
  };
  // Sums up to and with each thread's, and of all.
  auto scan = [&](uint64_t mine, uint64_t &all) {
    uint64_t upto = warp_upto(mine, lane);
    if (lane == 31) sh.sums[1][warp] = upto;
    __syncthreads();
    all = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) upto += sh.sums[1][w];
      all += sh.sums[1][w];
    }
    return upto;
  };
  // A thread has two neighbouring bins, or entries of the list.
  static_assert(kBins == 2 * kThreads && kList == 2 * kThreads, "two a thread");
  struct Two {
    uint64_t of[2], before;
  };
  // The cluster's sums of the bins: a CTA adds up its share of them and sends the sums to all.
  auto scan_bins = [&](bool weights, uint64_t &all) {
    cluster_sync();
    const int own = kBins / ctas;  // bins of this CTA; a thread adds up two numbers
    uint64_t n[2] = {};
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      const int item = threadIdx.x + e * kThreads, source = item / own, from_bin = rank * own + item % own;
      if (weights) {
#pragma unroll
        for (int l = 0; l < kLimbs; ++l)
          n[e] += static_cast<uint64_t>(ld_cluster_u32(mapa_shared(smem_u32(&sh.bins[1 + l][from_bin]), source))) << (kLimb * l);
      } else {
        n[e] = ld_cluster_u32(mapa_shared(smem_u32(&sh.bins[0][from_bin]), source));
      }
      sh.list[item] = n[e];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < own; i += kThreads) {
      uint64_t total = 0;
      for (int r = 0; r < ctas; ++r) total += sh.list[r * own + i];
      for (int r = 0; r < ctas; ++r) st_cluster_u64(mapa_shared(smem_u32(&sh.totals[rank * own + i]), r), total);
    }
    cluster_sync();
    Two t;
#pragma unroll
    for (int e = 0; e < 2; ++e) t.of[e] = sh.totals[2 * threadIdx.x + e];
    t.before = scan(t.of[0] + t.of[1], all) - t.of[0] - t.of[1];
    return t;
  };
  // The bin (in sh.piece) where the sum reaches `want`, and what is wanted of it (in found[1]);
  // the last bin if none does.
  auto find_bin = [&](const Two &t, uint64_t want) {
    __syncthreads();
    if (threadIdx.x == 0) sh.piece = kBins - 1;
    __syncthreads();
    uint64_t before = t.before;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
      if (before < want && want <= before + t.of[e]) sh.piece = 2 * threadIdx.x + e, sh.found[1] = want - before;
      before += t.of[e];
    }
    __syncthreads();
  };

  // The limit such that the first in order of the kept logits in the bins first_bin .. last_bin
  // are the fewest whose number (weights) comes to at least `want`, which all of them do.
  auto cut = [&](int first_bin, int last_bin, uint64_t want, bool weights) {
    int within = -1;  // a bin of the range, if not -1
    // logits outside of these are in other bins (with room for the roundings; NaN lets all through)
    const float slack = (fabsf(top) + static_cast<float>(last_bin + 1) / per_bin) * 0x1p-20f;
    const float low_end = top - (static_cast<float>(last_bin) + 0.5f) / per_bin - slack;
    const float high_end = top - (static_cast<float>(first_bin) - 0.5f) / per_bin + slack;
    auto belongs = [&](float l, int i) {
      if (l < low_end || l > high_end || !kept(l, i)) return false;
      const int bin = bin_of(l);
      return bin >= first_bin && bin <= last_bin && (within < 0 || bin_within(l, first_bin, last_bin) == within);
    };
    // how many there are; if not above kList, all of them in the first CTA's list (each CTA's own
    // come to its bins' memory first: nobody reads those any more)
    uint64_t *const mine = reinterpret_cast<uint64_t *>(&sh.bins[0][0]);
    static_assert(sizeof(sh.bins) >= kList * sizeof(uint64_t), "a list in the bins' place");
    auto gather = [&] {
      if (threadIdx.x == 0) sh.listed = 0;
      __syncthreads();
      each([&](float l, int i) {
        if (!belongs(l, i)) return;
        const uint32_t to = atomicAdd(&sh.listed, 1u);
        if (to < kList) mine[to] = entry_of(l, base + i);
      });
      __syncthreads();
      const uint32_t here = sh.listed;
      const int set = share(here);
      uint32_t before = 0, n = 0;
      for (int r = 0; r < ctas; ++r) {
        const uint32_t there = static_cast<uint32_t>(sh.slots[set][r]);
        if (r < rank) before += there;
        n += there;
      }
      if (n <= kList) {
        for (uint32_t i = threadIdx.x; i < here; i += kThreads)
          st_cluster_u64(mapa_shared(smem_u32(&sh.list[before + i]), 0), mine[i]);
        cluster_sync();
      }
      return n;
    };
    uint32_t n = gather();
    if (n > kList) {  // divide the range, too
      clear_bins();
      each([&](float l, int i) {
        if (!belongs(l, i)) return;
        if (weights)
          add_weight(bin_within(l, first_bin, last_bin), weight(l));
        else
          atomicAdd(&sh.bins[0][bin_within(l, first_bin, last_bin)], 1u);
      });
      uint64_t all;
      find_bin(scan_bins(weights, all), want);
      within = sh.piece;
      want = sh.found[1];
      n = gather();
    }
    if (n <= kList) {
      if (rank == 0) {
        // This CTA finds the one with which the sum is reached: by bins once more, now among the
        // entries, and in the bin found one by one.  `mine` takes the entries of that bin, its
        // second half their weights.
        auto within_of = [&](uint64_t entry) {
          const float l = key_logit(static_cast<uint32_t>(entry >> 32));
          if (within < 0) return bin_within(l, first_bin, last_bin);
          const float x = (place_of(l) - static_cast<float>(first_bin) + 0.5f) *
                          (static_cast<float>(kBins - 1) / static_cast<float>(last_bin - first_bin + 1));
          return __float_as_int((x - static_cast<float>(within) + 0.5f) * static_cast<float>(kBins - 1) + 0x1p23f) - 0x4B000000;
        };
        auto size_of = [&](uint64_t entry) {
          return weights ? weight(key_logit(static_cast<uint32_t>(entry >> 32))) : 1ull;
        };
        uint64_t *const sizes = mine + kList;
        static_assert(sizeof(sh.bins) >= 2 * kList * sizeof(uint64_t), "entries and weights in the bins' place");
        if (threadIdx.x == 0) sh.listed = n <= kFew ? n : 0;
        uint64_t rest = want;
        if (n <= kFew) {
          if (threadIdx.x < n) {
            mine[threadIdx.x] = sh.list[threadIdx.x];
            sizes[threadIdx.x] = size_of(sh.list[threadIdx.x]);
          }
        } else {
          for (int i = threadIdx.x; i < kBins; i += kThreads) sh.totals[i] = 0;
          __syncthreads();
          for (uint32_t i = threadIdx.x; i < n; i += kThreads)
            atomicAdd(reinterpret_cast<unsigned long long *>(&sh.totals[within_of(sh.list[i])]), size_of(sh.list[i]));
          __syncthreads();
          Two t;
#pragma unroll
          for (int e = 0; e < 2; ++e) t.of[e] = sh.totals[2 * threadIdx.x + e];
          uint64_t all;
          t.before = scan(t.of[0] + t.of[1], all) - t.of[0] - t.of[1];
          find_bin(t, want);
          const int third = sh.piece;
          rest = sh.found[1];
          for (uint32_t i = threadIdx.x; i < n; i += kThreads)
            if (within_of(sh.list[i]) == third) {
              const uint32_t to = atomicAdd(&sh.listed, 1u);
              mine[to] = sh.list[i];
              sizes[to] = size_of(sh.list[i]);
            }
        }
        __syncthreads();
        const uint32_t m = sh.listed;
        for (uint32_t i = threadIdx.x; i < m; i += kThreads) {
          uint64_t before = 0;
          for (uint32_t j = 0; j < m; ++j) before += mine[j] > mine[i] ? sizes[j] : 0;
          if (before < rest && rest <= before + sizes[i])
            for (int r = 0; r < ctas; ++r) st_cluster_u64(mapa_shared(smem_u32(&sh.found[0]), r), mine[i]);
        }
      }
      cluster_sync();
      limit = key_logit(static_cast<uint32_t>(sh.found[0] >> 32));
      limit_last = static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(sh.found[0]));
      return;
    }
    // Too many (equal logits, mostly): halve the range of keys, then find the index among those equal.
    auto total_of = [&](uint64_t v) {
      v = warp_total(v);
      __syncthreads();
      if (lane == 0) sh.sums[0][warp] = v;
      __syncthreads();
      uint64_t s = 0;
      for (int w = 0; w < kWarps; ++w) s += sh.sums[0][w];
      const int set = share(s);
      s = 0;
      for (int r = 0; r < ctas; ++r) s += sh.slots[set][r];
      return s;
    };
    auto above = [&](uint32_t key) {  // of the bin's kept ones with greater keys
      uint64_t v = 0;
      const float border = key_logit(key);
      each([&](float l, int i) {
        if (l > border && belongs(l, i)) v += weights ? weight(l) : 1;
      });
      return total_of(v);
    };
    uint32_t high = 0, low = 0xFFFFFFFFu;
    each([&](float l, int i) {
      if (belongs(l, i)) high = max(high, logit_key(l)), low = min(low, logit_key(l));
    });
    high = __reduce_max_sync(0xFFFFFFFFu, high);
    low = __reduce_min_sync(0xFFFFFFFFu, low);
    __syncthreads();
    if (lane == 0) sh.sums[0][warp] = static_cast<uint64_t>(high) << 32 | (0xFFFFFFFFu - low);
    __syncthreads();
    {
      uint32_t inverse = 0;
      high = 0;
      for (int w = 0; w < kWarps; ++w) {
        high = max(high, static_cast<uint32_t>(sh.sums[0][w] >> 32));
        inverse = max(inverse, static_cast<uint32_t>(sh.sums[0][w]));
      }
      const int set = share(static_cast<uint64_t>(high) << 32 | inverse);
      for (int r = 0; r < ctas; ++r) {
        high = max(high, static_cast<uint32_t>(sh.slots[set][r] >> 32));
        inverse = max(inverse, static_cast<uint32_t>(sh.slots[set][r]));
      }
      low = 0xFFFFFFFFu - inverse;
    }
    while (low < high) {  // the least key with less than `want` above it
      const uint32_t mid = low + (high - low) / 2;
      if (above(mid) >= want)
        low = mid + 1;
      else
        high = mid;
    }
    uint64_t rest = want - above(low);  // of those equal to it
    const float border = key_logit(low);
    if (weights) {
      const uint64_t one = weight(border);
      rest = (rest + one - 1) / one;
    }
    uint64_t equal = 0;
    each([&](float l, int) { equal += l == border; });
    equal = warp_total(equal);
    __syncthreads();
    if (lane == 0) sh.sums[0][warp] = equal;
    __syncthreads();
    uint64_t sum = 0, before = 0;
    for (int w = 0; w < kWarps; ++w) {
      if (w < warp) before += sh.sums[0][w];
      sum += sh.sums[0][w];
    }
    const int set = share(sum);
    for (int r = 0; r < rank; ++r) before += sh.slots[set][r];
    if (before < rest && rest <= before + equal) {
      for (int i0 = from; i0 < from + segment; i0 += 32) {
        const uint32_t which = __ballot_sync(0xFFFFFFFFu, logits[i0 + lane] == border);
        if (before + __popc(which) < rest) {
          before += __popc(which);
          continue;
        }
        const int bit = static_cast<int>(__fns(which, 0, static_cast<int>(rest - before)));
        if (lane < ctas) st_cluster_u64(mapa_shared(smem_u32(&sh.found[0]), lane), static_cast<uint64_t>(base + i0 + bit));
        break;
      }
    }
    cluster_sync();
    limit = border;
    limit_last = static_cast<int>(sh.found[0]);
  };

  bool dirty = false;
  if (top_k < a.vocab) {
    // The threads' largest logits first: the k-th of them is no larger than the k-th of all, and
    // not much lower where k is well below their number, so that few logits are left above it.
    set_span(kWholeSpan);
    dirty = true;
    if (high > -INFINITY) atomicAdd(&sh.bins[0][bin_of(high)], 1u);
    uint64_t threads;
    find_bin(scan_bins(false, threads), static_cast<uint64_t>(top_k));
    if (sh.piece < kBins - 1) {
      cut(0, sh.piece, static_cast<uint64_t>(top_k), false);
    } else {
      set_span(kSpan);
      for (;;) {
        if (dirty) clear_bins();
        dirty = true;
        uint32_t others = 0;
        const float far = far_end();
        each([&](float l, int) {
          const int bin = l < far ? kBins - 1 : bin_of(l);
          if (bin < kBins - 1)
            atomicAdd(&sh.bins[0][bin], 1u);
          else
            others += l > -INFINITY;
        });
        others = __reduce_add_sync(0xFFFFFFFFu, others);
        if (lane == 0) atomicAdd(&sh.bins[0][kBins - 1], others);
        uint64_t all;
        const Two bins = scan_bins(false, all);
        find_bin(bins, static_cast<uint64_t>(top_k));
        if (sh.piece < kBins - 1 || per_bin != narrow || all <= static_cast<uint64_t>(top_k)) break;
        set_span(kWholeSpan);
      }
      // (the k-th in the last bin, or less than k in all: what is cut off weighs nothing)
      if (sh.piece < kBins - 1) cut(sh.piece, sh.piece, sh.found[1], false);
    }
  }
  if (top_p < 1.0f) {
    set_span(kSpan);
    uint64_t all = 0, want = 0;
    for (;;) {
      if (dirty) clear_bins();
      dirty = true;
      uint64_t others = 0;
      if (endless) {
        each([&](float l, int i) {
          if (kept(l, i) && l == top) add_weight(0, 1ull << kUnit);
        });
      } else {
        RawSum sum;
        const float far = far_end();
        each_weight([&](float high, float low, float l) {
          const int bin = l < far ? kBins - 1 : bin_of(l);
          if (bin < kBins - 1)
            add_weight(bin, units_of(high, low));
          else
            sum.add(high, low);
        });
        others = sum.total();
      }
      others = warp_total(others);
      if (lane == 0 && others != 0) add_weight(kBins - 1, others);
      const Two bins = scan_bins(true, all);
      want = part_of(top_p, all);  // the least whole number that is not below top_p * all
      const uint32_t b = __float_as_uint(top_p);
      const uint64_t m = (b & 0x7FFFFFu) | ((b >> 23) ? 0x800000u : 0u);
      const int shift = 150 - max(static_cast<int>(b >> 23), 1);
      const bool whole = top_p <= 0.0f || (shift < 64 && ((m * all) & ((1ull << shift) - 1)) == 0);
      if (!whole) ++want;
      if (want < 1) want = 1;
      find_bin(bins, want);
      if (sh.piece < kBins - 1 || per_bin != narrow) break;
      set_span(kWholeSpan);
    }
    cut(sh.piece, sh.piece, sh.found[1], true);
  }
  const uint64_t floor_weight =
      min_p > 0.0f ? static_cast<uint64_t>(ceilf(min_p * static_cast<float>(1ull << kUnit))) : 1;
  auto final_weight = [&](float l, int i) -> uint64_t {
    if (!kept(l, i)) return 0;
    const uint64_t w = weight(l);
    return w >= floor_weight ? w : 0;
  };

  // the kept weights in the order of the indexes: by warps' segments, then within the one that
  // has the place, by all the CTA's warps
  uint64_t mine = 0;
  RawSum kept_sum;
  auto take_weight = [&](float high, float low) {
    if (floor_weight <= 1)
      kept_sum.add(high, low);
    else if (units_of(high, low) >= floor_weight)
      mine += units_of(high, low);
  };
  if (endless) {
    each([&](float l, int i) { mine += final_weight(l, i); });
  } else if (limit == -INFINITY) {
    each_weight([&](float high, float low, float) { take_weight(high, low); });
  } else {
    // those that are kept side by side (in the bins' place), so that the rest cost no weights
    __syncthreads();
    float *const dense = reinterpret_cast<float *>(&sh.bins[0][0]) + warp * 256;
    static_assert(sizeof(sh.bins) >= kWarps * 256 * sizeof(float), "each warp's kept logits in the bins' place");
    int n = 0;
    auto take = [&](int first, int count) {
      __syncwarp();
      const bool in[2] = {2 * lane < count, 2 * lane + 1 < count};
      const float2 l = make_float2(in[0] ? dense[first + 2 * lane] : top, in[1] ? dense[first + 2 * lane + 1] : top);
      const Raw w = weights_of(l, scale, sh.table, in);
      take_weight(w.high.x, w.low.x);
      take_weight(w.high.y, w.low.y);
      __syncwarp();
    };
    for (int i = from + lane * 4; i < from + segment; i += 128) {
      const float4 x = *reinterpret_cast<const float4 *>(logits + i);
      const float v[4] = {x.x, x.y, x.z, x.w};
      if (!__any_sync(0xFFFFFFFFu, fmaxf(fmaxf(v[0], v[1]), fmaxf(v[2], v[3])) >= limit)) continue;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const bool in = kept(v[j], i + j);
        const uint32_t which = __ballot_sync(0xFFFFFFFFu, in);
        if (in) dense[n + __popc(which & ((1u << lane) - 1))] = v[j];
        n += __popc(which);
      }
      while (n >= 64) n -= 64, take(n, 64);
    }
    if (n > 0) take(0, n);
  }
  mine = warp_total(mine + kept_sum.total());
  __syncthreads();
  if (lane == 0) sh.sums[0][warp] = mine;
  __syncthreads();
  uint64_t sum = 0, before = 0;
  for (int w = 0; w < kWarps; ++w) {
    if (w < warp) before += sh.sums[0][w];
    sum += sh.sums[0][w];
  }
  const int set = share(sum);
  uint64_t all = 0, cta_before = 0;
  for (int r = 0; r < ctas; ++r) {
    if (r < rank) cta_before += sh.slots[set][r];
    all += sh.slots[set][r];
  }
  const uint64_t target = part_of(uniform, all);  // the first place whose sum is above it
  if (cta_before <= target && target < cta_before + sum) {  // (one CTA's)
    before += cta_before;
    if (before <= target && target < before + mine && lane == 0) sh.piece = warp, sh.found[1] = before;
    __syncthreads();
    const int begin = sh.piece * segment;
    before = sh.found[1];
    // pieces of the segment, in order, a warp each
    const int length = (segment / 32 + kWarps - 1) / kWarps * 32;
    const int p0 = min(begin + warp * length, begin + segment), p1 = min(p0 + length, begin + segment);
    uint64_t part = 0;
    for (int i = p0 + lane; i < p1; i += 32) part += final_weight(logits[i], i);
    part = warp_total(part);
    __syncthreads();
    if (lane == 0) sh.sums[0][warp] = part;
    __syncthreads();
    for (int w = 0; w < warp; ++w) before += sh.sums[0][w];
    if (before <= target && target < before + part) {
      for (int i0 = p0; i0 < p1; i0 += 32) {
        const uint64_t w = final_weight(logits[i0 + lane], i0 + lane);
        const uint64_t upto = before + warp_upto(w, lane);
        const uint32_t over = __ballot_sync(0xFFFFFFFFu, upto > target);
        if (over != 0) {
          if (lane == __ffs(over) - 1 && in_bounds(row, 1, a.rows, a.status)) {
            a.ids[row] = base + i0 + lane;
            if (a.probability != nullptr)
              a.probability[row] = static_cast<float>(static_cast<double>(w) / static_cast<double>(all));
          }
          break;
        }
        before = __shfl_sync(0xFFFFFFFFu, upto, 31);
      }
    }
  }
  cluster_sync();  // (no CTA ends while another may still write to it)
}

// A launch of `grid` CTAs in clusters of `ctas`.
cudaLaunchConfig_t config_of(int64_t grid, int ctas, size_t smem, cudaStream_t s, cudaLaunchAttribute (&attr)[2]) {
  cudaLaunchConfig_t cfg = {};
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = ctas;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(grid));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cfg;
}

template <bool FP32>
cudaError_t launch(const SampleArgs &a, cudaStream_t s) {
  constexpr int kStep = kWarps * 128;  // a warp's segment is a multiple of 128
  const void *func = reinterpret_cast<const void *>(sample_kernel<FP32>);
  cudaLaunchAttribute attr[2];
  int most = kSamplePortableCtas;  // CTAs of a cluster
  if (!kernel_setup_get(func, &most)) {
    const cudaError_t e = cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                               kSampleMaxVocab / 8 * static_cast<int>(sizeof(float)));
    if (e != cudaSuccess) return e;
    const cudaError_t n = cudaFuncSetAttribute(func, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (n != cudaSuccess) return n;
    // is there room for the largest cluster with the largest slice (a part of a GPU may have none)?
    int clusters = 0;
    const cudaLaunchConfig_t largest =
        config_of(kMaxCtas, kMaxCtas, kSampleMaxVocab / kMaxCtas * sizeof(float), nullptr, attr);
    most = cudaOccupancyMaxActiveClusters(&clusters, func, &largest) == cudaSuccess && clusters > 0 ? kMaxCtas
                                                                                                    : kSamplePortableCtas;
    (void)cudaGetLastError();  // (an answer, not an error of this call)
    kernel_setup_put(func, most);
  }
  const int64_t rows = a.rows;
  const int ctas = sample_ctas(rows, a.vocab, a.num_sms, most);
  const int per = (a.vocab + ctas - 1) / ctas;
  const int slice = (per + kStep - 1) / kStep * kStep;
  const cudaLaunchConfig_t cfg = config_of(rows * ctas, ctas, static_cast<size_t>(slice) * sizeof(float), s, attr);
  const int sort_rows = a.top_p != nullptr && rows <= kThreads && rows * ctas > 2 * a.num_sms;
  return cudaLaunchKernelEx(&cfg, sample_kernel<FP32>, a, ctas, slice, sort_rows);
}

}  // namespace

cudaError_t launch_sample(const SampleArgs &a, cudaStream_t s) {
  return a.fp32 ? launch<true>(a, s) : launch<false>(a, s);
}

}  // namespace mx
