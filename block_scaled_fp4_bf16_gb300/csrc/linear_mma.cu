// mx_linear_bf16_workspace: a few BF16 rows times an FP4 weight, for weights of many
// bytes, on the FP4 tensor cores with the activations as sums of FP4 (fp4_digits.cuh).
//
// Two launches.  digits_kernel writes the digits of x to the workspace; the product,
// launched while that runs, fills its ring with weights meanwhile.  Its units are 256
// of K of 128 weight rows; the CTAs, one per SM, take equal consecutive shares of
// them, whatever tile they end in.  A tile that several CTAs share is finished by the
// last of them to arrive, which adds the sums of all in the order of K: the result
// does not depend on the order of arrival, and no CTA waits for another.
//
// Bound by the weights' bytes: 1 to 8 x 28672 x 8192 MXFP4 25.0 us, 5 TB/s of them over
// the whole call (its parts: 2 us until the first copies are under way, 20 to 22 us of
// streaming, 2 us of epilogue); 16 rows 26.5 us, 32 rows 32.9 us, where each SM reads
// twice as many bytes of digits from L2 as of weights.  NVFP4 26.2, 28.1, 35.9 us.
#include "fp4_digits.cuh"

namespace mx {
namespace {

// Warps: copies, product, two of the epilogue for each quarter of the lanes.
constexpr int kEpilogue = 8;
constexpr int kThreads = (2 + kEpilogue) * 32;
constexpr int kSmem = 227 * 1024;
constexpr int kMaxSlots = 12;
constexpr int kTile = 128 * 128;  // bytes of a stage's weights

struct Params {
  LinearArgs a;
  Image x;
  float *parts;      // [CTA][first or last tile of its share][tokens][128]
  uint32_t *counts;  // [tiles]: CTAs that have written their sums
  int tiles, stages;
  int each, more;                             // units of a CTA (Share)
  int slots, b_bytes;                         // stages in flight; bytes of a stage's digits
  int b_off, sfa_off, sfb_off, bar_off;       // shared memory (the weights at 0)
};

template <int FMT>
__global__ void __launch_bounds__(kDigitWarps<FMT> * 32) digits_kernel(const __grid_constant__ Params p) {
  __shared__ uint32_t tops[kDigitWarps<FMT>];
  warm_digits<FMT>(p.x);
  griddep_wait();
  griddep_launch_dependents();  // after the wait: what the product copies before its own
                                // wait is then older than this kernel
  const int cta = blockIdx.y * gridDim.x + blockIdx.x;
  for (int i = cta * blockDim.x + threadIdx.x; i < p.tiles; i += gridDim.x * gridDim.y * blockDim.x)
    p.counts[i] = 0;
  const LinearArgs &a = p.a;
  token_digits<FMT, kDigitWarps<FMT>>(p.x, a.x, a.ld_x, a.tokens, a.k, blockIdx.y, blockIdx.x, tops,
                                      a.status);
}

// ---------------------------------------------------------------- the product

// A CTA's share of the units (the first `more` CTAs have one more than `each`), and
// who shares a tile.
struct Share {
  int each, more;
  __device__ __forceinline__ int begin(int cta) const { return cta * each + min(cta, more); }
  __device__ __forceinline__ int owner(int unit) const {
    const int first = more * (each + 1);
    return unit < first ? unit / (each + 1) : more + (unit - first) / each;
  }
};

// NB: columns of the accumulator in units of 32 (four tokens' digits).
template <int FMT, int NB>
struct Shape {
  static constexpr int kAtoms = FMT == 0 ? 2 : 4;  // scale tiles (4 blocks) of a stage
  static constexpr int kSfa = kAtoms * 512;
  static constexpr int kHalves = NB == 8 ? 2 : 1;  // scale tiles of 128 digit rows
  static constexpr int kSfb = kHalves * kImageScales<FMT>;
  static constexpr int kAccCols = NB * 32;
  static constexpr int kBufs = NB == 8 ? 1 : 2;
  static constexpr int kSfbCols = kAtoms * 4 * kHalves;
  static constexpr int kSfCols = kAtoms * 4 + kSfbCols;
};

template <int FMT, int NB>
__global__ void __launch_bounds__(kThreads, 1)
    product_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ Params p) {
  using S = Shape<FMT, NB>;
  extern __shared__ __align__(1024) char smem[];
  const LinearArgs &a = p.a;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  uint64_t *full = reinterpret_cast<uint64_t *>(smem + p.bar_off);
  uint64_t *empty = full + p.slots;
  uint64_t *acc_full = empty + p.slots;  // [2]
  uint64_t *acc_empty = acc_full + 2;    // [2]
  uint64_t *done = acc_empty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
  volatile uint32_t *abort = tmem_slot + 1;
  volatile uint32_t *last = tmem_slot + 2;  // [first or last tile][before, after its sums]
  const Share share{p.each, p.more};
  const int begin = share.begin(blockIdx.x), end = share.begin(blockIdx.x + 1);
  const int katoms = static_cast<int>((a.k / (FMT == 0 ? 32 : 16) + 3) >> 2);
  const uint32_t slots = static_cast<uint32_t>(p.slots);
  const auto weights = [&](int unit, uint32_t s) {
    const int tile = unit / p.stages, st = unit - tile * p.stages;
    const uint32_t fb = smem_u32(&full[s]);
    const uint32_t bytes = static_cast<uint32_t>(min(S::kAtoms, katoms - st * S::kAtoms)) * 512u;
    mbar_arrive_expect_tx(fb, kTile + bytes + a.tokens * kImageCodes + S::kSfb);
    tma_load_2d(smem_u32(smem) + s * kTile, &map, st * 128, tile * 128, fb);
    bulk_load(smem_u32(smem + p.sfa_off) + s * S::kSfa,
              a.w.scales + (static_cast<int64_t>(tile) * katoms + st * S::kAtoms) * 512, bytes, fb);
  };
  const auto digits = [&](int unit, uint32_t s) {
    const int64_t st = unit % p.stages;
    const uint32_t fb = smem_u32(&full[s]);
    bulk_load(smem_u32(smem + p.b_off) + s * p.b_bytes, p.x.codes + st * a.tokens * kImageCodes,
              a.tokens * kImageCodes, fb);
    bulk_load(smem_u32(smem + p.sfb_off) + s * S::kSfb, p.x.scales + st * S::kSfb, S::kSfb, fb);
  };
  const int ahead = min(p.slots, end - begin);  // stages copied before the first wait
  if (warp == 0) {
    if (elect_one()) {
      for (int s = 0; s < p.slots; ++s) {
        mbar_init(smem_u32(&full[s]), 1);
        mbar_init(smem_u32(&empty[s]), 1);
      }
      for (int i = 0; i < 2; ++i) {
        mbar_init(smem_u32(&acc_full[i]), 1);
        mbar_init(smem_u32(&acc_empty[i]), kEpilogue);
      }
      mbar_init(smem_u32(done), 1);
      *abort = 0u;
      fence_barrier_init();
      // the weights before the digits are there
      for (int i = 0; i < ahead; ++i) weights(begin + i, i);
    }
    __syncwarp();
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  griddep_launch_dependents();
  __syncthreads();
  tc_fence_after();
  const uint32_t tmem = *tmem_slot;

  if (warp == 0) {
    griddep_wait();
    asm volatile("fence.proxy.async.global;" ::: "memory");
    if (elect_one())
      for (int i = 0; i < ahead; ++i) digits(begin + i, i);
    __syncwarp();
    uint32_t it = ahead, s = ahead == p.slots ? 0 : ahead, ph = ahead == p.slots ? 1 : 0;
    for (int unit = begin + ahead; unit < end && !*abort; ++unit) {
      if (!mbar_wait_warp(smem_u32(&empty[s]), ph ^ 1u, abort, a.status)) break;
      if (elect_one()) {
        weights(unit, s);
        digits(unit, s);
      }
      __syncwarp();
      ++it;
      if (++s == slots) s = 0, ph ^= 1u;
    }
    // no copy may land after the CTA has left
    for (uint32_t j = it < slots ? 0u : it - slots; j < it; ++j)
      mbar_drain(smem_u32(&full[j % slots]), (j / slots) & 1u);
  } else if (warp == 1) {
    // one thread issues every product: unrolled, descriptors stepped by constants
    const uint32_t w_ring = smem_u32(smem), b_ring = smem_u32(smem + p.b_off);
    const uint32_t sfa_ring = smem_u32(smem + p.sfa_off), sfb_ring = smem_u32(smem + p.sfb_off);
    const uint32_t sf_tmem = tmem + S::kBufs * S::kAccCols;
    const uint32_t columns = static_cast<uint32_t>(a.tokens * kDigits + 15) & ~15u;
    const uint32_t idesc0 = mma_idesc<FMT>(128, columns, 0), idesc2 = mma_idesc<FMT>(128, columns, 2);
    uint32_t s = 0, ph = 0, buf = 0, bph = 0;
    bool ok = true;
    for (int unit = begin; ok && unit < end;) {
      const int tile = unit / p.stages, st0 = unit - tile * p.stages;
      const int st1 = min(p.stages, st0 + end - unit);
      unit += st1 - st0;
      if (!(ok = mbar_wait_warp(smem_u32(&acc_empty[buf]), bph ^ 1u, abort, a.status))) break;
      tc_fence_after();
      const uint32_t acc = tmem + buf * S::kAccCols;
      for (int st = st0; st < st1; ++st) {
        if (!(ok = mbar_wait_warp(smem_u32(&full[s]), ph, abort, a.status))) break;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t sfa_t = sf_tmem + s * S::kSfCols, sfb_t = sfa_t + S::kAtoms * 4;
          const uint64_t sfa = smem_desc_scale_block(sfa_ring + s * S::kSfa);
          const uint64_t sfb = smem_desc_scale_block(sfb_ring + s * S::kSfb);
          const int atoms = min(S::kAtoms, katoms - st * S::kAtoms);
          const int steps = static_cast<int>(
              min(static_cast<int64_t>(4), (a.k - static_cast<int64_t>(st) * kImageK + 63) >> 6));
#pragma unroll
          for (int j = 0; j < S::kAtoms; ++j) {
#pragma unroll
            for (int h = 0; h < S::kHalves; ++h)
              tc_cp_32x128b_warpx4(sfb_t + (j * S::kHalves + h) * 4,
                                   sfb + ((h * kImageScales<FMT> + j * 512) >> 4));
          }
#pragma unroll
          for (int j = 0; j < S::kAtoms; ++j)
            if (j < atoms) tc_cp_32x128b_warpx4(sfa_t + j * 4, sfa + ((j * 512) >> 4));
          const uint64_t wd = smem_desc_sw128_kmajor(w_ring + s * kTile);
          const uint64_t bd = smem_desc_sw128_kmajor(b_ring + s * p.b_bytes);
#pragma unroll
          for (int kk = 0; kk < 4; ++kk) {
            if (kk < steps) {
              const int word = FMT == 0 ? kk >> 1 : kk;
              tc_mma_block_scaled<FMT>(acc, wd + 2 * kk, bd + 2 * kk,
                                       FMT == 0 && (kk & 1) ? idesc2 : idesc0, sfa_t + word * 4,
                                       sfb_t + word * 4 * S::kHalves, kk > 0 || st > st0 ? 1u : 0u);
            }
          }
          tc_commit(smem_u32(&empty[s]));
          if (st == st1 - 1) tc_commit(smem_u32(&acc_full[buf]));
        }
        __syncwarp();
        if (++s == slots) s = 0, ph ^= 1u;
      }
      if (++buf == S::kBufs) buf = 0, bph ^= 1u;
    }
    // every product issued has finished before the tensor memory goes
    if (elect_one()) tc_commit(smem_u32(done));
    __syncwarp();
    mbar_drain(smem_u32(done), 0u);
  } else {
    griddep_wait();
    const int q = warp & 3, row = q * 32 + lane, half = (warp - 2) >> 2;
    const float alpha = FMT == 1 ? *a.w.ts : 1.0f;
    // lane t has token t's factor
    const float factor = FMT == 1 && lane < a.tokens ? __ldcg(p.x.factors + lane) : 1.0f;
    const int64_t parts_extent = static_cast<int64_t>(gridDim.x) * 2 * a.tokens * 128;
    const bool leader = threadIdx.x == 64;
    // outputs of a warp (of a row): blocks of four tokens, every other one
    constexpr int kMine = NB == 1 ? 4 : NB * 2;
    const auto token = [&](int i) { return ((i >> 2) * 2 + half) * 4 + (i & 3); };
    uint32_t buf = 0, bph = 0;
    bool ok = true;
    for (int unit = begin; unit < end;) {
      const int tile = unit / p.stages, st0 = unit - tile * p.stages;
      const int st1 = min(p.stages, st0 + end - unit);
      const bool whole = st0 == 0 && st1 == p.stages;
      const int64_t at = static_cast<int64_t>(tile) * 128 + row;
      const int first = tile * p.stages;
      const int c0 = whole ? blockIdx.x : share.owner(first);
      const int c1 = whole ? blockIdx.x : share.owner(first + p.stages - 1);
      const int word = unit == begin ? 0 : 2;
      unit += st1 - st0;
      // CTA c's sums of this tile, token t
      const auto part = [&](int c, int t) {
        return ((c * 2 + (share.begin(c) >= first ? 0 : 1)) * a.tokens + t) * 128 + row;
      };
      const auto load_part = [&](int c, int i) {  // output i of this warp's
        const int o = part(c, min(token(i), a.tokens - 1));
        return in_bounds(o, 1, parts_extent, a.status) ? __ldcg(p.parts + o) : 0.0f;
      };
      const auto put = [&](float v, int i) {
        if (token(i) >= a.tokens || at >= a.n) return;
        if (FMT == 1) v *= alpha;
        // (a block that holds an infinity or NaN has digits that are NaN as a whole)
        if (!(fabsf(v) < __uint_as_float(0x7F800000u))) v = wide_sum<FMT>(a, at, token(i));
        put_linear(a, at, token(i), v);
      };
      // Of two CTAs the second to arrive, if it is clear before its own sums are there,
      // fetches the other's meanwhile; the order of two does not matter.
      const bool two = c1 - c0 == 1;
      bool finish = whole;
      float v[kMine] = {};
      if (two) {
        if (leader) last[word] = load_acquire(p.counts + tile);
        named_barrier_sync(1, kEpilogue * 32);
        finish = last[word] != 0;
        if (finish) {
#pragma unroll
          for (int i = 0; i < kMine; ++i) v[i] = load_part(c0 + c1 - blockIdx.x, i);
        }
      }
      // (a warp that gives up still meets the others below; nothing is counted then)
      ok = ok && mbar_wait_warp(smem_u32(&acc_full[buf]), bph, abort, a.status);
      tc_fence_after();
      const uint32_t acc = tmem + buf * S::kAccCols + (static_cast<uint32_t>(q * 32) << 16);
#pragma unroll
      for (int i = 0; i < kMine; i += 4) {
        if (!ok || token(i) >= a.tokens) break;
        uint32_t r[32];
        tc_ld_32x32b_x32(acc + token(i) * kDigits, r);
        tc_wait_ld();
        // the least digit first
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          float u = 0.0f;
#pragma unroll
          for (int dg = kDigits - 1; dg >= 0; --dg) {
            const float d = __uint_as_float(r[j * 8 + dg]);
            if constexpr (FMT == 0)
              u = __fadd_rn(u, d);
            else
              u = __fmaf_rn(d, 1.0f / static_cast<float>(1 << digit_shift(dg)), u);
          }
          if (FMT == 1) u *= __shfl_sync(0xFFFFFFFFu, factor, (token(i) + j) & 31);
          if (finish) {
            put(two ? v[i + j] + u : u, i + j);
          } else if (token(i) + j < a.tokens) {
            const int o = part(blockIdx.x, token(i) + j);
            if (in_bounds(o, 1, parts_extent, a.status)) p.parts[o] = u;
          }
        }
        __syncwarp();  // (an output may have taken some lanes through wide_sum)
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&acc_empty[buf]));
      if (++buf == S::kBufs) buf = 0, bph ^= 1u;
      if (finish) continue;
      // the last of the tile's CTAs adds the sums of all
      named_barrier_sync(1, kEpilogue * 32);
      if (leader)
        last[word + 1] = *abort == 0 &&
                         acquire_release_add(p.counts + tile) == static_cast<uint32_t>(c1 - c0);
      named_barrier_sync(1, kEpilogue * 32);
      if (last[word + 1] == 0) continue;
#pragma unroll
      for (int i = 0; i < kMine; ++i) v[i] = load_part(c0, i);
#pragma unroll(kMine <= 4 ? 4 : 2)
      for (int c = c0 + 1; c <= c1; ++c) {
#pragma unroll
        for (int i = 0; i < kMine; ++i) v[i] += load_part(c, i);
      }
#pragma unroll
      for (int i = 0; i < kMine; ++i) put(v[i], i);
      __syncwarp();
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

size_t round256(size_t v) { return (v + 255) / 256 * 256; }

struct Layout {
  size_t codes, scales, factors, parts, counts, bytes;
};
Layout layout_of(int fmt, int64_t tokens, int64_t n, int64_t k) {
  const size_t stages = static_cast<size_t>((k + kImageK - 1) / kImageK);
  Layout l;
  l.codes = 0;
  l.scales = round256(stages * static_cast<size_t>(tokens) * kImageCodes);
  l.factors = l.scales + round256(stages * static_cast<size_t>(tokens > kTileRows ? 2 : 1) *
                                  (fmt == 0 ? kImageScales<0> : kImageScales<1>));
  l.parts = l.factors + 256;
  l.counts = l.parts + static_cast<size_t>(kLinearCtas) * 2 * static_cast<size_t>(tokens) * 512;
  l.bytes = l.counts + round256(static_cast<size_t>((n + 127) / 128) * 4);
  return l;
}

template <int FMT, int NB>
cudaError_t launch_product(Params p, cudaStream_t s) {
  using S = Shape<FMT, NB>;
  const auto kernel = product_kernel<FMT, NB>;
  const void *func = reinterpret_cast<const void *>(kernel);
  if (!kernel_setup_get(func, nullptr)) {
    const cudaError_t e =
        cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    kernel_setup_put(func, 0);
  }
  const LinearArgs &a = p.a;
  p.b_bytes = (a.tokens + 1) / 2 * 2 * kImageCodes;  // (the product has 16 columns at least)
  const int per_slot = kTile + S::kSfa + p.b_bytes + S::kSfb;
  int slots = (kSmem - 512) / per_slot;
  constexpr int tmem_slots = (512 - S::kBufs * S::kAccCols) / S::kSfCols;
  slots = slots < tmem_slots ? slots : tmem_slots;
  p.slots = slots < kMaxSlots ? slots : kMaxSlots;
  if (p.slots < 2) return cudaErrorInvalidValue;
  p.b_off = p.slots * kTile;
  p.sfa_off = p.b_off + p.slots * p.b_bytes;
  p.sfb_off = p.sfa_off + p.slots * S::kSfa;
  p.bar_off = p.sfb_off + p.slots * S::kSfb;
  const int smem = p.bar_off + 8 * (2 * p.slots + 5) + 32;
  if (smem > kSmem) return cudaErrorInvalidValue;
  CUtensorMap map;
  if (!encode_codes_window_map(&map, a.w.codes, a.n, a.k, 128)) return cudaErrorInvalidValue;
  const int units = p.tiles * p.stages;
  int ctas = a.num_sms < kLinearCtas ? a.num_sms : kLinearCtas;
  // With many tokens every end of a share costs an epilogue of 2 us: tiles divided
  // evenly where that leaves few SMs idle (32 x 8192 x 8192 NVFP4: 22.1 us, so 20.1; 8 x
  // 8192 x 28672, bound by the weights, 30.7 us and would take 33.3).
  if (const int even = ctas / p.tiles * p.tiles; NB == 8 && even * 5 >= ctas * 4) ctas = even;
  if (ctas > units) ctas = units;
  p.each = units / ctas;
  p.more = units % ctas;
  return launch_pdl(kernel, dim3(static_cast<unsigned>(ctas)), dim3(kThreads), smem, s, map, p);
}

template <int FMT>
cudaError_t launch_fmt(const Params &p, cudaStream_t s) {
  const dim3 grid((p.stages + kDigitWarps<FMT> - 1) / kDigitWarps<FMT>,
                  static_cast<unsigned>(p.a.tokens));
  const dim3 block(kDigitWarps<FMT> * 32);
  cudaError_t e;
  if (FMT == 1 && p.a.tokens > 16) {
    // Launched early, so many CTAs crowd on the SMs that the kernel before it leaves
    // first and hold up the product's there (32 x 8192 x 8192: 27.9 us; so 22.1).
    digits_kernel<FMT><<<grid, block, 0, s>>>(p);
    e = cudaGetLastError();
  } else {
    e = launch_pdl(digits_kernel<FMT>, grid, block, 0, s, p);
  }
  if (e != cudaSuccess) return e;
  if (p.a.tokens <= 4) return launch_product<FMT, 1>(p, s);
  if (p.a.tokens <= 8) return launch_product<FMT, 2>(p, s);
  if (p.a.tokens <= 16) return launch_product<FMT, 4>(p, s);
  return launch_product<FMT, 8>(p, s);
}

}  // namespace

size_t linear_workspace_bytes(int fmt, int64_t tokens, int64_t n, int64_t k) {
  const int64_t tiles = (n + 127) / 128, stages = (k + kImageK - 1) / kImageK;
  if (tiles * stages >= (int64_t(1) << 31)) return 0;
  return layout_of(fmt, tokens, n, k).bytes;
}

cudaError_t launch_linear_mma(const LinearArgs &a, void *workspace, cudaStream_t s) {
  const Layout l = layout_of(a.fmt, a.tokens, a.n, a.k);
  uint8_t *ws = static_cast<uint8_t *>(workspace);
  Params p{};

  p.a = a;
  p.tiles = static_cast<int>((a.n + 127) / 128);
  p.stages = static_cast<int>((a.k + kImageK - 1) / kImageK);
  p.x = Image{ws + l.codes, ws + l.scales, reinterpret_cast<float *>(ws + l.factors), a.tokens,
              a.tokens > kTileRows ? 2 : 1};
  p.parts = reinterpret_cast<float *>(ws + l.parts);
  p.counts = reinterpret_cast<uint32_t *>(ws + l.counts);
  return a.fmt == 0 ? launch_fmt<0>(p, s) : launch_fmt<1>(p, s);
}

}  // namespace mx
