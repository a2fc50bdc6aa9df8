// The experts' products on the FP4 tensor cores, activations as sums of FP4
// (fp4_digits.cuh); M = 128 weight rows, N = the digits of a group's up to 16 pairs.
//
// One launch, one CTA per SM, resident together:
//   - every CTA groups the (token, slot) pairs by expert;
//   - the digits of x are written to the workspace (an "image": for a row and 256
//     elements of K the eight rows of 128 bytes as the product reads them, 128-byte
//     swizzle included, and their scales; its rows are the pairs sorted by expert, so
//     a group's lie together); a grid-wide count says that they are there;
//   - the sums of the gate and up rows; group by group, as its sums are complete, the
//     digits of h = act(gate) up; the sums of the down rows;
//   - after a second grid-wide count, y.
// The copies of weights run ahead of the counts: where a kernel boundary would leave
// the memory idle, weights stream.  (With grid-wide counts around the digits of h too:
// 64 x 4096 x 2048 of 64 173 us and 8 x 4096 x 2048 NVFP4 82 us; so 165 and 77.)
//
// Bound: at many pairs the weights' bytes (64 x 4096 x 2048 of 64 MXFP4 155 us, 5.5 TB/s
// of them; 8 x 4096 x 2048, 26 of 64 experts chosen, NVFP4 68 us, 5.5 TB/s); at few the
// chain of dependent steps (1 x 2048 x 1024 of 64 17 us: the launch before with x's digits 3,
// up sums 5, digits of h 3, down sums 2, y 2, the rest launches; the weights alone are 4).
#include "fp4_digits.cuh"
#include "moe_groups.cuh"

namespace mx {
namespace {

// ---------------------------------------------------------------- the product

// Warps: copies, product, four of the epilogue (one tensor-memory lane quarter
// each), and helpers; the last two kinds make the digits of h and y.
constexpr int kHelpers = 8;
constexpr int kWorkers = 4 + kHelpers;
constexpr int kThreads = (2 + kWorkers) * 32;
constexpr int kMaxSlots = 16;
constexpr int kSmem = 227 * 1024;
enum { kKnown, kLook, kWait };
constexpr int kTile = 128 * 128;  // bytes of a stage's weights, of one matrix
// The counts: CTAs that have written their part of the digits of x, of the down sums;
// then, for each group, items of its up sums, and its digits of h (tasks of them).
enum { kCountX, kCountDown, kCountGroups };

struct ExpertParams {
  MoeArgs a;
  Image x, h;
  int slots;      // stages in flight
  int bufs;       // accumulators (1 or 2)
  int b_off, sfa_off, sfb_off, bar_off, groups_at;  // shared memory (the weights at 0)
};

// One of the two products: UP: the gate and up rows, K = hidden, partial sums
// [parts][2][pairs (by place)][inter]; else the down rows, K = inter, [parts][pairs]
// [hidden].  An item is 128 rows (of each matrix) times a group's pairs over one
// range of K.  The items, group-major, go round the CTAs, the down items from where
// the up items end: a group is done early, and its digits of h made, while the up
// sums of the later ones run.
template <bool UP>
struct Product {
  static constexpr int kSegs = UP ? 2 : 1;
  int rows, k, stages, tiles, parts, begin, end, step;

  struct Item {
    int grp, tile, part, st0, st1;
  };
  __device__ __forceinline__ Product(const MoeArgs &a, int groups) {
    rows = UP ? a.inter : a.hidden;
    k = UP ? a.hidden : a.inter;
    stages = (k + kImageK - 1) / kImageK;
    tiles = (rows + 127) / 128;
    parts = UP ? a.up_parts : a.down_parts;
    end = groups * tiles * parts;
    step = gridDim.x;
    const int before = UP ? 0 : groups * ((a.inter + 127) / 128) * a.up_parts % step;
    begin = (static_cast<int>(blockIdx.x) - before + step) % step;
  }
  __device__ __forceinline__ Item at(int item) const {
    Item i;
    i.grp = item / (tiles * parts);
    const int r = item - i.grp * tiles * parts;
    i.tile = r / parts;
    i.part = r - i.tile * parts;
    i.st0 = stages * i.part / parts;
    i.st1 = stages * (i.part + 1) / parts;
    return i;
  }
};

// v / (1 + exp(-v)) by the exponential of -|v|, which cannot overflow: a divisor of 1 to 2,
// where the quotient is within 2 units of the last place (by exp(-v) it is 0 where that
// passes 2^126, v below -87.3).  Relative error below 2^-21, where v exp(v) is subnormal
// 2^-149 |v| besides.
__device__ __forceinline__ float silu(float v) {
  const float e = expf(-fabsf(v));
  return __fdividef(v >= 0.0f ? v : v * e, 1.0f + e);
}
// Not inlined, and called once before weights stream: as write_digits.
__device__ __noinline__ float4 act(float4 v, int gelu) {
  if (!gelu) return make_float4(silu(v.x), silu(v.y), silu(v.z), silu(v.w));
  const float2 lo = gelu_f32x2(make_float2(v.x, v.y)), hi = gelu_f32x2(make_float2(v.z, v.w));
  return make_float4(lo.x, lo.y, hi.x, hi.y);
}

// A product reads its 128 weight rows from shared memory in about 100 clocks
// however few columns it has (measured: tiles of 64 rows take as long), so tiles
// are whole 128 rows and a call with few items divides K instead.
//
// Shared memory: a ring of stages (256 of K): weights (128 rows x 128 bytes of each
// matrix), images (a kilobyte a pair), scale tiles of the weights and of the group.
// Tensor memory: accumulators [bufs][2][NB][32 columns], then a set of scale
// columns for each stage in flight, four columns for each scale tile.
// Every wait is bounded; after one that ran out the CTA's roles leave, its copies
// and products in flight are waited for, and the status word says so.
template <int FMT, int NB>
struct Expert {
  static constexpr int kGroup = 4 * NB;                 // pairs of a group at most
  // The up product multiplies the digits of all tokens with any group's weights (its time
  // does not depend on so few columns), and the epilogue takes the group's: the digits of x
  // need no order then and are made before this kernel.
  static constexpr bool kByToken = moe_by_token(FMT, kGroup);
  static constexpr int kAtoms = FMT == 0 ? 2 : 4;       // scale tiles (4 blocks) of a stage
  static constexpr int kSfa = kAtoms * 512;             // bytes, of one matrix
  static constexpr int kSfaCols = kAtoms * 4;
  static constexpr int kSfb = kImageScales<FMT>;
  static constexpr int kAccCols = 2 * NB * 32;
  static constexpr int kSfCols = 4 * kSfaCols;

  // Stages in a slot: two for the down product where the images and the second
  // stage's scales of the group fit one slot's room for images, for it has half the
  // weights of the up product in a stage and would have half as many bytes in flight
  // (8 x 4096 x 2048 NVFP4 of 64: 76.9 us with one, 69.5 so).
  template <bool UP>
  __device__ __forceinline__ int span(int grp) const {
    return !UP && 2 * g.size[grp] * kImageCodes + kSfb <= kGroup * kImageCodes ? 2 : 1;
  }

  const ExpertParams &p;
  char *smem;
  uint64_t *full, *empty, *acc_full, *acc_empty;
  volatile uint32_t *abort;
  uint32_t tmem;
  float *tops;  // [kWorkers]
  Groups g;
  uint16_t *places, *members;  // of the pairs, of the places
  int pairs;
  // the ring's place (copies or product) and the accumulator's (product or epilogue)
  uint32_t it = 0, s = 0, ph = 0, buf = 0, bph = 0;

  __device__ __forceinline__ void next_slot() {
    ++it;
    if (++s == static_cast<uint32_t>(p.slots)) s = 0, ph ^= 1u;
  }
  __device__ __forceinline__ void next_buf() {
    if (++buf == static_cast<uint32_t>(p.bufs)) buf = 0, bph ^= 1u;
  }

  // ---- copies of n stages into a slot, whose barrier expects the bytes of both kinds.
  // The second stage (of the down product) takes the place of the second matrix.
  template <bool UP>
  __device__ __forceinline__ void copy_weights(const Product<UP> &d, const CUtensorMap *m0,
                                               const CUtensorMap *m1,
                                               const typename Product<UP>::Item &im, int st, int n) {
    const MoeArgs &a = p.a;
    const int e = g.expert[im.grp], katoms = (d.k / (FMT == 0 ? 32 : 16) + 3) >> 2;
    const int64_t off = ((static_cast<int64_t>(e) * d.tiles + im.tile) * katoms + st * kAtoms) * 512;
    const uint32_t fb = smem_u32(&full[s]), w = smem_u32(smem) + s * 2 * kTile;
    const uint32_t sf = smem_u32(smem + p.sfa_off) + s * 2 * kSfa;
    const int row = e * d.rows + im.tile * 128;
    // bytes of scales, of one matrix; those of the second stage follow the first's
    const uint32_t bytes = static_cast<uint32_t>(min(n * kAtoms, katoms - st * kAtoms)) * 512u;
    mbar_arrive_expect_tx(fb, (UP ? 2 : n) * kTile + (UP ? 2 : 1) * bytes +
                                  n * (images<UP>(im.grp) * kImageCodes + kSfb));
    tma_load_2d(w, m0, st * 128, row, fb);
    bulk_load(sf, (UP ? a.gate.scales : a.down.scales) + off, bytes, fb);
    if constexpr (UP) {
      tma_load_2d(w + kTile, m1, st * 128, row, fb);
      bulk_load(sf + kSfa, a.up.scales + off, bytes, fb);
    } else if (n == 2) {
      tma_load_2d(w + kTile, m0, (st + 1) * 128, row, fb);
    }
  }
  template <bool UP>
  __device__ __forceinline__ int images(int grp) const {  // rows of images of a stage
    return UP && kByToken ? p.a.tokens : g.size[grp];
  }
  template <bool UP>
  __device__ __forceinline__ void copy_images(const Image &im, int grp, int st, uint32_t slot, int n) {
    const uint32_t fb = smem_u32(&full[slot]), size = images<UP>(grp) * kImageCodes;
    const uint32_t b = smem_u32(smem + p.b_off) + slot * kGroup * kImageCodes;
    if (UP && kByToken) {
      bulk_load(b, im.codes + static_cast<int64_t>(st) * size, size, fb);
      bulk_load(smem_u32(smem + p.sfb_off) + slot * kSfb, im.scales + static_cast<int64_t>(st) * kSfb,
                kSfb, fb);
      return;
    }
    const int64_t at = static_cast<int64_t>(st) * pairs;
    bulk_load(b, im.codes + (at + g.begin[grp]) * kImageCodes, size, fb);
    bulk_load(smem_u32(smem + p.sfb_off) + slot * kSfb, im.scales + (at + grp) * kSfb, kSfb, fb);
    if (n == 2) {
      bulk_load(b + size, im.codes + (at + pairs + g.begin[grp]) * kImageCodes, size, fb);
      bulk_load(b + 2 * size, im.scales + (at + pairs + grp) * kSfb, kSfb, fb);
    }
  }
  // The copies of a product.  ready(group, how): whether the group's images are there;
  // kKnown: as far as that is known without a look, kLook, kWait (whole warp; < 0:
  // given up).  Until they are, and while the ring has room, weights run ahead.
  template <bool UP, typename Ready>
  __device__ __forceinline__ bool copies(const Product<UP> &d, const CUtensorMap *m0,
                                         const CUtensorMap *m1, const Image &im, const Ready &ready) {
    if (d.begin >= d.end) return true;
    typename Product<UP>::Item cur{}, old = d.at(d.begin);
    int late_item = d.begin, late_st = old.st0, late = 0;  // slots whose images are still to come
    uint32_t late_slot = s;
    const auto catch_up = [&](int how) {
      while (late > 0) {
        const int there = ready(old.grp, how);
        if (there <= 0) return there == 0;
        const int by = span<UP>(old.grp);
        for (; late > 0 && late_st < old.st1; --late, late_st += by) {
          if (elect_one()) copy_images<UP>(im, old.grp, late_st, late_slot, min(by, old.st1 - late_st));
          __syncwarp();
          if (++late_slot == static_cast<uint32_t>(p.slots)) late_slot = 0;
        }
        if (late_st >= old.st1 && (late_item += d.step) < d.end) old = d.at(late_item), late_st = old.st0;
      }
      return true;
    };
    for (int item = d.begin; item < d.end; item += d.step) {
      cur = d.at(item);
      if (item != d.begin && !catch_up(kLook)) return false;
      const int by = span<UP>(cur.grp);
      for (int st = cur.st0; st < cur.st1; st += by) {
        // (the slots of the first stages come free with the products before them)
        if (late == p.slots && !catch_up(kWait)) return false;
        if (!mbar_wait_warp(smem_u32(&empty[s]), ph ^ 1u, abort, p.a.status)) return false;
        if (elect_one()) copy_weights<UP>(d, m0, m1, cur, st, min(by, cur.st1 - st));
        __syncwarp();
        ++late;
        next_slot();
        if (!catch_up(kKnown)) return false;
      }
    }
    return catch_up(kWait);
  }

  // ---- products.  One thread issues every one, so it has to cost few instructions:
  // the loops are unrolled and descriptors stepped by constants.
  template <bool UP>
  __device__ __forceinline__ bool products(const Product<UP> &d) {
    const uint32_t w_ring = smem_u32(smem), b_ring = smem_u32(smem + p.b_off);
    const uint32_t sfa_ring = smem_u32(smem + p.sfa_off), sfb_ring = smem_u32(smem + p.sfb_off);
    const uint32_t sf_tmem = tmem + p.bufs * kAccCols;
    const int katoms = (d.k / (FMT == 0 ? 32 : 16) + 3) >> 2;
    for (int item = d.begin; item < d.end; item += d.step) {
      const typename Product<UP>::Item im = d.at(item);
      // columns: the digits, to a multiple of 16
      const uint32_t columns = static_cast<uint32_t>(images<UP>(im.grp) * kDigits + 15) & ~15u;
      const uint32_t idesc0 = mma_idesc<FMT>(128, columns, 0);
      const uint32_t idesc2 = mma_idesc<FMT>(128, columns, 2);
      if (!mbar_wait_warp(smem_u32(&acc_empty[buf]), bph ^ 1u, abort, p.a.status)) return false;
      tc_fence_after();
      const uint32_t acc = tmem + buf * kAccCols;
      const int by = span<UP>(im.grp), size = g.size[im.grp] * kImageCodes;
      for (int st = im.st0; st < im.st1; st += by) {
        if (!mbar_wait_warp(smem_u32(&full[s]), ph, abort, p.a.status)) return false;
        tc_fence_after();
        if (elect_one()) {
          const uint32_t b = b_ring + s * kGroup * kImageCodes;
          const uint32_t sfa_t = sf_tmem + s * kSfCols, sfb_t = sfa_t + 2 * kSfaCols;
          const uint64_t sfa = smem_desc_scale_block(sfa_ring + s * 2 * kSfa);
          const uint64_t wd = smem_desc_sw128_kmajor(w_ring + s * 2 * kTile);
          const int last = min(by, im.st1 - st) - 1;  // of the slot's stages
          // h: the second matrix (UP), or the second stage, whose digits are its own
          const auto scales = [&](int h) {
            const uint64_t sfb =
                smem_desc_scale_block(h == 0 ? sfb_ring + s * kSfb : b + 2 * size);
            const int atoms = min(kAtoms, katoms - (UP ? st : st + h) * kAtoms);
            if (!UP || h == 0) {
#pragma unroll
              for (int j = 0; j < kAtoms; ++j)
                tc_cp_32x128b_warpx4(sfb_t + h * kSfaCols + j * 4, sfb + ((j * 512) >> 4));
            }
#pragma unroll
            for (int i = 0; i < kAtoms; ++i) {
              if (i < atoms)
                tc_cp_32x128b_warpx4(sfa_t + h * kSfaCols + i * 4, sfa + ((h * kSfa + i * 512) >> 4));
            }
          };
          const auto multiply = [&](int h, int kk, uint64_t bd) {
            const int word = FMT == 0 ? kk >> 1 : kk;
            tc_mma_block_scaled<FMT>(
                acc + (UP ? h * NB * 32 : 0), wd + h * (kTile >> 4) + 2 * kk, bd + 2 * kk,
                FMT == 0 && (kk & 1) ? idesc2 : idesc0, sfa_t + h * kSfaCols + word * 4,
                sfb_t + (UP ? 0 : h * kSfaCols) + word * 4,
                kk > 0 || st > im.st0 || (!UP && h > 0) ? 1u : 0u);
          };
          const auto steps = [&](int stage) { return min(4, (d.k - stage * kImageK + 63) >> 6); };
          const uint64_t bd = smem_desc_sw128_kmajor(b);
          scales(0);
          if constexpr (UP) {
            scales(1);
            const int n = steps(st);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk) {
              if (kk < n) {
                multiply(0, kk, bd);
                multiply(1, kk, bd);
              }
            }
          } else {
            if (last > 0) scales(1);
            const int n = steps(st);
#pragma unroll
            for (int kk = 0; kk < 4; ++kk)
              if (kk < n) multiply(0, kk, bd);
            if (last > 0) {
              const uint64_t bd1 = smem_desc_sw128_kmajor(b + size);
              const int n1 = steps(st + 1);
#pragma unroll
              for (int kk = 0; kk < 4; ++kk)
                if (kk < n1) multiply(1, kk, bd1);
            }
          }
          tc_commit(smem_u32(&empty[s]));
          if (st + last == im.st1 - 1) tc_commit(smem_u32(&acc_full[buf]));
        }
        __syncwarp();
        next_slot();
      }
      next_buf();
    }
    return true;
  }

  // ---- epilogue (a warp per lane quarter): the sums of the digits' columns.
  template <bool UP>
  __device__ __forceinline__ void epilogue(const Product<UP> &d, const float *factors) {
    constexpr int kSegs = Product<UP>::kSegs;
    constexpr bool by_token = UP && kByToken;
    const MoeArgs &a = p.a;
    const int q = (threadIdx.x >> 5) & 3, lane = threadIdx.x & 31;
    const int64_t extent = static_cast<int64_t>(d.parts) * kSegs * pairs * d.rows;
    bool ok = true;
    for (int item = d.begin; item < d.end; item += d.step) {
      const typename Product<UP>::Item im = d.at(item);
      const int e = g.expert[im.grp], n = g.size[im.grp], row = im.tile * 128 + q * 32 + lane;
      const float alpha0 = FMT == 1 ? (UP ? a.gate.ts : a.down.ts)[e] : 1.0f;
      const float alpha1 = FMT == 1 && UP ? a.up.ts[e] : 1.0f;
      // (a warp that gives up still meets the others below; nothing is counted then)
      ok = ok && mbar_wait_warp(smem_u32(&acc_full[buf]), bph, abort, a.status);
      tc_fence_after();
      const uint32_t acc = tmem + buf * kAccCols + (static_cast<uint32_t>(q * 32) << 16);
      // lane c has column block c's factor
      float factor = 1.0f;
      if (FMT == 1 && ok && lane < images<UP>(im.grp))
        factor = __ldcg(factors + (by_token ? lane : g.begin[im.grp] + lane));
      const auto put = [&](int m, int place, float v) {
        const int64_t o = (static_cast<int64_t>(im.part * kSegs + m) * pairs +
                           (UP ? place : g.list[place])) * d.rows + row;
        if (in_bounds(o, 1, extent, a.status)) (UP ? a.h : a.z)[o] = v;
      };
      for (int i = 0; ok && i < (images<UP>(im.grp) + 3) / 4; ++i) {
        float sum[kSegs][4];
#pragma unroll
        for (int m = 0; m < kSegs; ++m) {
          uint32_t r[32];
          tc_ld_32x32b_x32(acc + (m * NB + i) * 32, r);
          tc_wait_ld();
          // the least digit first
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            float t = 0.0f;
#pragma unroll
            for (int dg = kDigits - 1; dg >= 0; --dg) {
              const float v = __uint_as_float(r[j * 8 + dg]);
              if constexpr (FMT == 0)
                t = __fadd_rn(t, v);
              else
                t = __fmaf_rn(v, 1.0f / static_cast<float>(1 << digit_shift(dg)), t);
            }
            if (FMT == 1) t *= __shfl_sync(0xFFFFFFFFu, factor, i * 4 + j) * (m == 0 ? alpha0 : alpha1);
            sum[m][j] = t;
          }
        }
        if (by_token && row < d.rows) {
          for (int c = 0; c < n; ++c) {
            const int place = g.begin[im.grp] + c, t = g.list[place] / a.top_k;
            if (t >> 2 != i) continue;
#pragma unroll
            for (int m = 0; m < kSegs; ++m)
              put(m, place, (t & 2) != 0 ? (t & 1) != 0 ? sum[m][3] : sum[m][2]
                                         : (t & 1) != 0 ? sum[m][1] : sum[m][0]);
          }
        } else if (row < d.rows) {
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            if (i * 4 + j >= n) break;
#pragma unroll
            for (int m = 0; m < kSegs; ++m) put(m, g.begin[im.grp] + i * 4 + j, sum[m][j]);
          }
        }
        __syncwarp();  // (rows past the last have no outputs)
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(smem_u32(&acc_empty[buf]));
      next_buf();
      if constexpr (UP) {
        named_barrier_sync(2, 128);
        if (threadIdx.x == 64 && !*abort) release_add(up_counts() + im.grp);
      }
    }
  }

  // ---- digits of x.  A warp takes a token's stage; NVFP4's factor needs all of the
  // token: the warp looks through it first, or all the CTA's workers where only one of
  // them has a task (8 x 4096 x 2048 of 64 71.1 us, so 70.2; 1 x 8192 x 4096 of 8 40.3, so
  // 39.1).
  __device__ __forceinline__ uint4 load_x(int r, int at) const {
    const MoeArgs &a = p.a;
    const int64_t off = r * a.ld_x + at;
    return at < a.hidden && in_bounds(off, 8, (a.tokens - 1) * a.ld_x + a.hidden, a.status)
               ? *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(a.x) + off)
               : make_uint4(0, 0, 0, 0);
  }
  // The largest finite magnitude of a token; `warps` warps look, this one as number `warp`
  // (its part only).
  __device__ __noinline__ float x_top(int r, int warp, int warps) const {
    // eight loads in flight; magnitudes compare as integers, a magnitude of 0x7F80 or
    // more is no number and counts as 0
    uint32_t top = 0;
    const int lane_at = (threadIdx.x & 31) * 8;
    for (int st = warp; st * kImageK < p.a.hidden; st += 8 * warps) {
      uint4 q[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) q[i] = load_x(r, (st + i * warps) * kImageK + lane_at);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const uint32_t w[4] = {q[i].x, q[i].y, q[i].z, q[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          const uint32_t m = w[j] & 0x7FFF7FFFu;
          top = __vmaxu2(top, m & ~__vcmpgeu2(m, 0x7F807F80u));
        }
      }
    }
    top = __reduce_max_sync(0xFFFFFFFFu, max(top & 0xFFFFu, top >> 16));
    return __uint_as_float(top << 16);
  }
  // A warp's first task is loaded before the groups are made and weights stream.
  int x_stages, x_task;
  uint4 x_first;
  float x_first_top;
  __device__ __forceinline__ void fetch_x() {
    const MoeArgs &a = p.a;
    x_stages = (a.hidden + kImageK - 1) / kImageK;
    x_task = (static_cast<int>(threadIdx.x >> 5) - 2) * static_cast<int>(gridDim.x) +
             static_cast<int>(blockIdx.x);
    x_first_top = 0.0f;
    const int tasks = a.tokens * x_stages, worker = static_cast<int>(threadIdx.x >> 5) - 2;
    if (worker < 0) return;
    const bool together = FMT == 1 && tasks <= static_cast<int>(gridDim.x);
    if (x_task < tasks) {
      const int r = x_task / x_stages;
      x_first = load_x(r, (x_task - r * x_stages) * kImageK + (threadIdx.x & 31) * 8);
      if (FMT == 1 && !together) x_first_top = x_top(r, 0, 1);
    }
    if (together && static_cast<int>(blockIdx.x) < tasks) {
      const float top = x_top(static_cast<int>(blockIdx.x) / x_stages, worker, kWorkers);
      if ((threadIdx.x & 31) == 0) tops[worker] = top;
      named_barrier_sync(1, kWorkers * 32);
#pragma unroll
      for (int w = 0; w < kWorkers; ++w) x_first_top = fmaxf(x_first_top, tops[w]);
    }
  }
  __device__ __forceinline__ void split_x() {
    const MoeArgs &a = p.a;
    const int lane = threadIdx.x & 31;
    uint4 q = x_first;
    float top = x_first_top;
    for (int t = x_task; t < a.tokens * x_stages; t += kWorkers * gridDim.x) {
      const int r = t / x_stages, st = t - r * x_stages;
      if (t != x_task) {
        q = load_x(r, st * kImageK + lane * 8);
        if (FMT == 1) top = x_top(r, 0, 1);
      }
      const uint16_t *to = places + r * a.top_k;
      const uint32_t w[4] = {q.x, q.y, q.z, q.w};
      float v[8];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        v[2 * i] = __uint_as_float(w[i] << 16);
        v[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
      }
      int row_e = 0;
      if constexpr (FMT == 1) {
        row_e = row_exponent(top);
        if (st == 0 && lane < a.top_k && to[lane] != 0xFFFF) p.x.factors[to[lane]] = pow2(row_e);
      }
      write_digits<FMT>(p.x, st, v, row_e, a.top_k, to, 0, members);
    }
  }
  // ---- digits of h = act(gate) up, of the partial sums, by the helpers: a group's as
  // soon as its sums are there.  MXFP4: a warp takes a place's stage; NVFP4, whose
  // factor needs all of a place: the CTA's helpers take a place together.
  __device__ __forceinline__ uint32_t *up_counts() const { return p.a.counts + kCountGroups; }
  __device__ __forceinline__ uint32_t *h_counts() const { return up_counts() + pairs; }
  __device__ __forceinline__ int h_tasks(int grp) const {  // what h_counts()[grp] reaches
    return FMT == 0 ? g.size[grp] * ((p.a.inter + kImageK - 1) / kImageK) : g.size[grp];
  }
  __device__ __forceinline__ void split_h(const Product<true> &up, volatile uint32_t *flag) {
    const MoeArgs &a = p.a;
    const int lane = threadIdx.x & 31, helper = (threadIdx.x >> 5) - 6;
    const int groups = *g.count, stages = (a.inter + kImageK - 1) / kImageK;
    const int rows = groups == 0 ? 0 : g.begin[groups - 1] + g.size[groups - 1];
    const int64_t part = static_cast<int64_t>(pairs) * a.inter;
    const auto load = [&](int r, int at, float (&v)[8]) {
      float u[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = u[i] = 0.0f;
      if (at >= a.inter) return;
#pragma unroll
      for (int i = 0; i < 4; ++i) {  // (moe_max_parts is 4)
        if (i >= a.up_parts) break;
        const int64_t off = 2 * i * part + static_cast<int64_t>(r) * a.inter + at;
        if (!in_bounds(off, 8, 2 * a.up_parts * part, a.status) ||
            !in_bounds(off + part, 8, 2 * a.up_parts * part, a.status))
          continue;
        const float4 *s0 = reinterpret_cast<const float4 *>(a.h + off);
        const float4 *s1 = reinterpret_cast<const float4 *>(a.h + off + part);
        const float4 a0 = __ldcg(s0), a1 = __ldcg(s0 + 1), b0 = __ldcg(s1), b1 = __ldcg(s1 + 1);
        v[0] += a0.x, v[1] += a0.y, v[2] += a0.z, v[3] += a0.w;
        v[4] += a1.x, v[5] += a1.y, v[6] += a1.z, v[7] += a1.w;
        u[0] += b0.x, u[1] += b0.y, u[2] += b0.z, u[3] += b0.w;
        u[4] += b1.x, u[5] += b1.y, u[6] += b1.z, u[7] += b1.w;
      }
#pragma unroll
      for (int i = 0; i < 8; i += 4) {
        const float4 f = act(make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]), a.gelu);
        v[i] = f.x * u[i];
        v[i + 1] = f.y * u[i + 1];
        v[i + 2] = f.z * u[i + 2];
        v[i + 3] = f.w * u[i + 3];
      }
    };
    int grp = 0;
    const auto group_of = [&](int r) {  // (places only grow)
      while (r >= g.begin[grp] + g.size[grp]) ++grp;
    };
    const auto summed = [&]() {
      return count_reached(up_counts() + grp, up.tiles * up.parts, abort, a.status);
    };
    if constexpr (FMT == 0) {
      for (int t = helper * gridDim.x + blockIdx.x; t < rows * stages; t += kHelpers * gridDim.x) {
        const int r = t / stages, st = t - r * stages;
        group_of(r);
        if (!__all_sync(0xFFFFFFFFu, summed())) return;
        float v[8];
        load(r, st * kImageK + lane * 8, v);
        write_digits<FMT>(p.h, st, v, 0, 1, nullptr, r, members);
        __syncwarp();
        if (lane == 0) release_add(h_counts() + grp);
      }
    } else {
      const bool leader = helper == 0 && lane == 0;
      for (int r = blockIdx.x; r < rows; r += gridDim.x) {
        group_of(r);
        if (helper == 0) {
          const bool ok = __all_sync(0xFFFFFFFFu, summed());
          if (leader) *flag = ok ? 1u : 0u;
        }
        named_barrier_sync(3, kHelpers * 32);
        if (*flag == 0u) return;
        float top = 0.0f, v[8];
        load(r, helper * kImageK + lane * 8, v);
        raise_finite(top, v);
        for (int st = helper + kHelpers; st < stages; st += kHelpers) {
          float u[8];
          load(r, st * kImageK + lane * 8, u);
          raise_finite(top, u);
        }
        top = warp_max(top);
        if (lane == 0) tops[helper] = top;
        named_barrier_sync(3, kHelpers * 32);
#pragma unroll
        for (int w = 0; w < kHelpers; ++w) top = fmaxf(top, tops[w]);
        const int row_e = row_exponent(top);
        if (leader) p.h.factors[r] = pow2(row_e);
        for (int st = helper; st < stages; st += kHelpers) {
          if (st != helper) load(r, st * kImageK + lane * 8, v);
          write_digits<FMT>(p.h, st, v, row_e, 1, nullptr, r, members);
        }
        named_barrier_sync(3, kHelpers * 32);  // (the next place's flag and tops too)
        if (leader) release_add(h_counts() + grp);
      }
    }
  }

  // ---- y[t] = sum_j w_tj z[t, j], in the order of the slots; two columns a thread.
  __device__ __forceinline__ void combine(int worker) {
    const MoeArgs &a = p.a;
    const int lane = threadIdx.x & 31, spans = (a.hidden + 63) / 64;
    const int64_t part = static_cast<int64_t>(pairs) * a.hidden;
    for (int t = worker * gridDim.x + blockIdx.x; t < a.tokens * spans; t += kWorkers * gridDim.x) {
      const int token = t / spans, c = (t - token * spans) * 64 + lane * 2;
      // lane j has slot j's expert and weight
      int e = -1;
      float wt = 0.0f;
      if (lane < a.top_k) e = a.ids[token * a.top_k + lane], wt = a.weights[token * a.top_k + lane];
      float y0 = 0.0f, y1 = 0.0f;
      for (int j0 = 0; j0 < a.top_k; j0 += 8) {
        // all loads before any use; an empty slot's are made too and then dropped
        float2 z[8] = {};
#pragma unroll
        for (int i = 0; i < 4; ++i) {  // (moe_max_parts is 4)
          if (i >= a.down_parts) break;
          float2 v[8];
#pragma unroll
          for (int j = 0; j < 8; ++j) {
            const int slot = min(j0 + j, a.top_k - 1);
            const int64_t o = i * part + static_cast<int64_t>(token * a.top_k + slot) * a.hidden +
                              min(c, a.hidden - 2);
            v[j] = in_bounds(o, 2, a.down_parts * part, a.status)
                       ? __ldcg(reinterpret_cast<const float2 *>(a.z + o))
                       : make_float2(0.0f, 0.0f);
          }
#pragma unroll
          for (int j = 0; j < 8; ++j) z[j].x += v[j].x, z[j].y += v[j].y;
        }
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const int ej = __shfl_sync(0xFFFFFFFFu, e, (j0 + j) & 31);
          const float w = __shfl_sync(0xFFFFFFFFu, wt, (j0 + j) & 31);
          if (j0 + j < a.top_k && ej >= 0 && ej < a.experts) {
            y0 = __fmaf_rn(w, z[j].x, y0);
            y1 = __fmaf_rn(w, z[j].y, y1);
          }
        }
      }
      if (c >= a.hidden) continue;
      const int64_t o = token * a.ld_y + c;
      if (!in_bounds(o, 2, (a.tokens - 1) * a.ld_y + a.hidden, a.status)) continue;
      uint16_t *y = static_cast<uint16_t *>(a.y) + o;
      y[0] = bf16_bits(y0);
      y[1] = bf16_bits(y1);
    }
  }
};

template <int FMT, int NB>
__global__ void __launch_bounds__(kThreads, 1)
    expert_kernel(const __grid_constant__ CUtensorMap gate_map,
                  const __grid_constant__ CUtensorMap up_map,
                  const __grid_constant__ CUtensorMap down_map,
                  const __grid_constant__ ExpertParams p) {
  extern __shared__ __align__(1024) char smem[];
  const MoeArgs &a = p.a;
  const int warp = threadIdx.x >> 5;
  using X = Expert<FMT, NB>;
  X x{p, smem};
  x.full = reinterpret_cast<uint64_t *>(smem + p.bar_off);
  x.empty = x.full + p.slots;
  x.acc_full = x.empty + p.slots;   // [2]
  x.acc_empty = x.acc_full + 2;     // [2]
  uint64_t *done = x.acc_empty + 2;
  uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
  x.abort = tmem_slot + 1;
  volatile uint32_t *flag = tmem_slot + 2;
  x.tops = reinterpret_cast<float *>(tmem_slot + 4);
  x.g = Groups::at(smem + p.groups_at, a.tokens * a.top_k);
  x.places = reinterpret_cast<uint16_t *>(smem + p.groups_at + Groups::bytes(a.tokens * a.top_k));
  x.members = x.places + a.tokens * a.top_k;
  x.pairs = a.tokens * a.top_k;
  if (threadIdx.x == 0) {
    for (int s = 0; s < p.slots; ++s) {
      mbar_init(smem_u32(&x.full[s]), 1);
      mbar_init(smem_u32(&x.empty[s]), 1);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(smem_u32(&x.acc_full[i]), 1);
      mbar_init(smem_u32(&x.acc_empty[i]), 4);
    }
    mbar_init(smem_u32(done), 1);
    // the 128-byte swizzle needs 1024-byte aligned tiles
    const bool aligned = (smem_u32(smem) & 1023u) == 0;
    *x.abort = aligned ? 0u : 1u;
    if (!aligned) atomicOr(a.status, kStatusTimeout);
    fence_barrier_init();
    prefetch_tmap(&gate_map);
    prefetch_tmap(&up_map);
    prefetch_tmap(&down_map);
  }
  if (warp == 1) {
    tmem_alloc(smem_u32(tmem_slot), 512);
    tmem_relinquish();
  }
  tc_fence_before();
  griddep_launch_dependents();
  if (warp >= 2) {
    warm_digits<FMT>(p.x);
    // (the result is used, so that the call stays)
    asm volatile("" ::"f"(act(make_float4(0.0f, 0.0f, 0.0f, 0.0f), a.gelu).x));
  }
  griddep_wait();
  if constexpr (!X::kByToken) x.fetch_x();
  // (the scratch lies in the ring: a fence and a barrier before the first copy)
  make_groups<kThreads / 32>(x.g, x.places, x.members, smem, a.ids, x.pairs, a.experts, X::kGroup,
                             a.status);
  fence_proxy_async_smem();
  __syncthreads();
  tc_fence_after();
  x.tmem = *tmem_slot;
  const Product<true> up(a, *x.g.count);
  const Product<false> down(a, *x.g.count);

  if (warp == 0) {
    // the digits of x are there when every CTA has counted them
    int x_there = X::kByToken ? 1 : 0;
    if (X::kByToken) asm volatile("fence.proxy.async.global;" ::: "memory");
    const auto x_ready = [&](int, int how) {
      if (x_there == 0 && how == kWait) {
        const bool r = count_reached(a.counts + kCountX, gridDim.x, x.abort, a.status);
        x_there = __all_sync(0xFFFFFFFFu, r) != 0 ? 1 : -1;
        asm volatile("fence.proxy.async.global;" ::: "memory");  // bulk copies read what was counted
      }
      return x_there;
    };
    // those of h, of a group; a look takes in the 32 groups from it on
    int from = 0;
    uint32_t there = 0;
    const auto h_ready = [&](int grp, int how) {
      if (grp - from < 32 && (there >> (grp - from)) & 1u) return 1;
      if (how == kKnown) return 0;
      from = grp;
      const int look = grp + static_cast<int>(threadIdx.x & 31);
      const uint64_t t0 = globaltimer_ns();
      while (true) {
        there = __ballot_sync(0xFFFFFFFFu, look < *x.g.count &&
                                               load_acquire(x.h_counts() + look) >=
                                                   static_cast<uint32_t>(x.h_tasks(look)));
        if (how != kWait || (there & 1u) != 0) break;
        const bool late = globaltimer_ns() - t0 > kWaitTimeoutNs;
        if (!__any_sync(0xFFFFFFFFu, late || *x.abort != 0)) continue;
        if (late) {
          *x.abort = 1u;
          atomicOr(a.status, kStatusTimeout);
        }
        __syncwarp();
        return -1;
      }
      // (a vote orders no memory: what each lane acquired, for the lane that copies)
      __syncwarp();
      asm volatile("fence.proxy.async.global;" ::: "memory");
      return static_cast<int>(there & 1u);
    };
    if (!*x.abort && x.template copies<true>(up, &gate_map, &up_map, p.x, x_ready))
      x.template copies<false>(down, &down_map, &down_map, p.h, h_ready);
    // No copy may land after the CTA has left.  (After an abort a stage may lack
    // its images: that wait runs out, with no copy left behind it.)
    const uint32_t slots = static_cast<uint32_t>(p.slots);
    for (uint32_t j = x.it < slots ? 0u : x.it - slots; j < x.it; ++j)
      mbar_drain(smem_u32(&x.full[j % slots]), (j / slots) & 1u);
  } else if (warp == 1) {
    if (!*x.abort && x.template products<true>(up)) x.template products<false>(down);
    // every product issued has finished before the tensor memory goes
    if (elect_one()) tc_commit(smem_u32(done));
    __syncwarp();
    mbar_drain(smem_u32(done), 0u);
  } else {
    const bool epilogue = warp < 6, leader = threadIdx.x == 64;
    const auto add = [&](int i) { add_count(a.counts + i, kWorkers * 32, leader); };
    const auto wait = [&](int i) {
      return all_counted(a.counts + i, kWorkers * 32, leader, flag, x.abort, a.status);
    };
    if constexpr (!X::kByToken) {
      x.split_x();
      add(kCountX);
    }
    if (epilogue) {
      // (the factors it reads were counted before the products that it waits for)
      x.template epilogue<true>(up, p.x.factors);
      x.template epilogue<false>(down, p.h.factors);
    } else {
      x.split_h(up, flag);
    }
    add(kCountDown);
    if (wait(kCountDown)) x.combine(warp - 2);
  }
  tc_fence_before();
  __syncthreads();
  if (warp == 1) {
    __syncwarp();
    tc_fence_after();
    tmem_dealloc(x.tmem, 512);
  }
}

// What mx_moe_layer_bf16's router does there.
template <int FMT>
__global__ void __launch_bounds__(kDigitWarps<FMT> * 32)
    prepare_kernel(const __grid_constant__ MoeArgs a, const __grid_constant__ Image x, int n_counts,
                   int by_token) {
  __shared__ uint32_t tops[kDigitWarps<FMT>];
  griddep_launch_dependents();
  constexpr bool some = moe_by_token(FMT, 1);
  if (some && by_token) warm_digits<FMT>(x);
  griddep_wait();
  if (blockIdx.x == 0 && blockIdx.y == 0)
    for (int i = threadIdx.x; i < n_counts; i += kDigitWarps<FMT> * 32) a.counts[i] = 0;
  if (some && by_token)
    token_digits<FMT, kDigitWarps<FMT>>(x, a.x, a.ld_x, a.tokens, a.hidden, blockIdx.y, blockIdx.x,
                                        tops, a.status);
}

template <int FMT>
cudaError_t launch_prepare(const MoeArgs &a, cudaStream_t s) {
  const bool by_token = moe_by_token(FMT, a.tokens);
  constexpr int k = kDigitWarps<FMT> * kImageK;
  const dim3 grid(by_token ? static_cast<unsigned>((a.hidden + k - 1) / k) : 1u,
                  by_token ? static_cast<unsigned>(a.tokens) : 1u);
  return launch_pdl(prepare_kernel<FMT>, grid, dim3(kDigitWarps<FMT> * 32), 0, s, a,
                    moe_image_of(a, false), moe_counts(a.tokens * a.top_k), by_token ? 1 : 0);
}

template <int FMT, int NB>
cudaError_t launch_expert_kernel(const MoeArgs &a, cudaStream_t s) {
  using X = Expert<FMT, NB>;
  const auto kernel = expert_kernel<FMT, NB>;
  const void *func = reinterpret_cast<const void *>(kernel);
  if (!kernel_setup_get(func, nullptr)) {
    const cudaError_t e =
        cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
    if (e != cudaSuccess) return e;
    kernel_setup_put(func, 0);
  }
  const int pairs = a.tokens * a.top_k;
  ExpertParams p{};
  p.a = a;
  p.x = moe_image_of(a, false);
  p.h = moe_image_of(a, true);
  constexpr int per_slot = 2 * (kTile + X::kSfa) + X::kGroup * kImageCodes + X::kSfb;
  const int groups = Groups::bytes(pairs) + 4 * pairs;
  int slots = (kSmem - 512 - groups) / per_slot;
  slots = slots < kMaxSlots ? slots : kMaxSlots;
  p.bufs = 2 * X::kAccCols + 4 * X::kSfCols <= 512 ? 2 : 1;
  const int tmem_slots = (512 - p.bufs * X::kAccCols) / X::kSfCols;
  p.slots = slots < tmem_slots ? slots : tmem_slots;
  if (p.slots < 2) return cudaErrorInvalidValue;
  p.b_off = p.slots * 2 * kTile;
  p.sfa_off = p.b_off + p.slots * X::kGroup * kImageCodes;
  p.sfb_off = p.sfa_off + p.slots * 2 * X::kSfa;
  p.bar_off = p.sfb_off + p.slots * X::kSfb;
  p.groups_at = (p.bar_off + 8 * (2 * p.slots + 5) + 16 + kWorkers * 4 + 15) / 16 * 16;
  const int smem = p.groups_at + groups;
  // the groups' scratch lies in the weights' part of the ring
  if (smem > kSmem || p.b_off < 2 * (kThreads / 32 + 2) * a.experts) return cudaErrorInvalidValue;
  CUtensorMap gate, up, down;
  const int64_t inner = static_cast<int64_t>(a.experts) * a.inter;
  if (!encode_codes_window_map(&gate, a.gate.codes, inner, a.hidden, 128) ||
      !encode_codes_window_map(&up, a.up.codes, inner, a.hidden, 128) ||
      !encode_codes_window_map(&down, a.down.codes, static_cast<int64_t>(a.experts) * a.hidden,
                               a.inter, 128))
    return cudaErrorInvalidValue;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeCooperative;  // the CTAs wait on one another
  attr[1].val.cooperative = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(a.num_sms));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = static_cast<size_t>(smem);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, kernel, gate, up, down, p);
}

// Pairs of a group by the tokens of a call: 4, 8 or 16.
template <int FMT>
cudaError_t launch_fmt(const MoeArgs &a, cudaStream_t s) {
  if (a.tokens <= 4) return launch_expert_kernel<FMT, 1>(a, s);
  if (a.tokens <= 8) return launch_expert_kernel<FMT, 2>(a, s);
  return launch_expert_kernel<FMT, 4>(a, s);
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

cudaError_t launch_moe_prepare(const MoeArgs &a, cudaStream_t s) {
  return a.fmt == 0 ? launch_prepare<0>(a, s) : launch_prepare<1>(a, s);
}

cudaError_t launch_moe_experts(const MoeArgs &a, cudaStream_t s) {
  return a.fmt == 0 ? launch_fmt<0>(a, s) : launch_fmt<1>(a, s);
}

}  // namespace mx
