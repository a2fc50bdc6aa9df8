// The router of a mixture-of-experts layer for a few tokens.
//
// logits = x R^T, the k largest of a token and their softmax weights.  The router's
// weights (2 E H bytes) and a few dependent steps bound it, so the work is spread
// and joined once: a thread-block cluster takes eight tokens, each of its 16 CTAs a
// sixteenth of the experts; 16 warps divide K, each product is exact (BF16 times BF16
// on the 16 x 8 x 16 product, the experts on its 16-row side) and every 32 elements
// of K are added to binary32 sums; the logits go straight into the shared memory of
// the CTA that owns the token, and one warp of it chooses.  Registers leave room for two
// CTAs an SM: with one, seven clusters of 16 are resident and the eighth (64 tokens)
// runs after them (64 x 8192 of 256: 14.9 us, so 11.0; 1 x 2048 of 64: 3.4 us, latency).
#include "fp4_digits.cuh"

namespace mx {
namespace {

constexpr int kCtas = 16;      // of a cluster
constexpr int kWarps = 16;     // of a CTA
constexpr int kTokens = 8;     // of a cluster
constexpr int kBatch = 4;      // blocks of 32 of K that a warp loads at once
constexpr int kMaxRows = kMoeMaxExperts / kCtas;   // experts of a CTA
constexpr int kRowTiles = (kMaxRows + 15) / 16;
constexpr int kLaneExperts = kMoeMaxExperts / 32;  // logits of a lane in the choice

// Order of the logits as unsigned integers: NaN first, then descending.
__device__ __forceinline__ uint32_t logit_key(float v) {
  const uint32_t u = __float_as_uint(v);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2,
                                         uint32_t a3, uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, "
      "{%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint4 load16(const void *base, int64_t elem, bool valid, int64_t extent,
                                        uint32_t *status) {
  if (!valid || !in_bounds(elem, 8, extent, status)) return make_uint4(0, 0, 0, 0);
  return *reinterpret_cast<const uint4 *>(static_cast<const uint16_t *>(base) + elem);
}

// One warp: the choice of token t from its logits.
__device__ __forceinline__ void choose(const RouteArgs &a, int t, const float *logits) {
  const int lane = threadIdx.x & 31;
  float l[kLaneExperts];
  uint32_t key[kLaneExperts];
#pragma unroll
  for (int i = 0; i < kLaneExperts; ++i) {
    const int e = i * 32 + lane;
    l[i] = e < a.experts ? logits[e] : -INFINITY;
    key[i] = e < a.experts ? logit_key(l[i]) : 0u;
  }
  const uint32_t least = logit_key(-INFINITY);
  int id = -1;              // lane j: the j-th choice
  float chosen = 0.0f, top = 0.0f, sum = 0.0f;
  for (int j = 0; j < a.top_k; ++j) {
    uint32_t best = 0;
    int at = 0;
#pragma unroll
    for (int i = 0; i < kLaneExperts; ++i) {
      if (i * 32 >= a.experts) break;
      if (key[i] > best) best = key[i], at = i;  // (the lowest index of equal ones)
    }
    const uint32_t most = __reduce_max_sync(0xFFFFFFFFu, best);
    if (most <= least) break;  // nothing but -inf is left
    const uint32_t e = __reduce_min_sync(
        0xFFFFFFFFu, best == most ? static_cast<uint32_t>(at * 32 + lane) : 0xFFFFFFFFu);
    float v = 0.0f;
#pragma unroll
    for (int i = 0; i < kLaneExperts; ++i) {
      if (i * 32 >= a.experts) break;
      if (static_cast<uint32_t>(i * 32 + lane) == e) key[i] = 0u, v = l[i];
    }
    v = __shfl_sync(0xFFFFFFFFu, v, e & 31u);
    if (j == 0) top = v;
    if (lane == j) id = static_cast<int>(e), chosen = v;
  }
  if (a.normalize) {
    sum = id >= 0 ? expf(chosen - top) : 0.0f;
  } else {
#pragma unroll
    for (int i = 0; i < kLaneExperts; ++i)
      if (i * 32 + lane < a.experts) sum += expf(l[i] - top);
  }
#pragma unroll
  for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, m);
  if (lane < a.top_k) {
    a.ids[t * a.top_k + lane] = id;
    a.weights[t * a.top_k + lane] = id < 0 ? 0.0f : expf(chosen - top) / sum;
  }
}

// What the experts' kernel that follows needs (digits: of x, of the one format that
// moe_by_token has).
struct Next {
  Image x;
  int digits;
  uint32_t *counts;
  int n_counts;
};

__global__ void __launch_bounds__(kWarps * 32, 2)
    route_kernel(const __grid_constant__ RouteArgs a, const __grid_constant__ Next next) {
  __shared__ float red[kWarps][kRowTiles][4][32];
  __shared__ float logits[kMoeMaxExperts];  // of this CTA's token
  cluster_arrive_relaxed();
  griddep_launch_dependents();
  griddep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, g = lane >> 2, t = lane & 3;
  const int rank = static_cast<int>(cluster_ctarank()), t0 = static_cast<int>(cluster_id_x()) * kTokens;
  if (blockIdx.x == 0)
    for (int i = threadIdx.x; i < next.n_counts; i += blockDim.x) next.counts[i] = 0;
  const int rows = (a.experts + kCtas - 1) / kCtas, row0 = rank * rows;
  const int n_rows = min(rows, a.experts - row0);  // may be 0 or less
  const int blocks = a.hidden / 32;
  const int64_t x_extent = (a.tokens - 1) * a.ld_x + a.hidden;
  const int64_t r_extent = static_cast<int64_t>(a.experts) * a.hidden;
  const int64_t x_row = (t0 + g) * a.ld_x + t * 8;
  const bool x_in = t0 + g < a.tokens;
#pragma unroll
  for (int m = 0; m < kRowTiles; ++m) {
    float acc[4] = {0.0f, 0.0f, 0.0f, 0.0f};
    if (m * 16 < n_rows) {
      const int r0 = m * 16 + g, r1 = r0 + 8;
      const int64_t a_row0 = static_cast<int64_t>(row0 + r0) * a.hidden + t * 8;
      const int64_t a_row1 = a_row0 + static_cast<int64_t>(8) * a.hidden;
      // lane t holds elements 8 t .. 8 t + 7 of each 32 of K, of both operands
      for (int b0 = warp; b0 < blocks; b0 += kBatch * kWarps) {
        uint4 p[kBatch], q[kBatch], x[kBatch];
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          const int b = b0 + i * kWarps;
          p[i] = load16(a.router, a_row0 + b * 32, b < blocks && r0 < n_rows, r_extent, a.status);
          q[i] = load16(a.router, a_row1 + b * 32, b < blocks && r1 < n_rows, r_extent, a.status);
          x[i] = load16(a.x, x_row + b * 32, b < blocks && x_in, x_extent, a.status);
        }
#pragma unroll
        for (int i = 0; i < kBatch; ++i) {
          float d[4] = {0.0f, 0.0f, 0.0f, 0.0f};
          mma_bf16(d, p[i].x, q[i].x, p[i].y, q[i].y, x[i].x, x[i].y);
          mma_bf16(d, p[i].z, q[i].z, p[i].w, q[i].w, x[i].z, x[i].w);
#pragma unroll
          for (int j = 0; j < 4; ++j) acc[j] += d[j];
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) red[warp][m][i][lane] = acc[i];
  }
  __syncthreads();
  // the warps' sums, in their order, to the CTA of the token, which has begun by then
  cluster_wait();
  for (int u = threadIdx.x; u < kRowTiles * 128; u += kWarps * 32) {
    const int m = u >> 7, i = (u >> 5) & 3, l = u & 31;
    const int row = m * 16 + (l >> 2) + (i >> 1) * 8, token = (l & 3) * 2 + (i & 1);
    if (row >= n_rows) continue;
    float s = red[0][m][i][l];
#pragma unroll
    for (int w = 1; w < kWarps; ++w) s += red[w][m][i][l];
    if (a.bias != nullptr && in_bounds(row0 + row, 1, a.experts, a.status)) s += a.bias[row0 + row];
    st_cluster_f32(mapa_shared(smem_u32(&logits[row0 + row]), static_cast<uint32_t>(token)), s);
  }
  cluster_sync();
  if (rank < kTokens) {
    if (t0 + rank < a.tokens && warp == 0) choose(a, t0 + rank, logits);
  } else if (next.digits) {
    // (one cluster) the other CTAs make the digits of x meanwhile
    static_assert(!moe_by_token(1, 1), "MXFP4");
    const int groups = (a.hidden + kWarps * kImageK - 1) / (kWarps * kImageK);
    for (int i = rank - kTokens; i < a.tokens * groups; i += kCtas - kTokens)
      token_digits<0, kWarps>(next.x, a.x, a.ld_x, a.tokens, a.hidden, i / groups, i % groups, nullptr,
                              a.status);
  }
}

}  // namespace

cudaError_t launch_moe_route(const RouteArgs &a, const MoeArgs *experts, cudaStream_t s) {
  Next next{};
  if (experts != nullptr) {
    next.counts = experts->counts;
    next.n_counts = moe_counts(a.tokens * a.top_k);
    if (moe_by_token(experts->fmt, a.tokens)) {
      static_assert(!moe_by_token(0, kTokens + 1), "one cluster");
      next.x = moe_image_of(*experts, false);
      next.digits = 1;
    }
  }
  const void *func = reinterpret_cast<const void *>(route_kernel);
  if (!kernel_setup_get(func, nullptr)) {
    const cudaError_t e = cudaFuncSetAttribute(func, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    kernel_setup_put(func, 0);
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = kCtas;
  attr[1].val.clusterDim.y = 1;
  attr[1].val.clusterDim.z = 1;
  cfg.gridDim = dim3(static_cast<unsigned>(kCtas * ((a.tokens + kTokens - 1) / kTokens)));
  cfg.blockDim = dim3(kWarps * 32);
  cfg.stream = s;
  cfg.attrs = attr;
  cfg.numAttrs = 2;
  return cudaLaunchKernelEx(&cfg, route_kernel, a, next);
}

}  // namespace mx
