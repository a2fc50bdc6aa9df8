// Mixture of experts for a few tokens: the router, and the two products of the
// chosen experts.
#include <cstdlib>
#include "few_tokens.cuh"
#include "moe_groups.cuh"

namespace mx {
namespace {

constexpr int kWarps = 8;

// Order of the logits as unsigned integers: NaN first, then descending.
__device__ __forceinline__ uint32_t logit_key(float v) {
  const uint32_t u = __float_as_uint(v);
  if ((u & 0x7FFFFFFFu) > 0x7F800000u) return 0xFFFFFFFFu;
  return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

// One CTA per token: the logits by warps, the choice by the first warp.
__global__ void __launch_bounds__(kWarps * 32) route_kernel(const RouteArgs a) {
  __shared__ float logits[kMoeMaxExperts];
  griddep_launch_dependents();
  griddep_wait();
  const int t = blockIdx.x, warp = threadIdx.x / 32, lane = threadIdx.x & 31;
  for (int e = warp; e < a.experts; e += kWarps) {
    float acc = 0.0f;
    for (int k = lane; k < a.hidden; k += 32)
      acc = __fmaf_rn(bf16_value(a.router, static_cast<int64_t>(e) * a.hidden + k),
                      bf16_value(a.x, t * a.ld_x + k), acc);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) acc += __shfl_xor_sync(0xFFFFFFFFu, acc, m);
    if (lane == 0) logits[e] = a.bias ? acc + a.bias[e] : acc;
  }
  __syncthreads();
  if (warp != 0) return;
  float chosen[kMoeMaxTopK];
  int ids[kMoeMaxTopK];
  uint32_t taken = 0;  // bit i: this lane's i-th logit is taken
  for (int j = 0; j < a.top_k; ++j) {
    uint32_t best = 0, at = 0xFFFFFFFFu;
    for (int e = lane, i = 0; e < a.experts; e += 32, ++i) {
      const uint32_t key = logit_key(logits[e]);
      if (!((taken >> i) & 1u) && key > best) best = key, at = e;
    }
    const uint32_t top = __reduce_max_sync(0xFFFFFFFFu, best);
    const uint32_t id = __reduce_min_sync(0xFFFFFFFFu, best == top ? at : 0xFFFFFFFFu);
    const bool none = top <= logit_key(-INFINITY);
    ids[j] = none ? -1 : static_cast<int>(id);
    chosen[j] = none ? -INFINITY : logits[id];
    if (!none && (id & 31u) == lane) taken |= 1u << (id / 32);
  }
  float sum = 0.0f;
  if (a.normalize) {
    for (int j = 0; j < a.top_k; ++j) sum += ids[j] < 0 ? 0.0f : expf(chosen[j] - chosen[0]);
  } else {
    for (int e = lane; e < a.experts; e += 32) sum += expf(logits[e] - chosen[0]);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) sum += __shfl_xor_sync(0xFFFFFFFFu, sum, m);
  }
  if (lane < a.top_k) {
    int id = -1;
    float l = 0.0f;
    for (int j = 0; j < a.top_k; ++j)
      if (j == lane) id = ids[j], l = chosen[j];
    a.ids[t * a.top_k + lane] = id;
    a.weights[t * a.top_k + lane] = id < 0 ? 0.0f : expf(l - chosen[0]) / sum;
  }
}

// ---------------------------------------------------------------- the experts

struct MoeParams {
  MoeArgs a;
  few::Split split;
  int tiles;        // row tiles of a group
  int group;        // pairs of a group at most
  int groups_at;    // of the groups in shared memory, after the walk's part
};

// UP: tiles of 16 MT / 2 gate rows and as many up rows of `inter`, h as output.
// Else: 16 MT rows of `hidden`, z as output.  Items: group-major, so that a CTA's
// consecutive items share their activations.
template <int FMT, int MT, int W, bool UP>
struct ExpertPolicy {
  static constexpr int kRows = UP ? 8 * MT : 16 * MT;  // output rows of a warp
  static constexpr int kSegs = UP ? 2 : 1;
  const MoeParams &p;
  const CUtensorMap *map0, *map1;
  char *smem;  // the walk's part: scratch before its first copy
  Groups g;

  __device__ int rows() const { return UP ? p.a.inter : p.a.hidden; }
  __device__ int length() const { return UP ? p.a.hidden : p.a.inter; }

  __device__ void start(int &item, int &end) {
    griddep_wait();
    g = make_groups<W>(smem + p.groups_at, smem, p.a.ids, p.a.tokens * p.a.top_k, p.a.experts, p.group,
                    p.a.status);
    const int64_t items = static_cast<int64_t>(g.count) * p.tiles;
    item = static_cast<int>(items * blockIdx.x / gridDim.x);
    end = static_cast<int>(items * (blockIdx.x + 1) / gridDim.x);
    fence_proxy_async_smem();  // the scratch is overwritten by copies
    __syncthreads();
  }
  __device__ int group(int item) const { return item / p.tiles; }
  __device__ int count(int item) const { return g.size[item / p.tiles]; }
  __device__ int pair(int item, int i) const { return g.list[g.begin[item / p.tiles] + i]; }
  __device__ int64_t row_off(int item, int i) const {
    const int q = pair(item, i);
    return UP ? (q / p.a.top_k) * p.a.ld_x : static_cast<int64_t>(q) * p.a.inter;
  }
  __device__ void runs(int item, int wr, few::Run (&r)[kSegs]) const {
    const int e = g.expert[item / p.tiles];
    const int row = (item % p.tiles * p.split.rows_w + wr) * kRows;
    const int64_t blocks = length() / (FMT == 0 ? 32 : 16);
    const int64_t scale_bytes = (rows() + 127ll) / 128 * ((blocks + 3) / 4) * 512;
    // a tile past the last row reads rows of the next expert or zeros, and is dropped
    const int code_row = e * rows() + min(row, rows());
    const int in = min(row, (rows() - 1) / kRows * kRows);
    const FewMatrix &m0 = UP ? p.a.gate : p.a.down;
    r[0] = few::Run{map0, code_row, m0.scales + e * scale_bytes, in, scale_bytes};
    if constexpr (UP) r[1] = few::Run{map1, code_row, p.a.up.scales + e * scale_bytes, in, scale_bytes};
  }
  __device__ void put(int item, int wr, int m, int n, int lane, const float4 (&v)[kSegs]) const {
    const int e = g.expert[item / p.tiles], n_tokens = count(item);
    const float a0 = FMT == 1 ? (UP ? p.a.gate.ts : p.a.down.ts)[e] : 1.0f;
    float f[4] = {v[0].x * a0, v[0].y * a0, v[0].z * a0, v[0].w * a0};
    if constexpr (UP) {
      const float a1 = FMT == 1 ? p.a.up.ts[e] : 1.0f;
      const float up[4] = {v[1].x * a1, v[1].y * a1, v[1].z * a1, v[1].w * a1};
#pragma unroll
      for (int i = 0; i < 4; i += 2) {
        float2 act;
        if (p.a.gelu)
          act = gelu_f32x2(make_float2(f[i], f[i + 1]));
        else
          act = make_float2(f[i] / (1.0f + expf(-f[i])), f[i + 1] / (1.0f + expf(-f[i + 1])));
        f[i] = act.x * up[i];
        f[i + 1] = act.y * up[i + 1];
      }
    }
    const int row0 = (item % p.tiles * p.split.rows_w + wr) * kRows + m * 16 + (lane >> 2);
    const int col0 = n * 8 + (lane & 3) * 2;
    const int64_t extent = static_cast<int64_t>(p.a.tokens) * p.a.top_k * rows();
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int row = row0 + (i >> 1) * 8, col = col0 + (i & 1);
      if (row >= rows() || col >= n_tokens) continue;
      const int64_t o = static_cast<int64_t>(pair(item, col)) * rows() + row;
      if (in_bounds(o, 1, extent, p.a.status)) (UP ? p.a.h : p.a.z)[o] = f[i];
    }
  }
};

template <int FMT, int MT, int NT, int W, int S, bool UP>
__global__ void __launch_bounds__(W * 32, 1)
    expert_kernel(const __grid_constant__ CUtensorMap map0, const __grid_constant__ CUtensorMap map1,
                  const __grid_constant__ MoeParams p) {
  extern __shared__ __align__(1024) char smem[];
  griddep_launch_dependents();
  if (threadIdx.x == 0) {
    prefetch_tmap(&map0);
    if (UP) prefetch_tmap(&map1);
  }
  ExpertPolicy<FMT, MT, W, UP> policy{p, &map0, &map1, smem, {}};
  const MoeArgs &a = p.a;
  if constexpr (UP)
    few::walk<FMT, MT, NT, 2, W, S, uint16_t>(smem, policy, a.x,
                                              (a.tokens - 1) * a.ld_x + a.hidden, a.hidden, p.split,
                                              a.status);
  else
    few::walk<FMT, MT, NT, 1, W, S, float>(smem, policy, a.h,
                                           static_cast<int64_t>(a.tokens) * a.top_k * a.inter,
                                           a.inter, p.split, a.status);
}

// y[t] = sum_j w_tj z[t, j], in the order of the slots.
__global__ void __launch_bounds__(256) combine_kernel(const MoeArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int t = blockIdx.y, c = (blockIdx.x * 256 + threadIdx.x) * 2;
  if (c >= a.hidden) return;
  float y0 = 0.0f, y1 = 0.0f;
  for (int j = 0; j < a.top_k; ++j) {
    const int p = t * a.top_k + j, e = a.ids[p];
    if (e < 0 || e >= a.experts) continue;
    const float w = a.weights[p];
    const int64_t o = static_cast<int64_t>(p) * a.hidden + c;
    if (!in_bounds(o, 2, static_cast<int64_t>(a.tokens) * a.top_k * a.hidden, a.status)) continue;
    const float2 z = *reinterpret_cast<const float2 *>(a.z + o);
    y0 = __fmaf_rn(w, z.x, y0);
    y1 = __fmaf_rn(w, z.y, y1);
  }
  const int64_t o = t * a.ld_y + c;
  if (!in_bounds(o, 2, (a.tokens - 1) * a.ld_y + a.hidden, a.status)) return;
  uint16_t *y = static_cast<uint16_t *>(a.y) + o;
  y[0] = bf16_bits(y0);
  y[1] = bf16_bits(y1);
}

template <int FMT, int MT, int NT, int W, int S, bool UP>
cudaError_t launch_product(const MoeArgs &a, cudaStream_t s) {
  using L = few::Layout<FMT, MT, NT, UP ? 2 : 1, W, S>;
  const auto kernel = expert_kernel<FMT, MT, NT, W, S, UP>;
  const void *func = reinterpret_cast<const void *>(kernel);
  if (!kernel_setup_get(func, nullptr)) {
    const cudaError_t e =
        cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, few::kMaxSmem);
    if (e != cudaSuccess) return e;
    kernel_setup_put(func, 0);
  }
  const int k = UP ? a.hidden : a.inter, rows = UP ? a.inter : a.hidden;
  const int pairs = a.tokens * a.top_k;
  const int group = pairs < 8 * NT ? pairs : 8 * NT;
  const int most = a.experts < pairs ? a.experts : pairs;  // experts with a pair
  const int box = UP ? 8 * MT : 16 * MT;                   // output rows of a warp
  const int64_t row_tiles = (rows + box - 1) / box, all = row_tiles * (most + pairs / (8 * NT));
  const int64_t each = (all + a.num_sms - 1) / a.num_sms;
  MoeParams p{a, L::split(group, (k + few::kStageK - 1) / few::kStageK, getenv("LEAST") ? atoi(getenv("LEAST")) : 1,
                          static_cast<int>(each < 64 ? each : 64),
                          few::kMaxSmem - Groups::bytes(pairs)), 0, 8 * NT, 0};
  p.tiles = static_cast<int>((row_tiles + p.split.rows_w - 1) / p.split.rows_w);
  p.groups_at = L::total(group, p.split);
  CUtensorMap map0, map1;
  const int64_t stacked = static_cast<int64_t>(a.experts) * rows;
  if (!encode_few_map(&map0, UP ? a.gate.codes : a.down.codes, stacked, k, box) ||
      !encode_few_map(&map1, UP ? a.up.codes : a.down.codes, stacked, k, box))
    return cudaErrorInvalidValue;
  const int64_t items = static_cast<int64_t>(most + pairs / (8 * NT)) * p.tiles;
  const int grid = items < a.num_sms ? static_cast<int>(items) : a.num_sms;
  return launch_pdl(kernel, dim3(grid), dim3(W * 32), p.groups_at + Groups::bytes(pairs), s, map0,
                    map1, p);
}

template <int FMT, int NT, int W, int S>
cudaError_t launch_experts(const MoeArgs &a, cudaStream_t s) {
  cudaError_t e = launch_product<FMT, 4, NT, W, S, true>(a, s);
  if (e == cudaSuccess) e = launch_product<FMT, 4, NT, W, S, false>(a, s);
  if (e == cudaSuccess)
    e = launch_pdl(combine_kernel, dim3((a.hidden + 511) / 512, a.tokens), dim3(256), 0, s, a);
  return e;
}

}  // namespace

cudaError_t launch_moe_route(const RouteArgs &a, cudaStream_t s) {
  return launch_pdl(route_kernel, dim3(a.tokens), dim3(kWarps * 32), 0, s, a);
}

cudaError_t launch_moe_experts(const MoeArgs &a, cudaStream_t s) {
  if (!getenv("OLD")) {
    const cudaError_t e = launch_expert_products(a, s);
    if (e != cudaSuccess) return e;
    return launch_pdl(combine_kernel, dim3((a.hidden + 511) / 512, a.tokens), dim3(256), 0, s, a);
  }
  if (a.tokens <= 8) return a.fmt == 0 ? launch_experts<0, 1, 8, 3>(a, s) : launch_experts<1, 1, 8, 3>(a, s);
  return a.fmt == 0 ? launch_experts<0, 2, 8, 2>(a, s) : launch_experts<1, 2, 8, 2>(a, s);
}

}  // namespace mx
