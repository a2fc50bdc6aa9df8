// mx_linear_bf16: a few BF16 rows times an FP4 weight.
#include "few_tokens.cuh"

namespace mx {
namespace {

constexpr int kMaxSmem = 227 * 1024;

struct LinearParams {
  LinearArgs a;
  int tiles;   // row tiles of 16 MT rows
  int stages;  // ring depth of a warp
};

// Persistent over row tiles: tile blockIdx.x, + gridDim.x, ...  Each of the W
// warps takes its share of K in every tile.
template <int FMT, int MT, int NT, int W, int S>
__global__ void __launch_bounds__(W * 32, 1) linear_kernel(const LinearParams p) {
  extern __shared__ __align__(128) char smem[];
  constexpr int R = 16 * MT, kUnits = MT * NT * 32;
  const LinearArgs &a = p.a;
  griddep_launch_dependents();
  const int warp = threadIdx.x >> 5;
  const int k = static_cast<int>(a.k), n = static_cast<int>(a.n);
  const int stage_size = few::stage_bytes<FMT, MT, uint16_t>(a.tokens);
  float4 *red = reinterpret_cast<float4 *>(smem);
  const uint32_t ring = smem_u32(smem) + W * kUnits * 16 + warp * S * stage_size;
  const int all = (k + few::kStageK - 1) / few::kStageK;
  const int s_begin = all * warp / W, s_end = all * (warp + 1) / W;
  const int64_t blocks = k / (FMT == 0 ? 32 : 16);
  const few::Rows m0{a.w.codes, a.w.scales, 0, 0, a.n * (a.k / 2),
                     (a.n + 127) / 128 * ((blocks + 3) / 4) * 512};
  const few::Rows rows[2] = {m0, m0};
  const int64_t x_extent = ((a.tokens - 1) * a.ld_x + a.k) * 2;

  // the copies' place: tile and stage, ahead of the product's
  int ptile = blockIdx.x, ps = s_begin, pslot = 0;
  const auto issue = [&]() {
    if (s_begin < s_end && ptile < p.tiles) {
      const uint32_t dst = ring + pslot * stage_size;
      const int first[2] = {ptile * R, ptile * R + R / 2};
      few::load_weights<FMT, MT>(dst, rows, first, n, k, ps, a.status);
      few::load_x<uint16_t>(dst + R * (64 + (FMT == 0 ? 4 : 8)), a.x, x_extent, a.tokens, k, ps,
                            [&](int r) { return r * a.ld_x; }, a.status);
      if (++ps == s_end) ps = s_begin, ptile += gridDim.x;
      if (++pslot == S) pslot = 0;
    }
    few::cp_async_commit();
  };

  griddep_wait();
#pragma unroll
  for (int i = 0; i < S - 1; ++i) issue();
  const float alpha = FMT == 1 ? *a.w.ts : 1.0f;
  int slot = 0;
  for (int tile = blockIdx.x; tile < p.tiles; tile += gridDim.x) {
    float total[MT][NT][4] = {};
    for (int s = s_begin; s < s_end; ++s) {
      few::cp_async_wait<S - 2>();
      __syncwarp();
      issue();
      few::stage_product<FMT, MT, NT, uint16_t>(ring + slot * stage_size, a.tokens, total);
      if (++slot == S) slot = 0;
    }
    few::write_totals<MT, NT>(red, warp, total);
    __syncthreads();
    for (int u = threadIdx.x; u < kUnits; u += W * 32) {
      const float4 v = few::sum_totals<kUnits>(red, W, u);
      const int lane = u & 31, mn = u >> 5;
      const int row0 = tile * R + (mn / NT) * 16 + (lane >> 2), col0 = (mn % NT) * 8 + (lane & 3) * 2;
      const float f[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int row = row0 + (i >> 1) * 8, col = col0 + (i & 1);
        const int64_t at = col * a.ld_y + row;
        if (row >= n || col >= a.tokens ||
            !in_bounds(at, 1, (a.tokens - 1) * a.ld_y + a.n, a.status))
          continue;
        float y = FMT == 1 ? f[i] * alpha : f[i];
        if (a.beta != 0.0f)
          y = __fmaf_rn(a.beta, a.out_fp32 ? static_cast<const float *>(a.y)[at] : bf16_value(a.y, at),
                        y);
        if (a.bias != nullptr) y = __fadd_rn(y, a.bias[row]);
        if (a.gelu) y = gelu_f32x2(make_float2(y, y)).x;
        if (a.out_fp32)
          static_cast<float *>(a.y)[at] = y;
        else
          static_cast<uint16_t *>(a.y)[at] = bf16_bits(y);
      }
    }
    __syncthreads();
  }
}

template <int FMT, int MT, int NT, int W, int S>
cudaError_t launch(const LinearArgs &a, cudaStream_t s) {
  const auto kernel = linear_kernel<FMT, MT, NT, W, S>;
  const void *func = reinterpret_cast<const void *>(kernel);
  if (!kernel_setup_get(func, nullptr)) {
    const cudaError_t e =
        cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, kMaxSmem);
    if (e != cudaSuccess) return e;
    kernel_setup_put(func, 0);
  }
  LinearParams p{a, static_cast<int>((a.n + 16 * MT - 1) / (16 * MT)), S};
  const size_t smem = W * MT * NT * 512 +
                      static_cast<size_t>(W) * S * few::stage_bytes<FMT, MT, uint16_t>(a.tokens);
  const int grid = p.tiles < a.num_sms ? p.tiles : a.num_sms;
  return launch_pdl(kernel, dim3(grid), dim3(W * 32), smem, s, p);
}

template <int FMT>
cudaError_t launch_fmt(const LinearArgs &a, cudaStream_t s) {
  const bool small = a.n < 64 * static_cast<int64_t>(a.num_sms);
  if (a.tokens <= 8) return small ? launch<FMT, 2, 1, 8, 4>(a, s) : launch<FMT, 4, 1, 8, 3>(a, s);
  if (a.tokens <= 16) return small ? launch<FMT, 2, 2, 8, 3>(a, s) : launch<FMT, 4, 2, 8, 2>(a, s);
  return launch<FMT, 2, 4, 6, 2>(a, s);
}

}  // namespace

cudaError_t launch_linear(const LinearArgs &a, cudaStream_t s) {
  return a.fmt == 0 ? launch_fmt<0>(a, s) : launch_fmt<1>(a, s);
}

}  // namespace mx
