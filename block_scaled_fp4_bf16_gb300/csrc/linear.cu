// mx_linear_bf16: a few BF16 rows times an FP4 weight.
#include <cstdlib>
#include "few_tokens.cuh"

namespace mx {
namespace {


struct LinearParams {
  LinearArgs a;
  few::Split split;
  int items;  // of 16 kRowTiles split.rows_w rows
};

// Items are row tiles; all have the same tokens.
template <int FMT, int NT, int kRowTiles>
struct LinearPolicy {
  static constexpr int kRows = 16 * kRowTiles;
  const LinearParams &p;
  const CUtensorMap *map;
  int64_t scale_end;

  __device__ void start(int &item, int &end) const {
    item = static_cast<int>(static_cast<int64_t>(p.items) * blockIdx.x / gridDim.x);
    end = static_cast<int>(static_cast<int64_t>(p.items) * (blockIdx.x + 1) / gridDim.x);
    griddep_wait();
  }
  __device__ int group(int) const { return 0; }
  __device__ int count(int) const { return p.a.tokens; }
  __device__ int64_t row_off(int, int i) const { return i * p.a.ld_x; }
  __device__ void runs(int item, int wr, few::Run (&r)[1]) const {
    const int64_t row = (static_cast<int64_t>(item) * p.split.rows_w + wr) * kRows;
    // a tile past the last row gets zeros, and reads (and drops) the last one's scales
    r[0] = few::Run{map, static_cast<int>(min(row, p.a.n)), p.a.w.scales,
                    static_cast<int>(min(row, (p.a.n - 1) / kRows * kRows)), scale_end};
  }
  __device__ void put(int item, int wr, int m, int n, int lane, const float4 (&v)[1]) const {
    const LinearArgs &a = p.a;
    const float alpha = FMT == 1 ? *a.w.ts : 1.0f;
    const int64_t row0 =
        (static_cast<int64_t>(item) * p.split.rows_w + wr) * kRows + m * 16 + (lane >> 2);
    const int col0 = n * 8 + (lane & 3) * 2;
    const float f[4] = {v[0].x, v[0].y, v[0].z, v[0].w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t row = row0 + (i >> 1) * 8;
      const int col = col0 + (i & 1);
      const int64_t o = col * a.ld_y + row;
      if (row >= a.n || col >= a.tokens ||
          !in_bounds(o, 1, (a.tokens - 1) * a.ld_y + a.n, a.status))
        continue;
      float y = FMT == 1 ? f[i] * alpha : f[i];
      if (a.beta != 0.0f)
        y = __fmaf_rn(a.beta, a.out_fp32 ? static_cast<const float *>(a.y)[o] : bf16_value(a.y, o), y);
      if (a.bias != nullptr) y = __fadd_rn(y, a.bias[row]);
      if (a.gelu) y = gelu_f32x2(make_float2(y, y)).x;
      if (a.out_fp32)
        static_cast<float *>(a.y)[o] = y;
      else
        static_cast<uint16_t *>(a.y)[o] = bf16_bits(y);
    }
  }
};

template <int FMT, int NT, int kRowTiles, int W, int S>
__global__ void __launch_bounds__(W * 32, 1)
    linear_kernel(const __grid_constant__ CUtensorMap map, const __grid_constant__ LinearParams p) {
  extern __shared__ __align__(1024) char smem[];
  const LinearArgs &a = p.a;
  griddep_launch_dependents();
  if (threadIdx.x == 0) prefetch_tmap(&map);
  const int64_t blocks = a.k / (FMT == 0 ? 32 : 16);
  LinearPolicy<FMT, NT, kRowTiles> policy{p, &map, (a.n + 127) / 128 * ((blocks + 3) / 4) * 512};
  few::walk<FMT, kRowTiles, NT, 1, W, S, uint16_t>(smem, policy, a.x,
                                                   (a.tokens - 1) * a.ld_x + a.k,
                                                   static_cast<int>(a.k), p.split, a.status);
}

template <int FMT, int NT, int kRowTiles, int W, int S>
cudaError_t launch(const LinearArgs &a, cudaStream_t s) {
  using L = few::Layout<FMT, kRowTiles, NT, 1, W, S>;
  const auto kernel = linear_kernel<FMT, NT, kRowTiles, W, S>;
  const void *func = reinterpret_cast<const void *>(kernel);
  if (!kernel_setup_get(func, nullptr)) {
    const cudaError_t e =
        cudaFuncSetAttribute(func, cudaFuncAttributeMaxDynamicSharedMemorySize, few::kMaxSmem);
    if (e != cudaSuccess) return e;
    kernel_setup_put(func, 0);
  }
  constexpr int kRows = 16 * kRowTiles;
  const int stages = static_cast<int>((a.k + few::kStageK - 1) / few::kStageK);
  const int64_t row_tiles = (a.n + kRows - 1) / kRows;
  const int64_t each = (row_tiles + a.num_sms - 1) / a.num_sms;
  LinearParams p{a, L::split(a.tokens, stages, getenv("LEAST") ? atoi(getenv("LEAST")) : 1, static_cast<int>(each < 64 ? each : 64),
                             few::kMaxSmem), 0};
  const int64_t rows = kRows * p.split.rows_w;
  p.items = static_cast<int>((a.n + rows - 1) / rows);
  CUtensorMap map;
  if (!encode_few_map(&map, a.w.codes, a.n, a.k, kRows)) return cudaErrorInvalidValue;
  const int grid = p.items < a.num_sms ? p.items : a.num_sms;
  return launch_pdl(kernel, dim3(grid), dim3(W * 32), L::total(a.tokens, p.split), s, map, p);
}

template <int FMT>
cudaError_t launch_fmt(const LinearArgs &a, cudaStream_t s) {
  static const int v = getenv("V") ? atoi(getenv("V")) : 0;
  if (a.tokens <= 8) {
    if (v == 1) return launch<FMT, 1, 2, 8, 4>(a, s);
    if (v == 2) return launch<FMT, 1, 2, 16, 3>(a, s);
    if (v == 3) return launch<FMT, 1, 4, 8, 4>(a, s);
    return launch<FMT, 1, 4, 8, 3>(a, s);
  }
  if (a.tokens <= 16) {
    if (v == 1) return launch<FMT, 2, 2, 8, 3>(a, s);
    if (v == 2) return launch<FMT, 2, 2, 16, 2>(a, s);
    if (v == 3) return launch<FMT, 2, 4, 8, 3>(a, s);
    return launch<FMT, 2, 4, 8, 2>(a, s);
  }
  if (v == 1) return launch<FMT, 4, 2, 8, 3>(a, s);
  return launch<FMT, 4, 2, 8, 2>(a, s);
}

}  // namespace

cudaError_t launch_linear(const LinearArgs &a, cudaStream_t s) {
  return a.fmt == 0 ? launch_fmt<0>(a, s) : launch_fmt<1>(a, s);
}

}  // namespace mx
