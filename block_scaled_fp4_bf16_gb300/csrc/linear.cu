// mx_linear_bf16: a few BF16 rows times an FP4 weight.
#include "few_tokens.cuh"

namespace mx {
namespace {

constexpr int kWarps = 8;

template <int FMT, int OUT_F32>
__global__ void __launch_bounds__(kWarps * 32) linear_kernel(const LinearArgs a) {
  griddep_launch_dependents();
  griddep_wait();
  const int64_t row = static_cast<int64_t>(blockIdx.x) * kWarps + threadIdx.x / 32;
  if (row >= a.n) return;
  const float alpha = FMT == 1 ? *a.w.ts : 1.0f;
  for (int t0 = 0; t0 < a.tokens; t0 += 8) {
    float acc[8];
    warp_row_dot<FMT, 8>(a.w.codes, a.w.scales, row, a.k, a.tokens - t0,
                         [&](int i, int64_t k) { return bf16_value(a.x, (t0 + i) * a.ld_x + k); },
                         acc);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      if (t0 + i < a.tokens && (threadIdx.x & 31) == 0) {
        const int64_t at = (t0 + i) * a.ld_y + row;
        float v = acc[i] * alpha;
        if (a.beta != 0.0f)
          v = __fmaf_rn(a.beta, OUT_F32 ? static_cast<const float *>(a.y)[at] : bf16_value(a.y, at), v);
        if (a.bias) v = __fadd_rn(v, a.bias[row]);
        if (a.gelu) v = gelu_f32x2(make_float2(v, v)).x;
        if (OUT_F32)
          static_cast<float *>(a.y)[at] = v;
        else
          static_cast<uint16_t *>(a.y)[at] = bf16_bits(v);
      }
    }
  }
}

}  // namespace

cudaError_t launch_linear(const LinearArgs &a, cudaStream_t s) {
  const dim3 grid(static_cast<unsigned>((a.n + kWarps - 1) / kWarps)), block(kWarps * 32);
  if (a.fmt == 0)
    return a.out_fp32 ? launch_pdl(linear_kernel<0, 1>, grid, block, 0, s, a)
                      : launch_pdl(linear_kernel<0, 0>, grid, block, 0, s, a);
  return a.out_fp32 ? launch_pdl(linear_kernel<1, 1>, grid, block, 0, s, a)
                    : launch_pdl(linear_kernel<1, 0>, grid, block, 0, s, a);
}

}  // namespace mx
