// The products of a few tokens (linear.cu, linear_mma.cu, moe.cu, moe_mma.cu): arguments
// and launchers.
#pragma once

#include "mx_internal.h"

namespace mx {

// A stack of FP4 matrices [rows, k]: packed codes and tcgen05-order scales of
// each expert one after the other (one matrix for mx_linear_bf16).
struct FewMatrix {
  const uint8_t *codes;
  const uint8_t *scales;
  const float *ts;  // NVFP4: one per matrix; MXFP4: null
};

// Tensor map of a stack of packed code matrices as [rows, k / 2] bytes: boxes of 128
// bytes (256 codes) x box_rows rows, 128-byte swizzle, zeros outside (api.cu).  false
// when it could not be encoded.
bool encode_codes_window_map(CUtensorMap *tm, const void *codes, int64_t rows, int64_t k,
                             int box_rows);

// y[t, n] = epilogue(sum_k x[t, k] W[n, k]) for tokens <= kLinearMaxTokens.
constexpr int kLinearMaxTokens = 32;
struct LinearArgs {
  const void *x;
  int64_t ld_x;
  int tokens;
  int64_t n, k;
  int fmt;  // 0 MXFP4, 1 NVFP4
  FewMatrix w;
  void *y;
  int64_t ld_y;
  int out_fp32;
  const float *bias;
  float beta;
  int gelu;
  int num_sms;
  uint32_t *status;
};
cudaError_t launch_linear(const LinearArgs &a, cudaStream_t s);
// The two kernels for weights of many bytes (linear_mma.cu), their workspace, and
// whether they are the faster (linear.cu).
constexpr int kLinearCtas = 160;  // most CTAs of the product (one per SM)
bool linear_mma_better(int64_t tokens, int64_t n, int64_t k);
size_t linear_workspace_bytes(int fmt, int64_t tokens, int64_t n, int64_t k);
cudaError_t launch_linear_mma(const LinearArgs &a, void *workspace, cudaStream_t s);

constexpr int kMoeMaxTokens = 64;
constexpr int kMoeMaxExperts = 512;
constexpr int kMoeMaxTopK = 16;
constexpr int kMoeGroupMax = 16;  // pairs of an expert that a product takes together
struct RouteArgs {
  const void *x;
  int64_t ld_x;
  int tokens, hidden, experts, top_k, normalize;
  const void *router;
  const float *bias;
  int32_t *ids;
  float *weights;
  uint32_t *status;
};
// next: the experts' call that follows (null: none), for which it does launch_moe_prepare.
struct MoeArgs;
cudaError_t launch_moe_route(const RouteArgs &a, const MoeArgs *next, cudaStream_t s);

struct MoeArgs {
  const void *x;
  int64_t ld_x;
  int tokens, top_k, experts, hidden, inter;
  int fmt, gelu;
  const int32_t *ids;
  const float *weights;
  FewMatrix gate, up, down;
  void *y;
  int64_t ld_y;
  int up_parts, down_parts;  // ranges of K of the two products (moe_parts)
  float *h;            // sums of gate and up rows [up_parts][2][tokens * top_k][inter]
  float *z;            // [down_parts][tokens * top_k][hidden]
  uint8_t *image;      // digits of x, then of h (moe_image_bytes)
  float *factors;      // NVFP4: of the rows of x, then of h
  uint32_t *counts;    // moe_counts(tokens * top_k), cleared by the launch before
  int num_sms;
  uint32_t *status;
};
// Bytes of the digits of `rows` rows of k activations.
size_t moe_image_bytes(int64_t rows, int64_t k);
// Grid-wide counts, and those of the groups (moe_mma.cu).
constexpr int moe_counts(int pairs) { return 2 + 2 * pairs; }
// Ranges of K that a product is divided into, and the most for a number of pairs.
int moe_parts(int64_t pairs, int64_t experts, int64_t rows, int64_t k, int num_sms);
constexpr int moe_max_parts(int64_t pairs) { return pairs <= 16 ? 4 : pairs <= 64 ? 2 : 1; }
// Whether the digits of x are made by the launch before the experts' kernel, in the
// order of the tokens: MXFP4 and few tokens (us, so and in that kernel: 4 x 2048 x 1024 of
// 64 27.8 / 29.8, 1 x 8192 x 4096 of 8 29.3 / 32.4; but 8 x 4096 x 2048 76.1 / 71.3, where
// all tokens' digits cost more than a group's, and NVFP4, whose factor takes that launch
// 2 us, 4 x 4096 x 2048 of 8 35.7 / 32.2).
constexpr bool moe_by_token(int fmt, int tokens) { return fmt == 0 && tokens <= 4; }
// Clears a.counts, and makes the digits of x if moe_by_token.
cudaError_t launch_moe_prepare(const MoeArgs &a, cudaStream_t s);
cudaError_t launch_moe_experts(const MoeArgs &a, cudaStream_t s);

}  // namespace mx
