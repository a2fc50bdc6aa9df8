// The rest of a decoding step (qk_rope.cu, kv_append.cu, attention.cu, sample.cu):
// arguments and launchers.
#pragma once

#include "mx_internal.h"

namespace mx {

// Bit of the device status word set when a page, length or row number in device memory was
// out of range (and was skipped).
constexpr uint32_t kStatusIndexBit = 4u;

// Queries or keys of a layer: rows of heads, with the norm's weight.
struct Heads {
  const uint16_t *x;   // BF16 [tokens, heads, head_dim], row stride ld
  int64_t ld;
  const uint16_t *dy;  // backward: the outputs' gradients
  int64_t ld_dy;
  uint16_t *y;         // out: rotated rows, or the inputs' gradients
  int64_t ld_y;
  const uint16_t *weight;  // BF16 [head_dim] or null
  float *dweight;      // backward: FP32 [head_dim] or null
  int heads;
};

struct RopeArgs {
  Heads part[2];       // queries, keys
  int64_t tokens;
  const int32_t *positions;
  const float *inv_freq;
  int head_dim, rotary_dim, interleaved;
  float eps;
  float *partials;     // backward: [kRopeBackCtas][2][head_dim] sums of the CTAs
  int num_sms;
  uint32_t *status;
};
constexpr int kRopeMaxDim = 256;
constexpr int kRopeBackCtas = 320;  // most CTAs of the backward kernel
// Slices of a token's groups of heads: those with which the busiest warp has the least to do,
// an item's angles counted as half a group (8192 tokens of 18 groups on 2432 warps: whole
// tokens leave most warps with three and some with four, 57 us; halves 49).  Of the lengths that make
// as many slices only the least counts, so that the most heads take some 500 steps, not 65535.
inline void rope_slices(int64_t tokens, int groups, int64_t warps, int *slices, int *per_slice) {
  *slices = 1;
  *per_slice = groups;
  int64_t least = INT64_MAX;
  for (int p = groups; p >= 1; --p) {
    const int n = (groups + p - 1) / p;
    if (n > 1 && tokens * n >= (int64_t(1) << 31)) break;  // (the kernel divides 32-bit numbers)
    p = (groups + n - 1) / n;
    const int64_t cost = (tokens * n + warps - 1) / warps * (2 * p + 1);
    if (cost < least) least = cost, *slices = n, *per_slice = p;
  }
}
cudaError_t launch_qk_rope(const RopeArgs &a, cudaStream_t s);
cudaError_t launch_qk_rope_backward(const RopeArgs &a, cudaStream_t s);

constexpr int kCacheBlock = 32;  // tokens of a scale

// The cache as the kernels see it.
struct CacheArgs {
  uint8_t *codes[2];   // keys, values
  uint8_t *scales[2];
  int64_t pages;
  int page_tokens, heads, head_dim;
  const int32_t *table;    // [sequences, max_pages]
  int64_t max_pages;
  const int32_t *lengths;
  int sequences;
  uint32_t *status;
};

struct AppendArgs {
  CacheArgs c;
  const uint16_t *x[2];    // new keys, values
  int64_t ld[2];
  int64_t tokens;
  const int32_t *starts;   // null: each sequence has tokens / sequences
};
cudaError_t launch_kv_append(const AppendArgs &a, cudaStream_t s);

constexpr int kAttentionMaxQuery = 16;
constexpr int kAttentionMaxSequences = 4096;
constexpr int kAttentionMaxGroup = 64;
struct AttentionArgs {
  CacheArgs c;
  const uint16_t *q;
  int64_t ld_q;
  int q_heads, q_tokens;
  float scale;
  int64_t window;          // 0: none
  uint16_t *out;
  int64_t ld_out;
  float *lse;              // or null
  void *workspace;
  int num_sms;
};
// rows: of a (sequence, key head)
size_t attention_workspace_bytes(int64_t rows, int head_dim);
cudaError_t launch_attention(const AttentionArgs &a, cudaStream_t s);

constexpr int kSampleMaxVocab = 262144;
struct SampleArgs {
  const void *logits;
  int64_t ld;
  int rows, vocab, fp32;
  const float *temperature;
  const int32_t *top_k;
  const float *top_p, *min_p, *uniform;
  int32_t *ids;
  float *probability;
  int num_sms;
  uint32_t *status;
};
cudaError_t launch_sample(const SampleArgs &a, cudaStream_t s);
constexpr int kSampleMaxCtas = 16, kSamplePortableCtas = 8;
// The CTAs of a row: at least 4096 logits each; 16 (more than may be taken for granted: `most` is 8
// where the context has no room for such a cluster) for few rows, and where rows fill the GPU as few as hold
// a row in 16384 logits each (what a CTA does besides its logits takes 8 us; 256 x 32000: eight
// a row 73 us, two 41).
inline int sample_ctas(int64_t rows, int vocab, int num_sms, int most) {
  int ctas = 1;
  while (ctas < kSamplePortableCtas && ctas * 4096 < vocab) ctas *= 2;
  if (rows * ctas * 2 <= num_sms && ctas == kSamplePortableCtas && vocab > 32768) ctas = most;
  while (ctas > 1 && rows * ctas > 2 * num_sms && (vocab + ctas / 2 - 1) / (ctas / 2) <= 16384) ctas /= 2;
  return ctas;
}

}  // namespace mx
