// A router's scores between the logits and the gates, for the layer's router and
// the one for a few tokens: fp32's sigmoid is 0 below -88, its shares are not.
#pragma once

#include "moe_common.hpp"

namespace moe {

// A score as it is kept until the gates are formed: s = sigmoid(z), or the logit itself
// (negative) where fp32's s is 0.
__device__ __forceinline__ float kept_score(float z) {
  const float s = sigmoid_f32(z);
  return s == 0.f ? z : s;
}
__device__ __forceinline__ float score_of(float kept) { return kept < 0.f ? 0.f : kept; }

// The gate of the k-th selected score in lane k < top_k, of a wave; `sum` of those scores.
// Where s is 0 for some and tiny for all, s = e^z to 2^-100 and the gates go by the logits,
// from the largest on: of s they would be 0 / 0, or 0 beside a score no larger.
// `score`: s, for the backward, which needs s / sum and 1 - s.  There the former is the
// gate and the latter 1, so any multiple of the scores serves that fp32 holds: 2^-30 gate.
struct Selected {
  float gate, score;
};
__device__ __forceinline__ Selected selected(float kept, float sum, int k, int top_k) {
  const bool mine = k < top_k;
  if (!(sum < 0x1p-100f) || __ballot(mine && kept < 0.f) == 0) return {score_of(kept) / sum, score_of(kept)};
  const float z = !mine ? -INFINITY : kept < 0.f ? kept : logf(kept);
  float top = z;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
  const float p = mine ? expf(z - top) : 0.f;
  float total = p;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1) total += __shfl_xor(total, off);
  return {p / total, p / total * 0x1p-30f};
}

}  // namespace moe
