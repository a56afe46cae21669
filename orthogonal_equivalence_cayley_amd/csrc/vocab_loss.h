// What the kernels of the vocabulary's cross entropy share (k_vocab_loss.hip,
// k_vocab_loss_pipe.hip): the parts of their epilogues.
#pragma once

#include "linear_common.h"

namespace poetx {
namespace vocab {

// exp of fp32 logits by the library's function, of bf16 products by the hardware's (its
// result is summed beside thousands of others, or rounded to bf16)
template <bool F32>
__device__ __forceinline__ float exp_of(float x) {
  if constexpr (F32) return expf(x);
  else return __expf(x);
}

// What the backward needs of a row
struct Row {
  float lse, factor;
  long long target;   // -1: none (ignored, factor 0)
};
__device__ __forceinline__ Row token_of(const VocabArgs& a, long long t) {
  const long long target = a.target[t];
  if (target == a.ignore) return Row{0.0f, 0.0f, -1};
  // a target outside the vocabulary has no loss: its gradients are NaN
  const bool bad = target < 0 || target >= a.V;
  return Row{a.lse[t], bad ? __builtin_nanf("") : a.g_each ? a.g[t] : 1.0f, target};
}
// dL/dz of column v, but for a factor that all rows share (a.g without g_each)
template <bool F32>
__device__ __forceinline__ float grad_of(const Row& r, float z, long long v) {
  // an ignored row is zero whatever its logits are
  if (r.target < 0 && r.factor == 0.0f) return 0.0f;
  const float p = exp_of<F32>(z - r.lse);
  return (v == r.target ? p - 1.0f : p) * r.factor;
}

}  // namespace vocab
}  // namespace poetx
