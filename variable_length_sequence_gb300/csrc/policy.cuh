// The policy loss of one row, shared by the kernel over log-probabilities in
// hand and by the one that reads logits.
//
// With rho = exp(logp - old), A the advantage, z = ref - logp:
//   surrogate = -min(rho A, clip(rho, 1 - low, 1 + high) A),
//   kl = exp(z) - z - 1  (not negative, zero where the policies agree),
//   d/dlogp = -rho A (0 where the clip decides) - kl_coef (exp(z) - 1).
#pragma once

#include "train.cuh"

#ifdef __CUDACC__

namespace nsp {

struct PolicyRow {
  float surrogate, kl, clipped, grad;      // grad: of logp, all four times the row's weight
};

__device__ __forceinline__ PolicyRow policy_row(const PolicyRows& p, int64_t t, int doc, float logp) {
  const float w = __ldg(p.doc_weight + doc);
  const float adv = __ldg(p.advantages + (p.per_token ? t : (int64_t)doc));
  const float rho = expf(logp - __ldg(p.old_logp + t));
  const bool cut = (adv > 0.f && rho > 1.f + p.clip_high) || (adv < 0.f && rho < 1.f - p.clip_low);
  PolicyRow r;
  const float bound = adv > 0.f ? 1.f + p.clip_high : 1.f - p.clip_low;
  r.surrogate = -adv * (cut ? bound : rho);
  r.grad = cut ? 0.f : -adv * rho;
  r.clipped = cut ? w : 0.f;
  r.kl = 0.f;
  if (p.ref_logp != nullptr) {
    const float z = __ldg(p.ref_logp + t) - logp, e = expm1f(z);
    r.kl = w * (e - z);
    r.grad = fmaf(-p.kl_coef, e, r.grad);
  }
  r.surrogate *= w;
  r.grad *= w;
  return r;
}

}  // namespace nsp

#endif  // __CUDACC__
