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

// What a row's loss is made of, besides its logp.
struct PolicyScalars {
  float weight, advantage, old_logp, ref_logp;
};

__device__ __forceinline__ PolicyScalars policy_scalars(const PolicyRows& p, int64_t t, int doc) {
  return {__ldcg(p.doc_weight + doc), __ldg(p.advantages + (p.per_token ? t : (int64_t)doc)),
          __ldg(p.old_logp + t), p.ref_logp != nullptr ? __ldg(p.ref_logp + t) : 0.f};
}

__device__ __forceinline__ PolicyRow policy_row(const PolicyRows& p, const PolicyScalars& v, float logp) {
  const float w = v.weight, adv = v.advantage;
  const float rho = expf(logp - v.old_logp);
  const bool cut = (adv > 0.f && rho > 1.f + p.clip_high) || (adv < 0.f && rho < 1.f - p.clip_low);
  PolicyRow r;
  const float bound = adv > 0.f ? 1.f + p.clip_high : 1.f - p.clip_low;
  r.surrogate = -adv * (cut ? bound : rho);
  r.grad = cut ? 0.f : -adv * rho;
  r.clipped = cut ? w : 0.f;
  r.kl = 0.f;
  if (p.ref_logp != nullptr) {
    const float z = v.ref_logp - logp, e = expm1f(z);
    r.kl = w * (e - z);
    r.grad = fmaf(-p.kl_coef, e, r.grad);
  }
  r.surrogate *= w;
  r.grad *= w;
  return r;
}

}  // namespace nsp

#endif  // __CUDACC__
