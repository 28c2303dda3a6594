// Log-probability of a given token of every row of logits, and its gradient:
//   x_j = s logit_j,  lse = ln sum_j exp(x_j),  logp = x_y - lse,
//   d logit_j = s g ([j = y] - exp(x_j - lse)),
// g the gradient of logp: given (backward), or the policy loss's own, of the logp
// just computed (the row is then read once for both).  A row without a target
// (y < 0) is not read; its logp, lse and gradient are zero.
#include <cmath>

#include "policy.cuh"

namespace nsp {
namespace {

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;

// m and s of sum exp(x - m): the sum of both ranges'.
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
  const float top = fmaxf(m, m2);
  const float ref = top == -INFINITY ? 0.f : top;
  s = s * expf(m - ref) + s2 * expf(m2 - ref);
  m = top;
}

template <typename T, RowMode MODE>
__global__ void __launch_bounds__(kThreads) row_kernel(const __grid_constant__ RowArgs a) {
  __shared__ float s_m[kWarps], s_s[kWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (MODE == kRowPolicy && status_bad(a.p.hdr)) return;
  for (int64_t t = blockIdx.x; t < a.rows; t += gridDim.x) {
    const int y = __ldg(a.targets + t);
    const T* const x = reinterpret_cast<const T*>(a.logits) + t * a.row_stride;
    T* const dx = reinterpret_cast<T*>(a.dlogits) + t * a.out_stride;
    int doc = 0;
    bool scored = y >= 0;
    if (MODE == kRowPolicy) {
      scored = scored && t < (int64_t)__ldg(a.p.cu + a.p.ndoc);
      if (scored) doc = doc_of(a.p.cu, a.p.ndoc, t);
    }
    if (!scored) {
      if (MODE != kRowForward)
        for (int j = threadIdx.x; j < a.vocab; j += kThreads) st_out(dx + j, 0.f);
      if (MODE != kRowBackward && threadIdx.x == 0) {
        if (a.logp) a.logp[t] = 0.f;
        if (a.lse) a.lse[t] = 0.f;
        if (MODE == kRowPolicy)
          for (int i = 0; i < 3; ++i) a.p.terms[i * a.rows + t] = 0.f;
      }
      continue;
    }
    float lse, g;
    if constexpr (MODE == kRowBackward) {
      lse = __ldg(a.in_lse + t);
      g = __ldg(a.dlogp + t);
    } else {
      float m = -INFINITY, s = 0.f;
      for (int j = threadIdx.x; j < a.vocab; j += kThreads) {
        const float v = a.scale * to_f(x[j]);
        if (v > m) {
          s *= expf(m - v);
          m = v;
        }
        s += v == -INFINITY ? 0.f : expf(v - m);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1)
        join(m, s, __shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, s, o));
      __syncthreads();
      if (lane == 0) {
        s_m[warp] = m;
        s_s[warp] = s;
      }
      __syncthreads();
      m = s_m[0];
      s = s_s[0];
      for (int w = 1; w < kWarps; ++w) join(m, s, s_m[w], s_s[w]);
      const float rest = logf(s);
      lse = m + rest;
      float logp = y < a.vocab ? a.scale * to_f(x[y]) - m - rest : NAN;
      if (logp > 0.f) logp = 0.f;      // (by its rounding)
      if (threadIdx.x == 0) {
        if (a.logp) a.logp[t] = logp;
        if (a.lse) a.lse[t] = lse;
      }
      if constexpr (MODE == kRowPolicy) {
        const PolicyRow r = policy_row(a.p, t, doc, logp);
        g = r.grad;
        if (threadIdx.x == 0) {
          a.p.terms[t] = r.surrogate;
          a.p.terms[a.rows + t] = r.kl;
          a.p.terms[2 * a.rows + t] = r.clipped;
        }
        __syncthreads();               // (in place: x[y] has been read)
      }
    }
    if constexpr (MODE != kRowForward) {
      if (y >= a.vocab) g = NAN;
      const float sg = a.scale * g;
      for (int j = threadIdx.x; j < a.vocab; j += kThreads) {
        const float p = expf(a.scale * to_f(x[j]) - lse);
        st_out(dx + j, sg * ((j == y ? 1.f : 0.f) - p));
      }
    }
  }
}

template <typename T>
cudaError_t launch_typed(const RowArgs& a, RowMode mode, cudaStream_t s) {
  const unsigned blocks = (unsigned)(a.rows < 65536 ? a.rows : 65536);
  if (mode == kRowForward) row_kernel<T, kRowForward><<<blocks, kThreads, 0, s>>>(a);
  else if (mode == kRowBackward) row_kernel<T, kRowBackward><<<blocks, kThreads, 0, s>>>(a);
  else row_kernel<T, kRowPolicy><<<blocks, kThreads, 0, s>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rows(const RowArgs& a, RowMode mode, int32_t io_dtype, cudaStream_t s) {
  return io_dtype == NSP_BF16 ? launch_typed<__nv_bfloat16>(a, mode, s) : launch_typed<float>(a, mode, s);
}

}  // namespace nsp
