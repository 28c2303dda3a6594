// Per-row values of the differential attention backward, and the gradient of
// lambda.
//
// With delta_m = <dout, O_m> per (token, head), and out = O_1 - lambda O_2 and
// O_2 saved by the forward:
//   delta_2 = <dout, out2>,  delta_1 = <dout, out> + lambda delta_2,
//   dlambda = -delta_2 (of each token), or its sum over the tokens.
// Written as [2 Hq][Tp] rows (-delta, -lse log2 e) and [Hq][Tp] (c = -lambda, the
// factor of the second map's probabilities, and -c delta_2), padded with zeros to whole
// 128-row tiles.  Bound: HBM, one read of out, out2 and dout.
#include <algorithm>

#include "layer.cuh"

namespace nsp {
namespace {

constexpr int kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) diff_prep_kernel(const DiffProblem a) {
  constexpr int N = Vec<T>::N;
  constexpr int TPR = D / N;                       // threads of a row
  constexpr int RPW = 32 / TPR;                    // rows of a warp
  constexpr int ROWS = 4;                          // rows of a thread in flight
  const AttnProblem& p = a.p;
  grid_dep_trigger();
  if (status_bad(p.hdr)) return;
  const int lane = threadIdx.x & 31, sub = lane / TPR, part = lane % TPR;
  const int64_t warp = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5;
  const int64_t nwarps = ((int64_t)gridDim.x * kThreads) >> 5;
  const int64_t T_ = p.q_len, rows = T_ * p.Hq;
  const T* O = reinterpret_cast<const T*>(a.fout);
  const T* O2 = reinterpret_cast<const T*>(a.out2);
  const T* G = reinterpret_cast<const T*>(a.dout);
  const T* L = reinterpret_cast<const T*>(a.lambda);
  for (int64_t r0 = warp * RPW * ROWS; r0 < rows; r0 += nwarps * RPW * ROWS) {
    uint4 x[ROWS], y[ROWS], z[ROWS];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      const int64_t r = r0 + k * RPW + sub, off = r * D + part * N;
      x[k] = y[k] = z[k] = make_uint4(0, 0, 0, 0);
      if (r < rows) {
        x[k] = ld_once(O + off);
        y[k] = ld_once(O2 + off);
        z[k] = ld_once(G + off);
      }
    }
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      float u[N], v[N], g[N];
      Vec<T>::unpack(x[k], u);
      Vec<T>::unpack(y[k], v);
      Vec<T>::unpack(z[k], g);
      float d0 = 0.f, d2 = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        d0 = fmaf(g[i], u[i], d0);
        d2 = fmaf(g[i], v[i], d2);
      }
#pragma unroll
      for (int o = TPR / 2; o > 0; o >>= 1) {
        d0 += __shfl_xor_sync(0xffffffffu, d0, o);
        d2 += __shfl_xor_sync(0xffffffffu, d2, o);
      }
      const int64_t r = r0 + k * RPW + sub;
      if (r >= rows || part != 0) continue;
      const int64_t t = r / p.Hq;
      const int h = (int)(r - t * p.Hq);
      const float lam = to_f(L[(int64_t)h * a.n_lambda + (a.n_lambda > 1 ? t : 0)]);
      const int64_t v1 = (int64_t)h * 2 * a.Tp + t, v2 = v1 + a.Tp;
      a.ndelta[v1] = -fmaf(lam, d2, d0);
      a.ndelta[v2] = -d2;
      a.nlse2[v1] = -kLog2e * __ldg(p.lse + (int64_t)h * 2 * T_ + t);
      a.nlse2[v2] = -kLog2e * __ldg(p.lse + ((int64_t)h * 2 + 1) * T_ + t);
      a.coef[(int64_t)h * a.Tp + t] = -lam;
      a.cndelta[(int64_t)h * a.Tp + t] = lam * d2;
      if (a.n_lambda > 1) st_out(reinterpret_cast<T*>(a.dlambda) + (int64_t)h * T_ + t, -d2);
    }
  }
  // zero padding of the last tile's rows
  const int pad = (int)(a.Tp - T_);
  const int64_t tid = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  for (int64_t e = tid; e < (int64_t)pad * p.Hq; e += (int64_t)gridDim.x * kThreads) {
    const int64_t h = e / pad, t = T_ + (e - h * pad);
    a.ndelta[h * 2 * a.Tp + t] = a.ndelta[(h * 2 + 1) * a.Tp + t] = 0.f;
    a.nlse2[h * 2 * a.Tp + t] = a.nlse2[(h * 2 + 1) * a.Tp + t] = 0.f;
    a.coef[h * a.Tp + t] = a.cndelta[h * a.Tp + t] = 0.f;
  }
}

// dlambda[h] = sum_t -delta_2, one block of a head, in one fixed order.
template <typename T>
__global__ void __launch_bounds__(1024) diff_dlambda_kernel(const float* __restrict__ ndelta,
                                                            int64_t tokens, int64_t Tp, T* dlambda,
                                                            const WsHeader* hdr) {
  __shared__ float s[32];
  if (status_bad(hdr)) return;
  const float* row = ndelta + ((int64_t)blockIdx.x * 2 + 1) * Tp;
  float x = 0.f;
  for (int64_t t = threadIdx.x; t < tokens; t += 1024) x += __ldcg(row + t);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = x;
  __syncthreads();
  if (threadIdx.x >= 32) return;
  x = s[threadIdx.x];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if (threadIdx.x == 0) st_out(dlambda + blockIdx.x, x);
}

template <typename T>
cudaError_t prep(const DiffProblem& a, cudaStream_t s) {
  const int64_t blocks = std::min<int64_t>(
      ceil_div(a.p.q_len * a.p.Hq, kThreads / (a.p.d / Vec<T>::N) * 4), (int64_t)num_sms() * 8);
  if (a.p.d == 128)
    diff_prep_kernel<T, 128><<<(unsigned)blocks, kThreads, 0, s>>>(a);
  else
    diff_prep_kernel<T, 64><<<(unsigned)blocks, kThreads, 0, s>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

template <typename T>
cudaError_t dlambda(const DiffProblem& a, cudaStream_t s) {
  diff_dlambda_kernel<T><<<a.p.Hq, 1024, 0, s>>>(a.ndelta, a.p.q_len, a.Tp,
                                                 reinterpret_cast<T*>(a.dlambda), a.p.hdr);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_diff_prep(const DiffProblem& a, cudaStream_t s) {
  return a.p.io_dtype == NSP_BF16 ? prep<__nv_bfloat16>(a, s) : prep<float>(a, s);
}

cudaError_t launch_diff_dlambda(const DiffProblem& a, cudaStream_t s) {
  if (a.n_lambda > 1) return cudaSuccess;          // written row by row already
  return a.p.io_dtype == NSP_BF16 ? dlambda<__nv_bfloat16>(a, s) : dlambda<float>(a, s);
}

}  // namespace nsp
