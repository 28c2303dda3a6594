// Per-row values of the differential attention backward, and the gradient of
// lambda.
//
// With delta_m = <dout, O_m> per (token, head), and out = O_1 - lambda O_2 and
// O_2 saved by the forward:
//   delta_2 = <dout, out2>,  delta_1 = <dout, out> + lambda delta_2,
//   dlambda = -delta_2 (of each token), or its sum over the tokens.
// With bf16 tensors dlambda is not taken from here: out2 is rounded, and a head's sum
// over the tokens cancels; the dQ kernel puts -sum_j P_2 dP in float32 in delta_2's place.
// Written as [Hq / P][2][Tp][P] (-delta, -lse log2 e) and [Hq / P][Tp][P] (c = -lambda,
// the factor of the second map's probabilities, and -c delta_2) for the P = 2^shift
// heads of a query item, padded with zeros to whole 128-row tiles.  Bound: HBM, one read
// of out, out2 and dout: 201 MB of 16384 tokens, 16 heads, d = 128 in 37 us, 5.5 TB/s.
#include <algorithm>

#include "layer.cuh"

namespace nsp {
namespace {

constexpr int kThreads = 256;
constexpr float kLog2e = 1.4426950408889634f;

// Rows in the order of the vectors: row j of a head group is token j >> shift, head
// j % 2^shift.  A warp takes kRows consecutive ones (its neighbours the next groups'),
// so that the values it writes are neighbours.
template <typename T, int D>
struct PrepShape {
  static constexpr int TPR = D / Vec<T>::N;                       // threads of a row
  static constexpr int RPW = 32 / TPR;                            // rows of a warp at once
  static constexpr int ROWS = 4;                                  // rows of a thread in flight
  static constexpr int kRows = RPW * ROWS;
};

template <typename T, int D>
__global__ void __launch_bounds__(kThreads) diff_prep_kernel(const DiffProblem a) {
  constexpr int N = Vec<T>::N;
  using S = PrepShape<T, D>;
  const AttnProblem& p = a.p;
  grid_dep_trigger();
  if (status_bad(p.hdr)) return;
  const int lane = threadIdx.x & 31, sub = lane / S::TPR, part = lane % S::TPR;
  const int64_t warp = ((int64_t)blockIdx.x * kThreads + threadIdx.x) >> 5;
  const int64_t nwarps = ((int64_t)gridDim.x * kThreads) >> 5;
  const int64_t T_ = p.q_len, n = T_ << a.shift, np = a.Tp << a.shift;
  const int groups = p.Hq >> a.shift, last = (1 << a.shift) - 1;
  const int64_t units = (n + S::kRows - 1) / S::kRows * groups;
  const T* O = reinterpret_cast<const T*>(a.fout);
  const T* O2 = reinterpret_cast<const T*>(a.out2);
  const T* G = reinterpret_cast<const T*>(a.dout);
  const T* L = reinterpret_cast<const T*>(a.lambda);
  for (int64_t u = warp; u < units; u += nwarps) {
    const int64_t chunk = u / groups, j0 = chunk * S::kRows;
    const int hg = (int)(u - chunk * groups);
    uint4 x[S::ROWS], y[S::ROWS], z[S::ROWS];
#pragma unroll
    for (int k = 0; k < S::ROWS; ++k) {
      const int64_t j = j0 + k * S::RPW + sub;
      const int h = (hg << a.shift) + (int)(j & last);
      const int64_t off = ((j >> a.shift) * p.Hq + h) * D + part * N;
      x[k] = y[k] = z[k] = make_uint4(0, 0, 0, 0);
      if (j < n) {
        x[k] = ld_once(O + off);
        y[k] = ld_once(O2 + off);
        z[k] = ld_once(G + off);
      }
    }
    float m0 = 0.f, m2 = 0.f;                      // of row j0 + lane (lanes below kRows)
#pragma unroll
    for (int k = 0; k < S::ROWS; ++k) {
      float v[N], w[N], g[N];
      Vec<T>::unpack(x[k], v);
      Vec<T>::unpack(y[k], w);
      Vec<T>::unpack(z[k], g);
      float d0 = 0.f, d2 = 0.f;
#pragma unroll
      for (int i = 0; i < N; ++i) {
        d0 = fmaf(g[i], v[i], d0);
        d2 = fmaf(g[i], w[i], d2);
      }
#pragma unroll
      for (int o = S::TPR / 2; o > 0; o >>= 1) {
        d0 += __shfl_xor_sync(0xffffffffu, d0, o);
        d2 += __shfl_xor_sync(0xffffffffu, d2, o);
      }
      d0 = __shfl_sync(0xffffffffu, d0, (lane % S::RPW) * S::TPR);
      d2 = __shfl_sync(0xffffffffu, d2, (lane % S::RPW) * S::TPR);
      if (lane / S::RPW == k) {
        m0 = d0;
        m2 = d2;
      }
    }
    const int64_t j = j0 + lane, t = j >> a.shift;
    const int h = (hg << a.shift) + (int)(j & last);
    if (lane >= S::kRows || j >= n) continue;
    const float lam = to_f(L[(int64_t)h * a.n_lambda + (a.n_lambda > 1 ? t : 0)]);
    const int64_t v1 = (int64_t)hg * 2 * np + j, v2 = v1 + np, vc = (int64_t)hg * np + j;
    a.ndelta[v1] = -fmaf(lam, m2, m0);
    a.nlse2[v1] = -kLog2e * __ldg(p.lse + (int64_t)h * 2 * T_ + t);
    a.nlse2[v2] = -kLog2e * __ldg(p.lse + ((int64_t)h * 2 + 1) * T_ + t);
    a.coef[vc] = -lam;
    a.cndelta[vc] = lam * m2;
    if constexpr (sizeof(T) == 4) {
      a.ndelta[v2] = -m2;
      if (a.n_lambda > 1) st_out(reinterpret_cast<T*>(a.dlambda) + (int64_t)h * T_ + t, -m2);
    }
  }
  // zero padding of the last tile's rows
  const int64_t pad = np - n;
  const int64_t tid = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  for (int64_t e = tid; e < pad * groups; e += (int64_t)gridDim.x * kThreads) {
    const int64_t hg = e / pad, j = n + (e - hg * pad);
    a.ndelta[hg * 2 * np + j] = a.ndelta[(hg * 2 + 1) * np + j] = 0.f;
    a.nlse2[hg * 2 * np + j] = a.nlse2[(hg * 2 + 1) * np + j] = 0.f;
    a.coef[hg * np + j] = a.cndelta[hg * np + j] = 0.f;
  }
}

// dlambda[h] = sum_t -delta_2 (float32 rows), one block of a head, in one fixed order.
template <typename T>
__global__ void __launch_bounds__(1024) diff_dlambda_kernel(const float* __restrict__ ndelta,
                                                            int64_t tokens, int64_t Tp, int shift,
                                                            T* dlambda, const WsHeader* hdr) {
  __shared__ float s[32];
  if (status_bad(hdr)) return;
  const int hg = blockIdx.x >> shift;
  const float* row = ndelta + (((int64_t)hg * 2 + 1) * Tp << shift) + (blockIdx.x - (hg << shift));
  float x = 0.f;
  for (int64_t t = threadIdx.x; t < tokens; t += 1024) x += __ldcg(row + (t << shift));
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

template <typename T, int D>
cudaError_t prep_d(const DiffProblem& a, cudaStream_t s) {
  const int64_t units = ceil_div(a.p.q_len << a.shift, PrepShape<T, D>::kRows) * (a.p.Hq >> a.shift);
  const int64_t blocks = std::min<int64_t>(ceil_div(units, kThreads / 32), (int64_t)num_sms() * 8);
  diff_prep_kernel<T, D><<<(unsigned)blocks, kThreads, 0, s>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

template <typename T>
cudaError_t prep(const DiffProblem& a, cudaStream_t s) {
  return a.p.d == 128 ? prep_d<T, 128>(a, s) : prep_d<T, 64>(a, s);
}

template <typename T>
cudaError_t dlambda(const DiffProblem& a, cudaStream_t s) {
  diff_dlambda_kernel<T><<<a.p.Hq, 1024, 0, s>>>(a.ndelta, a.p.q_len, a.Tp, a.shift,
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
