// The learned weight of a head's second map,
//   lambda = exp(<q1, k1>) - exp(<q2, k2>) + init,
// and the gradients of its four vectors.  One set of vectors for each head
// (n = heads) or one shared by all (n = 1: every head gets the same lambda,
// and the gradient sums the heads' gradients in a fixed order).
//
// A few kilobytes: bound by the launch.  One warp per set, lanes along the
// vectors, one launch for the whole expression: 13 us a call for 16 heads of 64
// columns, 22 us for the gradients of 40 heads on one set, most of it the host's.
#include "layer.cuh"

namespace nsp {
namespace {

constexpr int kThreads = 128;
constexpr int kWarps = kThreads / 32;

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

template <typename T>
struct Vectors {
  const T *q1, *k1, *q2, *k2;
};

template <typename T>
__device__ __forceinline__ void exps(const Vectors<T>& v, int64_t row, int dl, int lane, float& e1,
                                     float& e2) {
  float d1 = 0.f, d2 = 0.f;
  for (int i = lane; i < dl; i += 32) {
    d1 = fmaf(to_f(v.q1[row + i]), to_f(v.k1[row + i]), d1);
    d2 = fmaf(to_f(v.q2[row + i]), to_f(v.k2[row + i]), d2);
  }
  e1 = expf(warp_sum(d1));
  e2 = expf(warp_sum(d2));
}

template <typename T>
__global__ void __launch_bounds__(kThreads) diff_lambda_kernel(Vectors<T> v, int n, int dl,
                                                               int heads, float init,
                                                               T* __restrict__ lambda) {
  const int r = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (r >= n) return;
  float e1, e2;
  exps(v, (int64_t)r * dl, dl, lane, e1, e2);
  const float x = e1 - e2 + init;
  if (n == heads) {
    if (lane == 0) st_out(lambda + r, x);
  } else {
    for (int h = lane; h < heads; h += 32) st_out(lambda + h, x);
  }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) diff_lambda_bwd_kernel(const T* __restrict__ dlambda,
                                                                   Vectors<T> v, int n, int dl,
                                                                   int heads, T* dq1, T* dk1,
                                                                   T* dq2, T* dk2) {
  const int r = blockIdx.x * kWarps + (threadIdx.x >> 5), lane = threadIdx.x & 31;
  if (r >= n) return;
  const int64_t row = (int64_t)r * dl;
  float g = 0.f;
  if (n == heads) {
    g = to_f(dlambda[r]);
  } else {
    for (int h = lane; h < heads; h += 32) g += to_f(dlambda[h]);
    g = warp_sum(g);
  }
  float e1, e2;
  exps(v, row, dl, lane, e1, e2);
  const float g1 = g * e1, g2 = -g * e2;
  for (int i = lane; i < dl; i += 32) {
    st_out(dq1 + row + i, g1 * to_f(v.k1[row + i]));
    st_out(dk1 + row + i, g1 * to_f(v.q1[row + i]));
    st_out(dq2 + row + i, g2 * to_f(v.k2[row + i]));
    st_out(dk2 + row + i, g2 * to_f(v.q2[row + i]));
  }
}

template <typename T>
Vectors<T> vectors(const void* const* v) {
  return {reinterpret_cast<const T*>(v[0]), reinterpret_cast<const T*>(v[1]),
          reinterpret_cast<const T*>(v[2]), reinterpret_cast<const T*>(v[3])};
}

template <typename T>
cudaError_t fwd(const void* const* v, int n, int dl, int heads, float init, void* lambda,
                cudaStream_t s) {
  diff_lambda_kernel<T><<<(n + kWarps - 1) / kWarps, kThreads, 0, s>>>(
      vectors<T>(v), n, dl, heads, init, reinterpret_cast<T*>(lambda));
  count_launches(1);
  return cudaGetLastError();
}

template <typename T>
cudaError_t bwd(const void* dlambda, const void* const* v, int n, int dl, int heads,
                void* const* dvec, cudaStream_t s) {
  diff_lambda_bwd_kernel<T><<<(n + kWarps - 1) / kWarps, kThreads, 0, s>>>(
      reinterpret_cast<const T*>(dlambda), vectors<T>(v), n, dl, heads,
      reinterpret_cast<T*>(dvec[0]), reinterpret_cast<T*>(dvec[1]), reinterpret_cast<T*>(dvec[2]),
      reinterpret_cast<T*>(dvec[3]));
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_diff_lambda(const void* const* v, int32_t n, int32_t dl, int32_t heads,
                               float init, int32_t io_dtype, void* lambda, cudaStream_t s) {
  return io_dtype == NSP_BF16 ? fwd<__nv_bfloat16>(v, n, dl, heads, init, lambda, s)
                              : fwd<float>(v, n, dl, heads, init, lambda, s);
}

cudaError_t launch_diff_lambda_bwd(const void* dlambda, const void* const* v, int32_t n, int32_t dl,
                                   int32_t heads, int32_t io_dtype, void* const* dvec,
                                   cudaStream_t s) {
  return io_dtype == NSP_BF16 ? bwd<__nv_bfloat16>(dlambda, v, n, dl, heads, dvec, s)
                              : bwd<float>(dlambda, v, n, dl, heads, dvec, s);
}

}  // namespace nsp
