// Global norm of many gradients, and the gradients scaled by what is left of it:
//   norm = |unscale| (sum g^2)^(1/2)  or  |unscale| max |g|,
//   out = g unscale min(1, max_norm / (norm + eps)).
#include <algorithm>
#include <cmath>

#include "sums.cuh"
#include "train.cuh"

namespace nsp {
namespace {

constexpr int kThreads = 256;
constexpr int kSumThreads = 1024;
constexpr int64_t kChunk = 32768;          // elements of a partial sum

// The tensors of one launch travel as a kernel parameter, so that a captured graph
// of the call carries them.
struct GradTensor {
  const void* in;
  void* out;
  int64_t count;
  int32_t chunk0;                          // its first chunk, of the launch's
  int32_t types;                           // 1: bf16 in, 2: bf16 out
};
template <int CAP>
struct GradTable {
  GradTensor t[CAP];
  int32_t n, chunks;
};

template <int CAP>
__device__ __forceinline__ int tensor_of(const GradTable<CAP>& g, int chunk) {
  int lo = 0, hi = g.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (g.t[mid].chunk0 <= chunk) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ float load(const void* p, int64_t i, bool bf16) {
  return bf16 ? to_f(reinterpret_cast<const __nv_bfloat16*>(p)[i]) : reinterpret_cast<const float*>(p)[i];
}

// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) { return a > b || isnan(a) ? a : b; }

template <int CAP>
__global__ void __launch_bounds__(kThreads) grad_norm_kernel(const __grid_constant__ GradTable<CAP> g,
                                                             int kind, Sum2* __restrict__ partial) {
  __shared__ Sum2 s_sum[kThreads / 32];
  for (int c = blockIdx.x; c < g.chunks; c += gridDim.x) {
    const GradTensor& t = g.t[tensor_of(g, c)];
    const int64_t first = (int64_t)(c - t.chunk0) * kChunk, last = min(first + kChunk, t.count);
    Sum2 x = {0.f, 0.f};
    for (int64_t i = first + threadIdx.x; i < last; i += kThreads) {
      const float v = load(t.in, i, t.types & 1);
      if (kind == NSP_NORM_2) x.add(v * v); else x.hi = max_nan(x.hi, fabsf(v));
    }
    __syncthreads();
    if (kind == NSP_NORM_2) {
      x = block_sum<kThreads / 32>(x, s_sum);
    } else {
      for (int o = 16; o > 0; o >>= 1) x.hi = max_nan(x.hi, __shfl_xor_sync(0xffffffffu, x.hi, o));
      if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = x;
      __syncthreads();
      for (int w = 0; w < kThreads / 32; ++w) x.hi = max_nan(x.hi, s_sum[w].hi);
    }
    if (threadIdx.x == 0) partial[c] = x;
  }
}

// norm, and the factor of the gradients, from the chunks' partial sums.
__global__ void __launch_bounds__(kSumThreads) grad_total_kernel(const Sum2* __restrict__ partial, int64_t n,
                                                                 int kind, float unscale, float max_norm,
                                                                 float eps, float* norm, float* factor) {
  __shared__ Sum2 s_sum[kSumThreads / 32];
  Sum2 x = {0.f, 0.f};
  for (int64_t i = threadIdx.x; i < n; i += kSumThreads) {
    if (kind == NSP_NORM_2) x.add(partial[i]); else x.hi = max_nan(x.hi, partial[i].hi);
  }
  double v;
  if (kind == NSP_NORM_2) {
    v = sqrt(block_sum<kSumThreads / 32>(x, s_sum).value());
  } else {
    for (int o = 16; o > 0; o >>= 1) x.hi = max_nan(x.hi, __shfl_xor_sync(0xffffffffu, x.hi, o));
    if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = x;
    __syncthreads();
    for (int w = 0; w < kSumThreads / 32; ++w) x.hi = max_nan(x.hi, s_sum[w].hi);
    v = x.hi;
  }
  if (threadIdx.x != 0) return;
  v *= fabs((double)unscale);
  norm[0] = (float)v;
  const double f = (double)max_norm / (v + (double)eps);
  factor[0] = (float)((f < 1.0 || isnan(f) ? f : 1.0) * (double)unscale);
}

template <int CAP>
__global__ void __launch_bounds__(kThreads) grad_scale_kernel(const __grid_constant__ GradTable<CAP> g,
                                                              const float* __restrict__ factor) {
  const float f = __ldcg(factor);
  for (int c = blockIdx.x; c < g.chunks; c += gridDim.x) {
    const GradTensor& t = g.t[tensor_of(g, c)];
    if (f == 1.f && t.in == t.out) continue;           // (in place: nothing changes)
    const int64_t first = (int64_t)(c - t.chunk0) * kChunk, last = min(first + kChunk, t.count);
    for (int64_t i = first + threadIdx.x; i < last; i += kThreads) {
      const float v = load(t.in, i, t.types & 1) * f;
      if (t.types & 2) st_out(reinterpret_cast<__nv_bfloat16*>(t.out) + i, v);
      else reinterpret_cast<float*>(t.out)[i] = v;
    }
  }
}

constexpr int kSmall = 64, kLarge = 768;

// Tables of at most CAP tensors, one launch each.
template <int CAP, typename F>
cudaError_t for_tables(const GradArgs& a, F launch) {
  GradTable<CAP> g;
  int64_t base = 0;
  for (int32_t i = 0; i < a.n;) {
    g.n = 0;
    g.chunks = 0;
    while (i < a.n && g.n < CAP) {
      const int64_t chunks = ceil_div(a.counts[i], kChunk);
      if (g.n > 0 && g.chunks + chunks > (1 << 30)) break;
      if (chunks > 0) {
        g.t[g.n++] = {a.in[i], a.out ? a.out[i] : nullptr, a.counts[i], g.chunks,
                      (a.in_dtypes[i] == NSP_BF16 ? 1 : 0) |
                          (a.out && a.out_dtypes[i] == NSP_BF16 ? 2 : 0)};
        g.chunks += (int32_t)chunks;
      }
      ++i;
    }
    if (g.chunks == 0) break;
    launch(g, base);
    count_launches(1);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    base += g.chunks;
  }
  return cudaSuccess;
}

template <int CAP>
cudaError_t run(const GradArgs& a, cudaStream_t s) {
  float* const factor = reinterpret_cast<float*>(a.workspace);
  Sum2* const partial = reinterpret_cast<Sum2*>(a.workspace + 256);
  const int64_t most = (int64_t)num_sms() * 8;
  int64_t chunks = 0;
  for (int32_t i = 0; i < a.n; ++i) chunks += ceil_div(a.counts[i], kChunk);
  cudaError_t e = for_tables<CAP>(a, [&](const GradTable<CAP>& g, int64_t base) {
    grad_norm_kernel<CAP><<<(unsigned)std::min<int64_t>(g.chunks, most), kThreads, 0, s>>>(g, a.kind, partial + base);
  });
  if (e != cudaSuccess) return e;
  grad_total_kernel<<<1, kSumThreads, 0, s>>>(partial, chunks, a.kind, a.unscale, a.max_norm, a.eps, a.norm, factor);
  count_launches(1);
  e = cudaGetLastError();
  if (e != cudaSuccess || !a.out) return e;
  return for_tables<CAP>(a, [&](const GradTable<CAP>& g, int64_t) {
    grad_scale_kernel<CAP><<<(unsigned)std::min<int64_t>(g.chunks, most), kThreads, 0, s>>>(g, factor);
  });
}

}  // namespace

size_t grad_ws_size(const int64_t* counts, int32_t n) {
  size_t chunks = 0;
  for (int32_t i = 0; i < n; ++i) chunks += (size_t)ceil_div(counts[i], kChunk);
  return 256 + chunks * sizeof(Sum2);
}

cudaError_t launch_grads(const GradArgs& a, cudaStream_t s) {
  return a.n <= kSmall ? run<kSmall>(a, s) : run<kLarge>(a, s);
}

}  // namespace nsp
