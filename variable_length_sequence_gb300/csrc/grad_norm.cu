// Global norm of many gradients, and the gradients scaled by what is left of it:
//   norm = |unscale| (sum g^2)^(1/2)  or  |unscale| max |g|,
//   out = g unscale min(1, max_norm / (norm + eps)).
//
// Bound: HBM, one read of every gradient for the norm, one read and one write for the
// scaling.  All gradients one behind the other are cut in pieces of kPiece elements, and
// each of kBlocks blocks takes every kBlocks-th piece, whatever tensor it lies in, so that
// one launch serves hundreds of tensors and all blocks read and write close to one another
// (runs of neighbouring pieces a block: 659 us to scale 500 million elements).  A thread adds 16 float32 squares at a time and those sums in pairs of
// floats; the blocks' sums are added by every block that scales, or by one more.  The
// scaling starts at the end, where L2 still holds what the norm read last.  300 million
// float32 in 400 views of one buffer: 176 us, 6.8 TB/s; 500 million elements in 60 tensors
// of both types, clipped into others: 615 us, the norm 205 and the scaling 410 of them, 6.4
// TB/s of the bytes that they move.
#include <algorithm>
#include <cmath>

#include "sums.cuh"
#include "tc_ptx.cuh"
#include "train.cuh"

namespace nsp {
namespace {

using namespace tc;

constexpr int kThreads = 256, kWarps = kThreads / 32;
constexpr int kBlocks = 912;               // of a launch, whatever the device: six of an SM
constexpr int64_t kPiece = 8192;           // elements
constexpr int kBytes = 64, kScaleBytes = 32;   // that a thread has in flight (64 to scale: 712 us of the clipping above)

// The tensors of one launch travel as a kernel parameter, so that a captured graph
// of the call carries them.
struct GradTensor {
  const void* in;
  void* out;
  int64_t count;
  int32_t piece0;                          // its first piece, of the launch's
  int32_t types;                           // 1: bf16 in, 2: bf16 out
};
template <int CAP>
struct GradTable {
  GradTensor t[CAP];
  int32_t n, pieces;
};

template <int CAP>
__device__ __forceinline__ int tensor_of(const GradTable<CAP>& g, int piece) {
  int lo = 0, hi = g.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (g.t[mid].piece0 <= piece) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// max that keeps a NaN
__device__ __forceinline__ float max_nan(float a, float b) { return a > b || isnan(a) ? a : b; }

// Elements of a gradient before its first 16-byte border, at most n.
template <typename T>
__device__ __forceinline__ int head_of(const T* p, int64_t n) {
  return (int)min(n, (int64_t)(((16 - (reinterpret_cast<uintptr_t>(p) & 15)) & 15) / sizeof(T)));
}

// Calls f(tensor, first, last) for the elements of every kBlocks-th piece, from the first
// or from the last on: the blocks together sweep the gradients in order.  All pieces but
// a tensor's first begin at a 16-byte border.
template <int CAP, typename F>
__device__ __forceinline__ void for_pieces(const GradTable<CAP>& g, bool backwards, F f) {
  int p = backwards ? g.pieces - 1 - (int)blockIdx.x : (int)blockIdx.x;
  if (p < 0 || p >= g.pieces) return;
  int k = tensor_of(g, p);
  for (;;) {
    const GradTensor& t = g.t[k];
    const int head = t.types & 1 ? head_of(reinterpret_cast<const __nv_bfloat16*>(t.in), t.count)
                                 : head_of(reinterpret_cast<const float*>(t.in), t.count);
    const int64_t j = p - t.piece0;
    const int64_t first = j == 0 ? 0 : head + j * kPiece, last = min(head + (j + 1) * kPiece, t.count);
    if (first < last) f(t, first, last);
    if (backwards) {
      if ((p -= (int)gridDim.x) < 0) return;
      while (g.t[k].piece0 > p) --k;
    } else {
      if ((int)gridDim.x >= g.pieces - p) return;
      p += (int)gridDim.x;
      while (k + 1 < g.n && g.t[k + 1].piece0 <= p) ++k;
    }
  }
}

// W elements, 16-byte aligned.
template <typename T, int W>
struct Unit {
  static constexpr int N = Vec<T>::N, V = W / N;
  uint4 v[V];
  __device__ __forceinline__ void load(const T* p) {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = ld_once(p + i * N);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < V; ++i) v[i] = make_uint4(0, 0, 0, 0);
  }
  __device__ __forceinline__ void get(float (&x)[W]) const {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float t[N];
      Vec<T>::unpack(v[i], t);
#pragma unroll
      for (int j = 0; j < N; ++j) x[i * N + j] = t[j];
    }
  }
  __device__ __forceinline__ static void store(T* p, const float (&x)[W]) {
#pragma unroll
    for (int i = 0; i < V; ++i) {
      float t[N];
#pragma unroll
      for (int j = 0; j < N; ++j) t[j] = x[i * N + j];
      st_once(p + i * N, Vec<T>::pack(t));
    }
  }
};

template <typename T, bool MAX>
__device__ __forceinline__ void take_piece(const T* p, int64_t n, Sum2& x) {
  constexpr int W = Vec<T>::N, kFlight = kBytes / 16;
  const int head = head_of(p, n);
  const int units = (int)((n - head) / W);
  const int rest = (int)(n - units * W);                // before and behind the units: 14 at most
  if ((int)threadIdx.x < rest) {
    const float v = to_f(p[(int)threadIdx.x < head ? (int)threadIdx.x : units * W + (int)threadIdx.x]);
    if (MAX) x.hi = max_nan(x.hi, fabsf(v)); else x.add(v * v);
  }
  p += head;
  for (int i = threadIdx.x; i < units; i += kThreads * kFlight) {
    Unit<T, W> u[kFlight];
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      if (i + f * kThreads < units) u[f].load(p + (int64_t)(i + f * kThreads) * W);
      else u[f].zero();
    }
    uint64_t s[2] = {0, 0};
#pragma unroll
    for (int f = 0; f < kFlight; ++f) {
      float e[W];
      u[f].get(e);
#pragma unroll
      for (int j = 0; j < W / 2; ++j) {
        if constexpr (MAX) {
          x.hi = max_nan(max_nan(x.hi, fabsf(e[2 * j])), fabsf(e[2 * j + 1]));
        } else {
          const uint64_t v = f2_pack(e[2 * j], e[2 * j + 1]);
          s[f & 1] = f2_fma(v, v, s[f & 1]);
        }
      }
    }
    if constexpr (!MAX) {
      float a, b;
      f2_unpack(f2_add(s[0], s[1]), a, b);
      x.add(a + b);
    }
  }
}

// Over the block, in every thread.
template <bool MAX>
__device__ __forceinline__ Sum2 block_total(Sum2 x, Sum2* s) {
  if constexpr (!MAX) return block_sum<kWarps>(x, s);
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x.hi = max_nan(x.hi, __shfl_xor_sync(0xffffffffu, x.hi, o));
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = x;
  __syncthreads();
  for (int w = 0; w < kWarps; ++w) x.hi = max_nan(x.hi, s[w].hi);
  return x;
}

template <int CAP, bool MAX>
__global__ void __launch_bounds__(kThreads, 6) grad_norm_kernel(const __grid_constant__ GradTable<CAP> g,
                                                                Sum2* __restrict__ partial) {
  __shared__ Sum2 s_sum[kWarps];
  grid_dep_trigger();
  Sum2 x = {0.f, 0.f};
  for_pieces(g, false, [&](const GradTensor& t, int64_t first, int64_t last) {
    if (t.types & 1) take_piece<__nv_bfloat16, MAX>(reinterpret_cast<const __nv_bfloat16*>(t.in) + first, last - first, x);
    else take_piece<float, MAX>(reinterpret_cast<const float*>(t.in) + first, last - first, x);
  });
  x = block_total<MAX>(x, s_sum);
  if (threadIdx.x == 0) partial[blockIdx.x] = x;
}

struct Total {
  const Sum2* partial;
  int n;
  float unscale, max_norm, eps;
  float* norm;
};

// The norm, and the factor of the gradients, in every thread.
template <bool MAX>
__device__ __forceinline__ float total_of(const Total& t, bool write) {
  __shared__ Sum2 s_sum[kWarps];
  __shared__ float s_factor;
  Sum2 x = {0.f, 0.f};
#pragma unroll 4
  for (int i = threadIdx.x; i < t.n; i += kThreads) {
    const float2 p = __ldcg(reinterpret_cast<const float2*>(t.partial) + i);
    const Sum2 o = {p.x, p.y};
    if (MAX) x.hi = max_nan(x.hi, o.hi); else x.add(o);
  }
  x = block_total<MAX>(x, s_sum);
  if (threadIdx.x == 0) {
    const double v = (MAX ? (double)x.hi : sqrt(x.value())) * fabs((double)t.unscale);
    const double f = (double)t.max_norm / (v + (double)t.eps);
    s_factor = (float)((f < 1.0 || isnan(f) ? f : 1.0) * (double)t.unscale);
    if (write) t.norm[0] = (float)v;
  }
  __syncthreads();
  return s_factor;
}

template <bool MAX>
__global__ void __launch_bounds__(kThreads) grad_total_kernel(const __grid_constant__ Total t) {
  grid_dep_wait();
  total_of<MAX>(t, true);
}

template <typename TI, typename TO>
__device__ __forceinline__ void scale_piece(const TI* p, TO* o, int64_t n, float f) {
  constexpr int W = Vec<TI>::N > Vec<TO>::N ? Vec<TI>::N : Vec<TO>::N;
  constexpr int kFlight = kScaleBytes / (W * (int)sizeof(TI));
  const int head = head_of(p, n);
  const int units = (int)((n - head) / W);
  const int rest = (int)(n - units * W);
  if ((int)threadIdx.x < rest) {
    const int i = (int)threadIdx.x < head ? (int)threadIdx.x : units * W + (int)threadIdx.x;
    st_out(o + i, to_f(p[i]) * f);
  }
  p += head;
  o += head;
  const bool whole = (reinterpret_cast<uintptr_t>(o) & 15) == 0;
  for (int i = threadIdx.x; i < units; i += kThreads * kFlight) {
    Unit<TI, W> u[kFlight];
#pragma unroll
    for (int k = 0; k < kFlight; ++k)
      if (i + k * kThreads < units) u[k].load(p + (int64_t)(i + k * kThreads) * W);
#pragma unroll
    for (int k = 0; k < kFlight; ++k) {
      if (i + k * kThreads >= units) break;
      float e[W];
      u[k].get(e);
#pragma unroll
      for (int j = 0; j < W; ++j) e[j] *= f;
      TO* const q = o + (int64_t)(i + k * kThreads) * W;
      if (whole) {
        Unit<TO, W>::store(q, e);
      } else {
#pragma unroll
        for (int j = 0; j < W; ++j) st_out(q + j, e[j]);
      }
    }
  }
}

template <int CAP, bool MAX>
__global__ void __launch_bounds__(kThreads, 6) grad_scale_kernel(const __grid_constant__ GradTable<CAP> g,
                                                                 const __grid_constant__ Total total, bool write) {
  using B = __nv_bfloat16;
  grid_dep_wait();
  const float f = total_of<MAX>(total, write && blockIdx.x == 0);
  for_pieces(g, true, [&](const GradTensor& t, int64_t first, int64_t last) {
    if (f == 1.f && t.in == t.out) return;              // (in place: nothing changes)
    const int64_t n = last - first;
    if (t.types == 0) scale_piece(reinterpret_cast<const float*>(t.in) + first, reinterpret_cast<float*>(t.out) + first, n, f);
    else if (t.types == 3) scale_piece(reinterpret_cast<const B*>(t.in) + first, reinterpret_cast<B*>(t.out) + first, n, f);
    else if (t.types == 1) scale_piece(reinterpret_cast<const B*>(t.in) + first, reinterpret_cast<float*>(t.out) + first, n, f);
    else scale_piece(reinterpret_cast<const float*>(t.in) + first, reinterpret_cast<B*>(t.out) + first, n, f);
  });
}

// Tables of few tensors are a short parameter.
constexpr int kSmall = 64, kLarge = 768;

// Calls launch(table, number of the launch) for tables of at most CAP tensors.
template <int CAP, typename F>
cudaError_t for_tables(const GradArgs& a, F launch) {
  GradTable<CAP> g;
  int at = 0;
  for (int32_t i = 0; i < a.n;) {
    g.n = 0;
    int64_t pieces = 0;
    for (; i < a.n && g.n < CAP; ++i) {
      const int64_t more = ceil_div(a.counts[i], kPiece);
      if (more == 0) continue;
      if (pieces + more > INT32_MAX) break;             // (one tensor has 2^27 pieces at most)
      g.t[g.n++] = {a.in[i], a.out ? a.out[i] : nullptr, a.counts[i], (int32_t)pieces,
                    (a.in_dtypes[i] == NSP_BF16 ? 1 : 0) | (a.out && a.out_dtypes[i] == NSP_BF16 ? 2 : 0)};
      pieces += more;
    }
    g.pieces = (int32_t)pieces;
    if (g.n == 0) break;
    const cudaError_t e = launch(g, at);
    count_launches(1);
    if (e != cudaSuccess) return e;
    ++at;
  }
  return cudaSuccess;
}

template <int CAP, bool MAX>
cudaError_t run(const GradArgs& a, cudaStream_t s) {
  Sum2* const partial = reinterpret_cast<Sum2*>(a.workspace);
  Total total = {partial, 0, a.unscale, a.max_norm, a.eps, a.norm};
  auto blocks = [](const GradTable<CAP>& g) { return (unsigned)std::min(g.pieces, kBlocks); };
  cudaError_t e = for_tables<CAP>(a, [&](const GradTable<CAP>& g, int) {
    grad_norm_kernel<CAP, MAX><<<blocks(g), kThreads, 0, s>>>(g, partial + total.n);
    total.n += (int)blocks(g);
    return cudaGetLastError();
  });
  if (e != cudaSuccess) return e;
  if (!a.out || total.n == 0) {
    count_launches(1);
    return launch_dependent(grad_total_kernel<MAX>, dim3(1), dim3(kThreads), 0, s, total);
  }
  return for_tables<CAP>(a, [&](const GradTable<CAP>& g, int at) {
    return launch_dependent(grad_scale_kernel<CAP, MAX>, dim3(blocks(g)), dim3(kThreads), 0, s, g, total, at == 0);
  });
}

}  // namespace

// Sums of at most kBlocks blocks of each launch: of kSmall tensors or fewer one, then
// one for kLarge tensors, or for 2^31 pieces.
size_t grad_ws_size(const int64_t* counts, int32_t n) {
  int64_t pieces = 0;
  for (int32_t i = 0; i < n; ++i) pieces += ceil_div(counts[i], kPiece);
  const int64_t launches = 1 + n / kLarge + 2 * (pieces >> 31);
  return (size_t)std::max<int64_t>(1, std::min<int64_t>(launches * kBlocks, pieces)) * sizeof(Sum2);
}

cudaError_t launch_grads(const GradArgs& a, cudaStream_t s) {
  if (a.kind == NSP_NORM_2) return a.n <= kSmall ? run<kSmall, false>(a, s) : run<kLarge, false>(a, s);
  return a.n <= kSmall ? run<kSmall, true>(a, s) : run<kLarge, true>(a, s);
}

}  // namespace nsp
