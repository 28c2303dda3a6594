// Root-mean-square norm of every head's row, scaled and optionally gated:
//   r = 1 / sqrt(mean(x^2) + eps),  n = x r,  y = s w n [sigmoid(g)],
// and its backward, with c = s w [sigmoid(g)] and u = dy c:
//   dx = r (u - n mean(u n)),  dw = sum over rows of s dy n [sigmoid(g)],
//   dg = s w dy n sigmoid(g) (1 - sigmoid(g)).
//
// Bound: HBM, one read of every input and one write of every output.  A row
// is read once into the registers of a group of lanes (16 bytes a lane and
// step; 16 lanes for 128 bf16 columns, so a warp takes two rows), reduced by
// shuffles and written from there, with several rows of a group in flight.
// The weight's gradient is summed by every thread for its own columns over
// its rows, then over the block in shared memory, and over the blocks by a
// second small kernel, always in the same order.  32768 x 16 rows of 128 bf16 columns
// with gate and weight: 61.7 us, 6.5 TB/s; backward of 16383 x 16 such rows: 58.5 us a
// call, 5.7 TB/s (some 2.5 of them the second kernel).
#include <cfloat>
#include <algorithm>

#include "layer.cuh"
#include "tc_ptx.cuh"

namespace nsp {
namespace {

using namespace tc;

constexpr int kThreads = 256;

// 1 / (1 + exp(-g)), and exp(-g).  With float32 tensors exp is off by 2 ulp at most; with
// bf16 ones the short form is off by some 2 + 1.2 |g| ulp, 2^-16 of the value for the
// smallest gates that do not give zero, next to a rounding of 2^-8.  The reciprocal (of 1
// at least) is off by 1 ulp; below 2^-126 (a gate under -87) it is zero.
template <typename T>
__device__ __forceinline__ float sigmoid(float g, float& e) {
  e = sizeof(T) == 4 ? expf(-g) : __expf(-g);
  float x;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(x) : "f"(1.f + e));
  return x;
}

// A vector's values as packed pairs: two of them an instruction.
template <typename T>
__device__ __forceinline__ void unpack2(const uint4& u, uint64_t (&x)[Vec<T>::N / 2]) {
  float t[Vec<T>::N];
  Vec<T>::unpack(u, t);
#pragma unroll
  for (int i = 0; i < Vec<T>::N / 2; ++i) x[i] = f2_pack(t[2 * i], t[2 * i + 1]);
}
template <typename T>
__device__ __forceinline__ uint4 pack2(const uint64_t (&x)[Vec<T>::N / 2]) {
  float t[Vec<T>::N];
#pragma unroll
  for (int i = 0; i < Vec<T>::N / 2; ++i) f2_unpack(x[i], t[2 * i], t[2 * i + 1]);
  return Vec<T>::pack(t);
}
// A pair's sigmoids; `rest` becomes 1 - sigmoid = exp(-g) sigmoid, which a difference
// from 1 would not have for a large gate.  (exp may be infinite where sigmoid is zero.)
template <typename T>
__device__ __forceinline__ uint64_t sigmoid2(uint64_t g, uint64_t& rest) {
  float a, b, ea, eb;
  f2_unpack(g, a, b);
  const uint64_t s = f2_pack(sigmoid<T>(a, ea), sigmoid<T>(b, eb));
  rest = f2_mul(f2_pack(fminf(ea, FLT_MAX), fminf(eb, FLT_MAX)), s);
  return s;
}

__device__ __forceinline__ float group_sum(float x, int lanes) {
  for (int o = lanes >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// First element of a row of x: packed, or tokens x_stride apart.
__device__ __forceinline__ int64_t x_offset(const NormArgs& a, int64_t row) {
  if (a.x_stride == (int64_t)a.heads * a.d) return row * a.d;
  const int64_t t = row / a.heads;
  return t * a.x_stride + (row - t * a.heads) * a.d;
}

// V: 16-byte vectors of a lane; ROWS: rows of a group in flight.
template <typename T, int V, int ROWS>
__global__ void __launch_bounds__(kThreads) head_norm_kernel(const NormArgs a, int lanes) {
  constexpr int N = Vec<T>::N;
  const int lane = threadIdx.x & (lanes - 1);
  const int groups = kThreads / lanes, group = threadIdx.x / lanes;
  const int nvec = a.d / N;
  const int64_t rows = a.tokens * a.heads;
  const float inv_d = 1.f / (float)a.d;
  const T* const X = reinterpret_cast<const T*>(a.x);
  const T* const G = reinterpret_cast<const T*>(a.gate);
  T* const Y = reinterpret_cast<T*>(a.y);
  float w[V][N];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = lane + v * lanes;
#pragma unroll
    for (int i = 0; i < N; ++i) w[v][i] = a.scale;
    if (a.weight != nullptr && c < nvec) {
      float t[N];
      Vec<T>::unpack(__ldg(reinterpret_cast<const uint4*>(a.weight) + c), t);
#pragma unroll
      for (int i = 0; i < N; ++i) w[v][i] *= t[i];
    }
  }
  const int64_t step = (int64_t)gridDim.x * groups * ROWS;
  // every lane of a warp takes the same number of turns (shuffles inside)
  for (int64_t r0 = (int64_t)blockIdx.x * groups * ROWS; r0 < rows; r0 += step) {
    uint4 x[ROWS][V], g[ROWS][V];
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      const int64_t row = r0 + k * groups + group;
      const T* src = X + x_offset(a, row);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = lane + v * lanes;
        const bool in = row < rows && c < nvec;
        x[k][v] = in ? ld_once(src + (int64_t)c * N) : make_uint4(0, 0, 0, 0);
        if (G != nullptr) g[k][v] = in ? ld_once(G + row * a.d + c * N) : make_uint4(0, 0, 0, 0);
      }
    }
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      const int64_t row = r0 + k * groups + group;
      float ss = 0.f;
#pragma unroll
      for (int v = 0; v < V; ++v) {
        float t[N];
        Vec<T>::unpack(x[k][v], t);
#pragma unroll
        for (int i = 0; i < N; ++i) ss = fmaf(t[i], t[i], ss);
      }
      const float r = rsqrtf(fmaf(group_sum(ss, lanes), inv_d, a.eps));
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = lane + v * lanes;
        if (row >= rows || c >= nvec) continue;
        float t[N], q[N];
        Vec<T>::unpack(x[k][v], t);
        if (G != nullptr) Vec<T>::unpack(g[k][v], q);
#pragma unroll
        for (int i = 0; i < N; ++i) {
          t[i] = t[i] * r * w[v][i];
          float e;
          if (G != nullptr) t[i] *= sigmoid<T>(q[i], e);
        }
        st_once(Y + row * a.d + c * N, Vec<T>::pack(t));
      }
    }
  }
}

template <typename T, int V, int ROWS>
__global__ void __launch_bounds__(kThreads, V == 1 ? 2 : 1) head_norm_bwd_kernel(const NormArgs a, int lanes) {
  constexpr int N = Vec<T>::N;
  extern __shared__ float s_dw[];                 // [groups][d]
  grid_dep_trigger();
  const int lane = threadIdx.x & (lanes - 1);
  const int groups = kThreads / lanes, group = threadIdx.x / lanes;
  const int nvec = a.d / N;
  const int64_t rows = a.tokens * a.heads;
  const float inv_d = 1.f / (float)a.d;
  const T* const X = reinterpret_cast<const T*>(a.x);
  const T* const G = reinterpret_cast<const T*>(a.gate);
  const T* const DY = reinterpret_cast<const T*>(a.dy);
  T* const DX = reinterpret_cast<T*>(a.dx);
  T* const DG = reinterpret_cast<T*>(a.dgate);
  constexpr int P = N / 2;                        // pairs of a vector
  uint64_t w[V][P], dw[V][P];
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = lane + v * lanes;
#pragma unroll
    for (int i = 0; i < P; ++i) {
      w[v][i] = f2_pack(1.f, 1.f);
      dw[v][i] = 0;
    }
    if (a.weight != nullptr && c < nvec)
      unpack2<T>(__ldg(reinterpret_cast<const uint4*>(a.weight) + c), w[v]);
  }
  const int64_t step = (int64_t)gridDim.x * groups * ROWS;
  // the next rows are on their way while these are worked on
  uint4 nx[ROWS][V], ng[ROWS][V], ny[ROWS][V];
  auto load = [&](int64_t r0) {
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      const int64_t row = r0 + k * groups + group;
      const T* src = X + x_offset(a, row);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = lane + v * lanes;
        const bool in = row < rows && c < nvec;
        nx[k][v] = in ? ld_once(src + (int64_t)c * N) : make_uint4(0, 0, 0, 0);
        ny[k][v] = in ? ld_once(DY + row * a.d + c * N) : make_uint4(0, 0, 0, 0);
        if (G != nullptr) ng[k][v] = in ? ld_once(G + row * a.d + c * N) : make_uint4(0, 0, 0, 0);
      }
    }
  };
  load((int64_t)blockIdx.x * groups * ROWS);
  for (int64_t r0 = (int64_t)blockIdx.x * groups * ROWS; r0 < rows; r0 += step) {
    uint4 x[ROWS][V], g[ROWS][V], y[ROWS][V];
#pragma unroll
    for (int k = 0; k < ROWS; ++k)
#pragma unroll
      for (int v = 0; v < V; ++v) {
        x[k][v] = nx[k][v];
        y[k][v] = ny[k][v];
        if (G != nullptr) g[k][v] = ng[k][v];
      }
    if (r0 + step < rows) load(r0 + step);
#pragma unroll
    for (int k = 0; k < ROWS; ++k) {
      const int64_t row = r0 + k * groups + group;
      // sums of x^2 and of x u (n and u scale out of the second one)
      uint64_t ss = 0, su = 0;
      uint64_t t[V][P], us[V][P], uw[V][P], sg[V][P];
#pragma unroll
      for (int v = 0; v < V; ++v) {
        unpack2<T>(x[k][v], t[v]);
        unpack2<T>(y[k][v], us[v]);
        if (G != nullptr) unpack2<T>(g[k][v], sg[v]);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          if (G != nullptr) {
            us[v][i] = f2_mul(us[v][i], sigmoid2<T>(sg[v][i], sg[v][i]));   // (sg: 1 - sigmoid from here on)
          }
          uw[v][i] = f2_mul(us[v][i], w[v][i]);
          ss = f2_fma(t[v][i], t[v][i], ss);
          su = f2_fma(t[v][i], uw[v][i], su);
        }
      }
      float s0, s1, u0, u1;
      f2_unpack(ss, s0, s1);
      f2_unpack(su, u0, u1);
      const float r = rsqrtf(fmaf(group_sum(s0 + s1, lanes), inv_d, a.eps));
      const float mean = group_sum(u0 + u1, lanes) * r * inv_d;      // mean(u n) / s
      const float sr = a.scale * r;
      const uint64_t sr2 = f2_pack(sr, sr), nm2 = f2_pack(-sr * mean * r, -sr * mean * r);
#pragma unroll
      for (int v = 0; v < V; ++v) {
        const int c = lane + v * lanes;
        if (row >= rows || c >= nvec) continue;
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const uint64_t st = f2_mul(t[v][i], sr2);                  // s n
          dw[v][i] = f2_fma(st, us[v][i], dw[v][i]);
          if (G != nullptr) sg[v][i] = f2_mul(f2_mul(st, uw[v][i]), sg[v][i]);
          t[v][i] = f2_fma(uw[v][i], sr2, f2_mul(t[v][i], nm2));
        }
        st_once(DX + row * a.d + c * N, pack2<T>(t[v]));
        if (G != nullptr) st_once(DG + row * a.d + c * N, pack2<T>(sg[v]));
      }
    }
  }
  if (a.partial == nullptr) return;
#pragma unroll
  for (int v = 0; v < V; ++v) {
    const int c = lane + v * lanes;
    if (c >= nvec) continue;
#pragma unroll
    for (int i = 0; i < P; ++i)
      f2_unpack(dw[v][i], s_dw[group * a.d + c * N + 2 * i], s_dw[group * a.d + c * N + 2 * i + 1]);
  }
  __syncthreads();
  for (int c = threadIdx.x; c < a.d; c += kThreads) {
    float x = 0.f;
    for (int k = 0; k < groups; ++k) x += s_dw[k * a.d + c];
    a.partial[(int64_t)blockIdx.x * a.d + c] = x;
  }
}

// dw[c] = sum of the blocks' partial sums; 32 columns of a block, 32 warps
// taking every 32nd partial row.
constexpr int kSumThreads = 1024;
template <typename T>
__global__ void __launch_bounds__(kSumThreads) norm_weight_grad_kernel(
    const float* __restrict__ partial, int n, int d, T* dw) {
  __shared__ float s[32][33];
  grid_dep_wait();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
  float x = 0.f;
  if (c < d) {
#pragma unroll 4
    for (int k = warp; k < n; k += 32) x += __ldcg(partial + (int64_t)k * d + c);
  }
  s[warp][lane] = x;
  __syncthreads();
  // column `warp` of the block: its 32 sums are one warp's lanes now
  x = s[lane][warp];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  if (lane == 0 && blockIdx.x * 32 + warp < d) st_out(dw + blockIdx.x * 32 + warp, x);
}

// Lanes of a row (a power of two) and vectors of a lane.
template <typename T>
void shape(int d, int& lanes, int& vecs) {
  const int nvec = d / (16 / (int)sizeof(T));
  lanes = 1;
  while (lanes < 32 && lanes < nvec) lanes *= 2;
  vecs = (nvec + lanes - 1) / lanes;
}

template <typename T>
cudaError_t fwd(const NormArgs& a, cudaStream_t s) {
  int lanes, vecs;
  shape<T>(a.d, lanes, vecs);
  const int64_t rows = a.tokens * a.heads;
  auto go = [&](auto kern, int in_flight) {
    const int64_t per = (int64_t)(kThreads / lanes) * in_flight;
    const int64_t blocks = std::min<int64_t>(ceil_div(rows, per), (int64_t)num_sms() * 8);
    kern<<<(unsigned)blocks, kThreads, 0, s>>>(a, lanes);
  };
  if (vecs == 1) go(head_norm_kernel<T, 1, 4>, 4);
  else if (vecs == 2) go(head_norm_kernel<T, 2, 2>, 2);
  else go(head_norm_kernel<T, 4, 1>, 1);
  count_launches(1);
  return cudaGetLastError();
}

template <typename T>
cudaError_t bwd(const NormArgs& a, cudaStream_t s) {
  int lanes, vecs;
  shape<T>(a.d, lanes, vecs);
  const int64_t rows = a.tokens * a.heads;
  const size_t smem = a.partial ? sizeof(float) * (size_t)(kThreads / lanes) * a.d : 0;
  int64_t blocks = 1;
  auto go = [&](auto kern, int in_flight) {
    const int64_t per = (int64_t)(kThreads / lanes) * in_flight;
    blocks = std::min<int64_t>(ceil_div(rows, per), norm_bwd_blocks(rows));
    kern<<<(unsigned)blocks, kThreads, smem, s>>>(a, lanes);
  };
  if (vecs == 1) go(head_norm_bwd_kernel<T, 1, 2>, 2);
  else if (vecs == 2) go(head_norm_bwd_kernel<T, 2, 1>, 1);
  else go(head_norm_bwd_kernel<T, 4, 1>, 1);
  count_launches(1);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !a.partial) return e;
  e = launch_dependent(norm_weight_grad_kernel<T>, dim3((a.d + 31) / 32), dim3(kSumThreads), 0, s,
                       (const float*)a.partial, (int)blocks, (int)a.d,
                       reinterpret_cast<T*>(a.dweight));
  count_launches(1);
  return e;
}

}  // namespace

// At most 304 blocks, two on each of 152 SMs, as many as fit at once with two rows
// of a group worked on and two more on their way (16383 x 16 x 128 with gate: 56.7 us;
// three blocks without rows on their way 63.3, four blocks of one row and one 57.1),
// fewer for few rows: the size of the workspace must not depend on the device.
int norm_bwd_blocks(int64_t rows) {
  return (int)std::max<int64_t>(1, std::min<int64_t>(304, ceil_div(rows, 8)));
}

cudaError_t launch_head_norm(const NormArgs& a, int32_t io_dtype, cudaStream_t s) {
  return io_dtype == NSP_BF16 ? fwd<__nv_bfloat16>(a, s) : fwd<float>(a, s);
}

cudaError_t launch_head_norm_bwd(const NormArgs& a, int32_t io_dtype, cudaStream_t s) {
  return io_dtype == NSP_BF16 ? bwd<__nv_bfloat16>(a, s) : bwd<float>(a, s);
}

}  // namespace nsp
