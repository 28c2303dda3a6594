// Root-mean-square norm of every query and key head with the rotation by its
// token's position in the same pass:
//   r = 1 / sqrt(mean(x^2) + eps),  n = x r,  y = R(w n),
// R the rotation of rope.cu (its factor included), and the backward, with
// z = R^T dy and u = w z:
//   dx = r (u - n mean(u n)),  dw = sum over rows of n z.
#include <algorithm>

#include "train.cuh"

namespace nsp {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kBwdBlocks = 304;

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// The blocks of a grid that a tensor's rows are given to.
struct Share {
  int first[kRopeMaxTensors + 1];
};

// One row a warp, one element (of a pair) a lane and step: any d, stride and
// alignment.  Columns of pair i < rot / 2, then the unrotated ones.
template <typename T, bool BACK>
__global__ void __launch_bounds__(kThreads) qk_element_kernel(const __grid_constant__ QkArgs a,
                                                              const Share share) {
  extern __shared__ float s_dw[];                  // BACK: [kWarps][d]
  int k = 0;
  while ((int)blockIdx.x >= share.first[k + 1]) ++k;
  const QkTensor& q = a.t[k];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int block = blockIdx.x - share.first[k], blocks = share.first[k + 1] - share.first[k];
  const int half = a.rot / 2, units = half + a.d - a.rot;
  const T* const W = reinterpret_cast<const T*>(q.weight);
  float* const dw = s_dw + warp * a.d;
  if (BACK)
    for (int c = lane; c < a.d; c += 32) dw[c] = 0.f;
  __syncwarp();
  const int64_t rows = a.len * q.heads;
  for (int64_t row = (int64_t)block * kWarps + warp; row < rows; row += (int64_t)blocks * kWarps) {
    const int64_t t = row / q.heads;
    const int h = (int)(row - t * q.heads);
    int64_t pos;
    if (!position_of(Positions{a.positions, a.cu, a.ndoc, a.start}, t, pos)) continue;
    const T* const x = reinterpret_cast<const T*>(q.x) + t * q.x_stride + (int64_t)h * a.d;
    const int64_t at = row_offset(t, h, q.y_stride, q.heads, q.groups, a.len, a.d);
    const T* const dy = reinterpret_cast<const T*>(q.dy) + at;
    float ss = 0.f, su = 0.f;
    for (int c = lane; c < a.d; c += 32) {
      const float v = to_f(x[c]);
      ss = fmaf(v, v, ss);
    }
    const float r = rsqrtf(fmaf(warp_sum(ss), 1.f / (float)a.d, a.eps));
    // (a, b) of unit i: its columns, or one column twice; z of both
    auto unit = [&](int i, int& ca, int& cb, float& za, float& zb, bool load) {
      if (i >= half) {
        ca = cb = a.rot + i - half;
        if (load) za = zb = to_f(dy[ca]);
        return false;
      }
      ca = a.interleaved ? 2 * i : i;
      cb = a.interleaved ? 2 * i + 1 : i + half;
      return true;
    };
    float mean = 0.f;
    for (int pass = BACK ? 0 : 1; pass < 2; ++pass) {
      for (int i = lane; i < units; i += 32) {
        int ca, cb;
        float za = 0.f, zb = 0.f, c, s;
        const bool pair = unit(i, ca, cb, za, zb, BACK);
        const float wa = W ? to_f(W[ca]) : 1.f, wb = W ? to_f(W[cb]) : 1.f;
        const float xa = to_f(x[ca]), xb = to_f(x[cb]);
        if (pair) turn(pos, fixed_turns(a.freqs[i]), a.mscale, BACK, c, s);
        if constexpr (!BACK) {
          T* const y = reinterpret_cast<T*>(q.y) + at;
          const float na = xa * r * wa, nb = xb * r * wb;
          if (pair) {
            st_out(y + ca, na * c - nb * s);
            st_out(y + cb, na * s + nb * c);
          } else {
            st_out(y + ca, na);
          }
        } else {
          if (pair) {
            const float ga = to_f(dy[ca]), gb = to_f(dy[cb]);
            za = ga * c - gb * s;
            zb = ga * s + gb * c;
          }
          if (pass == 0) {
            su = fmaf(wa * za, xa, su);
            if (pair) su = fmaf(wb * zb, xb, su);
          } else {
            T* const dx = reinterpret_cast<T*>(q.dx) + t * q.dx_stride + (int64_t)h * a.d;
            st_out(dx + ca, r * (wa * za - xa * r * mean));
            dw[ca] += xa * r * za;
            if (pair) {
              st_out(dx + cb, r * (wb * zb - xb * r * mean));
              dw[cb] += xb * r * zb;
            }
          }
        }
      }
      if (BACK && pass == 0) mean = warp_sum(su) * r * (1.f / (float)a.d);     // mean(u n)
      __syncwarp();            // (in place: every lane has read the row's x and dy, or will read its own)
    }
  }
  if (!BACK || q.dweight == nullptr) return;
  __syncthreads();
  for (int c = threadIdx.x; c < a.d; c += kThreads) {
    float x = 0.f;
    for (int w = 0; w < kWarps; ++w) x += s_dw[w * a.d + c];
    a.partial[(int64_t)blockIdx.x * a.d + c] = x;
  }
}

// dw[c] of a tensor: the sum of its blocks' partial sums, 32 columns of a block,
// 32 warps taking every 32nd of them.
constexpr int kSumThreads = 1024;
template <typename T>
__global__ void __launch_bounds__(kSumThreads) qk_weight_grad_kernel(const __grid_constant__ QkArgs a,
                                                                     const Share share) {
  __shared__ float s[32][33];
  grid_dep_wait();
  const int k = blockIdx.y, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  T* const dw = reinterpret_cast<T*>(a.t[k].dweight);
  if (dw == nullptr) return;
  const int c = blockIdx.x * 32 + lane;
  float x = 0.f;
  if (c < a.d) {
#pragma unroll 4
    for (int b = share.first[k] + warp; b < share.first[k + 1]; b += 32)
      x += __ldcg(a.partial + (int64_t)b * a.d + c);
  }
  s[warp][lane] = x;
  __syncthreads();
  x = warp_sum(s[lane][warp]);
  if (lane == 0 && blockIdx.x * 32 + warp < a.d) st_out(dw + blockIdx.x * 32 + warp, x);
}

template <typename T>
cudaError_t fwd(const QkArgs& a, cudaStream_t s) {
  Share share;
  share.first[0] = 0;
  for (int i = 0; i < kRopeMaxTensors; ++i) {
    const int64_t rows = i < a.n ? a.len * a.t[i].heads : 0;
    const int64_t blocks = std::min<int64_t>(ceil_div(rows, kWarps), (int64_t)num_sms() * 8);
    share.first[i + 1] = share.first[i] + (int)blocks;
  }
  qk_element_kernel<T, false><<<share.first[a.n], kThreads, 0, s>>>(a, share);
  count_launches(1);
  return cudaGetLastError();
}

template <typename T>
cudaError_t bwd(const QkArgs& a, cudaStream_t s) {
  Share share;
  share.first[0] = 0;
  bool weights = false;
  for (int i = 0; i < kRopeMaxTensors; ++i) {
    const int64_t rows = i < a.n ? a.len * a.t[i].heads : 0;
    share.first[i + 1] = share.first[i] + (i < a.n ? qk_bwd_blocks(rows) : 0);
    weights = weights || (i < a.n && a.t[i].dweight != nullptr);
  }
  qk_element_kernel<T, true><<<share.first[a.n], kThreads, sizeof(float) * kWarps * a.d, s>>>(a, share);
  count_launches(1);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !weights) return e;
  e = launch_dependent(qk_weight_grad_kernel<T>, dim3((a.d + 31) / 32, a.n), dim3(kSumThreads), 0, s,
                       a, share);
  count_launches(1);
  return e;
}

}  // namespace

int qk_bwd_blocks(int64_t rows) {
  return (int)std::max<int64_t>(1, std::min<int64_t>(kBwdBlocks, ceil_div(rows, kWarps)));
}

cudaError_t launch_qk_norm_rope(const QkArgs& a, int32_t io_dtype, cudaStream_t s) {
  return io_dtype == NSP_BF16 ? fwd<__nv_bfloat16>(a, s) : fwd<float>(a, s);
}

cudaError_t launch_qk_norm_rope_bwd(const QkArgs& a, int32_t io_dtype, cudaStream_t s) {
  return io_dtype == NSP_BF16 ? bwd<__nv_bfloat16>(a, s) : bwd<float>(a, s);
}

}  // namespace nsp
