// Sums of many float32 terms to more than float32's precision: a pair hi + lo,
// each addition's rounding error kept in lo (Knuth's two-sum: exact for any
// order of magnitudes).  float64 units are few on this GPU: one addition of a
// double takes the issue slots of some 30 of these.
#pragma once

#ifdef __CUDACC__

namespace nsp {

struct Sum2 {
  float hi, lo;
  __device__ __forceinline__ void add(float x) {
    const float s = hi + x, b = s - hi;
    lo += (hi - (s - b)) + (x - b);
    hi = s;
  }
  __device__ __forceinline__ void add(const Sum2& o) {
    add(o.hi);
    lo += o.lo;
  }
  // (where hi is not finite lo is NaN: what the sum is, hi says)
  __device__ __forceinline__ double value() const {
    return isfinite(hi) ? (double)hi + (double)lo : (double)hi;
  }
};

__device__ __forceinline__ Sum2 warp_sum(Sum2 x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) {
    Sum2 y;
    y.hi = __shfl_xor_sync(0xffffffffu, x.hi, o);
    y.lo = __shfl_xor_sync(0xffffffffu, x.lo, o);
    x.add(y);
  }
  return x;
}

// Sum over a block of W warps, in every thread, always in the same order; `s`: W
// entries of shared memory that no earlier sum uses any more.
template <int W>
__device__ __forceinline__ Sum2 block_sum(Sum2 x, Sum2* s) {
  x = warp_sum(x);
  if ((threadIdx.x & 31) == 0) s[threadIdx.x >> 5] = x;
  __syncthreads();
  x = {0.f, 0.f};
  if ((threadIdx.x & 31) < W) x = s[threadIdx.x & 31];
  return warp_sum(x);
}

}  // namespace nsp

#endif  // __CUDACC__
