// Angles of the rotation and the layouts its tensors come in: shared by the
// rotation itself (rope.cu) and by the head norm with the rotation in the same
// pass (qk_norm.cu).
#pragma once

#include "layer.cuh"

#ifdef __CUDACC__

namespace nsp {

// The row of head h at range row t: packed (token stride), or head-group-major.
__device__ __forceinline__ int64_t row_offset(int64_t t, int h, int64_t stride, int heads,
                                              int groups, int64_t len, int d) {
  if (groups <= 1) return t * stride + (int64_t)h * d;
  const int hpg = heads / groups, g = h / hpg;
  return (((int64_t)g * len + t) * hpg + (h - g * hpg)) * d;
}

// (of the magnitude, then negated: 1 minus a small fraction would lose its bits)
__device__ __forceinline__ uint64_t fixed_turns(double f) {
  double x = fabs(f) * 0.15915494309189533576888;    // 1 / (2 pi)
  x -= floor(x);
  const uint64_t u = __double2ull_rn(x * 18446744073709551616.0);
  return f < 0 ? 0 - u : u;
}

__device__ __forceinline__ void turn(int64_t pos, uint64_t fx, float m, bool inverse, float& c,
                                     float& s) {
  const int32_t hi = (int32_t)(((uint64_t)pos * fx) >> 32);
  sincospif((float)hi * 4.656612873077393e-10f, &s, &c);       // 2^-31: half turns
  c *= m;
  s *= inverse ? -m : m;
}

// Where a row's position comes from.
struct Positions {
  const int32_t* positions;          // given, or null: the distance from the document's start
  const int32_t* cu;
  int32_t ndoc;
  int64_t start;
};

// Position of range row t; false for a row past the last document.
__device__ __forceinline__ bool position_of(const Positions& a, int64_t t, int64_t& pos) {
  if (a.positions != nullptr) {
    pos = __ldg(a.positions + t);
    return true;
  }
  const int64_t g = a.start + t;
  if (g >= (int64_t)__ldg(a.cu + a.ndoc)) return false;
  pos = g - (int64_t)__ldg(a.cu + doc_of(a.cu, a.ndoc, g));
  return true;
}

}  // namespace nsp

#endif  // __CUDACC__
