// Declarations of the operators around differential attention (rotary
// positions, the difference weight, the head norm, differential attention
// itself) and the vector loads and stores their streaming kernels share.
#pragma once

#include <cuda.h>

#include "nsp_internal.cuh"

namespace nsp {

// ---- rotary positions (rope.cu)
constexpr int kRopeMaxTensors = 4;
constexpr int kRopeMaxDim = 1024;

struct RopeTensor {
  const void* in;
  void* out;
  int64_t in_stride, out_stride;     // elements between tokens
  int32_t heads;
  int32_t in_groups, out_groups;     // > 1: head-group-major [P][len][heads / P][d]
  int32_t hpg;                       // heads of a group
  int64_t in_jump, out_jump;         // from behind a group's last head to the next one's first
};

struct RopeArgs {
  RopeTensor t[kRopeMaxTensors];
  int32_t n;
  const int32_t* cu;
  int32_t ndoc;
  const int32_t* positions;
  int64_t start, len;
  int32_t d, rot, interleaved, inverse;
  const double* freqs;
  float mscale;
};
cudaError_t launch_rope(const RopeArgs& a, int32_t io_dtype, cudaStream_t s);

// ---- difference weight (diff_lambda.cu)
cudaError_t launch_diff_lambda(const void* const* v, int32_t n, int32_t dl, int32_t heads,
                               float init, int32_t io_dtype, void* lambda, cudaStream_t s);
cudaError_t launch_diff_lambda_bwd(const void* dlambda, const void* const* v, int32_t n, int32_t dl,
                                   int32_t heads, int32_t io_dtype, void* const* dvec,
                                   cudaStream_t s);

// ---- head norm (head_norm.cu)
constexpr int kNormMaxDim = 512;

struct NormArgs {
  const void *x, *gate, *weight, *dy;
  void *y, *dx, *dgate, *dweight;
  int64_t x_stride;                  // elements between tokens of x
  int64_t tokens;
  int32_t heads, d;
  float eps, scale;
  float* partial;                    // backward: [norm_bwd_blocks][d] weight gradient sums
};
int norm_bwd_blocks(int64_t rows);   // upper bound of the backward's grid, whatever the device
cudaError_t launch_head_norm(const NormArgs& a, int32_t io_dtype, cudaStream_t s);
cudaError_t launch_head_norm_bwd(const NormArgs& a, int32_t io_dtype, cudaStream_t s);

// ---- differential attention (diff_simt.cu, diff_fwd_tc.cu, diff_bwd_tc.cu)
// Whole packed stream of T tokens.  q, out, out2, dout, dq: [T, Hq, d]; k, v,
// dk, dv: [T, Hkv, d]; map m of a head is columns [m d/2, (m + 1) d/2) of q
// and k; lse: [Hq][2][T]; lambda: [Hq][n_lambda], n_lambda 1 or T.
struct DiffProblem {
  AttnProblem p;                     // q, k, v, cu, ranges (the whole stream), heads, header
  const void* lambda;
  int64_t n_lambda;
  void* out2;                        // second map's output (forward: may be null)
  const void *fout, *dout;           // backward
  void *dq, *dk, *dv, *dlambda;
  int shift;                         // log2 of the heads P of a query item (0 for float32)
  float *ndelta, *nlse2;             // backward workspace: [Hq / P][2][Tp][P]
  float *coef, *cndelta;             // [Hq / P][Tp][P]
  int64_t Tp;
  float* parts;                      // bf16 backward: shares of dV and dK of a key tile's parts
  float *dk_heads, *dv_heads;        // float32 backward, Hq > Hkv: [T, Hq, d] shares of the heads
};
// Heads of a tensor-core query item: the power of two in a group's heads, 8 at most
// (16 gained no more), and rows that 32 bits count.
constexpr int kMaxItemHeads = 8;
inline int item_shift(int group, int64_t T) {
  int shift = 0;
  while ((2 << shift) <= kMaxItemHeads && group % (2 << shift) == 0 &&
         (T << (shift + 1)) <= ((int64_t)1 << 30))
    ++shift;
  return shift;
}
// Most parts that the bf16 backward splits a key tile into, each some of the tile's (head
// group, query tile) pairs: as many as give each of 152 SMs one (not the device's count: the
// workspace's size depends on it).  One document of 4000 tokens, 4 heads on 1: 358 us whole,
// 146 in 8 parts; 8000 tokens in documents around 1024, 8 heads on 2: 369 whole, 231 in 2;
// 16384 tokens, 16 heads on 4, 512 key tiles: 555 whole, 618 in 2 (the shares' way through
// memory).  The rule counts tiles, not their work: one causal document loses some 15 % just
// past the border, where the first tiles, with twice the mean work, are whole again (8 heads
// on 2: 752 us at 9600 tokens, 895 at 9728; 16 on 4: 420 at 4736, 478 at 4864).
inline int key_parts(int64_t T, int Hkv) {
  const int64_t items = ceil_div(T, 128) * Hkv;
  int n = 1;
  while (n < 8 && items * n < 152 && T > 256) n *= 2;
  return n;
}
cudaError_t launch_diff_fwd_tc(const DiffProblem& a, const FwdWsLayout& L, char* ws, cudaStream_t s);
// A map of [rows, cols] bf16 whose copies are 128 rows of 64 columns, 128-byte
// swizzled; false without tensor-map support in the driver.
bool diff_tile_map(CUtensorMap* m, const void* base, int64_t rows, int64_t cols);
// The same of [T, H, d] in copies of `heads` heads at 128 / heads tokens.
bool diff_heads_map(CUtensorMap* m, const void* base, int64_t T, int64_t H, int64_t d, int heads);
cudaError_t launch_diff_fwd_simt(const DiffProblem& a, cudaStream_t s);
cudaError_t launch_diff_bwd_tc(const DiffProblem& a, const BwdWsLayout& L, char* ws, cudaStream_t s);
cudaError_t launch_diff_bwd_simt(const DiffProblem& a, cudaStream_t s);
// ndelta, nlse2, coef and cndelta of the backward, and dlambda of each token
cudaError_t launch_diff_prep(const DiffProblem& a, cudaStream_t s);
// dlambda of each head (n_lambda = 1), from ndelta
cudaError_t launch_diff_dlambda(const DiffProblem& a, cudaStream_t s);

#ifdef __CUDACC__

__device__ __forceinline__ float to_f(float x) { return x; }
__device__ __forceinline__ float to_f(__nv_bfloat16 x) { return __bfloat162float(x); }

// 16 bytes of T as float32 values, and back (round to nearest even).
template <typename T> struct Vec;
template <> struct Vec<float> {
  static constexpr int N = 4;
  __device__ static __forceinline__ void unpack(const uint4& u, float (&x)[N]) {
    x[0] = __uint_as_float(u.x); x[1] = __uint_as_float(u.y);
    x[2] = __uint_as_float(u.z); x[3] = __uint_as_float(u.w);
  }
  __device__ static __forceinline__ uint4 pack(const float (&x)[N]) {
    return make_uint4(__float_as_uint(x[0]), __float_as_uint(x[1]), __float_as_uint(x[2]),
                      __float_as_uint(x[3]));
  }
};
template <> struct Vec<__nv_bfloat16> {
  static constexpr int N = 8;
  __device__ static __forceinline__ void unpack(const uint4& u, float (&x)[N]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      x[2 * i] = __uint_as_float(w[i] << 16);
      x[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ static __forceinline__ uint4 pack(const float (&x)[N]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 b = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&b);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// Data touched once: loaded and stored past L1.  (Not the non-coherent load:
// an operator may write the buffer it reads.)
__device__ __forceinline__ uint4 ld_once(const void* p) {
  uint4 r;
  asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
               : "=r"(r.x), "=r"(r.y), "=r"(r.z), "=r"(r.w) : "l"(p) : "memory");
  return r;
}
__device__ __forceinline__ void st_once(void* p, const uint4& v) {
  asm volatile("st.global.L1::no_allocate.v4.u32 [%0], {%1,%2,%3,%4};" ::"l"(p), "r"(v.x),
               "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

#endif  // __CUDACC__

}  // namespace nsp
