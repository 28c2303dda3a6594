// Differential attention on the CUDA cores: the path of float32 inputs, in
// true float32 arithmetic (no TF32).
//
// Per document of the packed stream, with map m of a head reading columns
// [m D/2, (m + 1) D/2) of q and k:
//   P_m = softmax over the visible keys of scale q_m k_m^T,  O_m = P_m V,
//   out = O_1 - lambda O_2.
// Backward, with delta_m = <dout, O_m> and dP = dout V^T (one product for both
// maps):
//   dS_1 = P_1 (dP - delta_1),  dS_2 = -lambda P_2 (dP - delta_2),
//   dQ_m = scale dS_m K_m,  dK_m = scale dS_m^T Q_m,  dV = (P_1 - lambda P_2)^T dout.
//
// Bound: reads of shared memory beside the FP32 pipes, with the two blocks of four
// warps of an SM that 255 registers a thread leave (FMA pipes 50 to 55 % busy, issue
// slots 60 to 67 %).  Every product is tiled in registers, 16
// threads wide, from float32 tiles in shared memory, rows padded by 4 floats so
// that 16 rows read at one column fall into different banks; a thread's 8 rows by
// 4 keys take 12 reads for 128 FMAs (8 x 4 x d = 64; 4 x 4, 8 for 64, took 625 us
// forward and 1707 back against 570 and 1415 at 3001 tokens, 6 heads, d = 64,
// bidirectional).  At d = 128 registers or shared memory leave room for less:
// 8 x 2 forward (1165 us against 1293 at 3001 tokens, 8 heads, causal documents),
// 4 x 4 with twice the threads back (2530 us; 8 x 4 spills: 3112).  Asynchronous
// copies fill the buffer that a product has done with while the next one runs.
// Forward: both maps' scores, online softmax (Milakov and Gimelshein) and outputs
// stay in the registers of one thread row, 36 TFLOP/s.  Backward: one kernel over
// key tiles and query heads (dK, dV of the head; a small kernel sums a group's
// heads), one over query tiles (dQ), each recomputing both maps' P and dP, so
// every gradient is summed in one fixed order without atomics; 34 TFLOP/s.
#include "layer.cuh"

namespace nsp {
namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kThreads = 128;             // forward: 8 rows of 16 threads, and the group sum's
constexpr int kRows = 8;                  // forward: rows 8 ty + i of a thread

__device__ __forceinline__ float4 fma4(float s, const float4& x, const float4& y) {
  return make_float4(fmaf(s, x.x, y.x), fmaf(s, x.y, y.y), fmaf(s, x.z, y.z), fmaf(s, x.w, y.w));
}
__device__ __forceinline__ float4 scaled(float s, const float4& x) {
  return make_float4(s * x.x, s * x.y, s * x.z, s * x.w);
}
__device__ __forceinline__ float dot4(const float4& a, const float4& b, float acc) {
  return fmaf(a.w, b.w, fmaf(a.z, b.z, fmaf(a.y, b.y, fmaf(a.x, b.x, acc))));
}

__device__ __forceinline__ float4 ld4(const float* p) {
  return __ldg(reinterpret_cast<const float4*>(p));
}
__device__ __forceinline__ void st4(float* p, const float4& x) {
  *reinterpret_cast<float4*>(p) = x;
}

// ROWS rows of one head (row stride `stride` elements) into padded shared rows,
// by asynchronous copies that the caller waits for; rows at or past `end` read as
// zero.
template <int D, int ROWS, int THREADS>
__device__ __forceinline__ void load_tile(float (*dst)[D + 4], const float* src, int64_t stride,
                                          int64_t row0, int64_t end) {
#pragma unroll 4
  for (int e = threadIdx.x; e < ROWS * (D / 4); e += THREADS) {
    const int r = e / (D / 4), c = (e % (D / 4)) * 4;
    const bool in = row0 + r < end;
    const float* from = src + (in ? row0 + r : 0) * stride + c;
    const uint32_t to = (uint32_t)__cvta_generic_to_shared(&dst[r][c]);
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(to), "l"(from), "r"(in ? 16 : 0) : "memory");
  }
}
__device__ __forceinline__ void copies_wait() { asm volatile("cp.async.wait_all;" ::: "memory"); }

// Visible keys [lo, hi) of stream row t.
__device__ __forceinline__ void visible(const AttnProblem& p, int64_t t, int& lo, int& hi) {
  const int b = doc_of(p.cu, p.ndoc, t);
  lo = __ldg(p.cu + b);
  hi = p.causal ? (int)t + 1 : (int)min((int64_t)__ldg(p.cu + b + 1), p.kv_len);
}

__device__ __forceinline__ float lambda_of(const DiffProblem& a, int h, int64_t t) {
  const int64_t i = (int64_t)h * a.n_lambda + (a.n_lambda > 1 ? t : 0);
  return reinterpret_cast<const float*>(a.lambda)[i];
}

// ---------------------------------------------------------------- forward

constexpr int kFwdM = 64;

// Keys of a thread, tx + 16 j, which lie beside each other in a row of p: 4 at
// d = 64; at d = 128 shared memory holds two blocks of an SM with 2 only.
template <int D>
struct FwdSmem {
  static constexpr int kKeys = D == 64 ? 4 : 2, kN = 16 * kKeys;
  float q[kFwdM][D + 4];
  float k[kN][D + 4];
  float v[kN][D + 4];
  float p[2][kFwdM][kN + 4];
  int lo[kFwdM], hi[kFwdM];
};

// The key that column c of such a row holds.
template <int KEYS>
__device__ __forceinline__ int key_row(int c) { return c / KEYS + 16 * (c % KEYS); }

template <int D>
__global__ void __launch_bounds__(kThreads, 2) diff_fwd_simt_kernel(const DiffProblem a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  FwdSmem<D>& sm = *reinterpret_cast<FwdSmem<D>*>(smem_raw);
  const AttnProblem& p = a.p;
  if (status_bad(p.hdr)) return;
  constexpr int kCols = D / 64;                    // float4 columns of a thread
  constexpr int kKeys = FwdSmem<D>::kKeys, kN = FwdSmem<D>::kN;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int h = blockIdx.y, g = h / (p.Hq / p.Hkv);
  // longest rows first: causal tiles late in the stream see the most keys
  const int64_t row0 = (int64_t)(gridDim.x - 1 - blockIdx.x) * kFwdM;
  const int64_t T = p.q_len;
  const float* Q = reinterpret_cast<const float*>(p.q) + (int64_t)h * D;
  const float* K = reinterpret_cast<const float*>(p.k) + (int64_t)g * D;
  const float* V = reinterpret_cast<const float*>(p.v) + (int64_t)g * D;
  const int64_t qs = (int64_t)p.Hq * D, ks = (int64_t)p.Hkv * D;

  load_tile<D, kFwdM, kThreads>(sm.q, Q, qs, row0, T);
  if (threadIdx.x < kFwdM) {
    int lo = 0, hi = 0;
    if (row0 + threadIdx.x < T) visible(p, row0 + threadIdx.x, lo, hi);
    sm.lo[threadIdx.x] = lo;
    sm.hi[threadIdx.x] = hi;
  }
  __syncthreads();
  // the tile's keys: from its first row's document to its last row's end
  const int last = (int)min((int64_t)kFwdM, T - row0) - 1;
  const int key_lo = sm.lo[0] / kN * kN;
  const int key_hi = sm.hi[last];
  load_tile<D, kN, kThreads>(sm.k, K, ks, key_lo, p.kv_len);
  float m[2][kRows], l[2][kRows];
  float4 o[2][kRows][kCols];
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      m[t][i] = -INFINITY;
      l[t][i] = 0.f;
#pragma unroll
      for (int c = 0; c < kCols; ++c) o[t][i][c] = make_float4(0.f, 0.f, 0.f, 0.f);
    }
  }
  const float sl2 = p.scale * kLog2e;

  // K's buffer is filled while P V of the tile before runs, V's while S does.
  for (int j0 = key_lo; j0 < key_hi; j0 += kN) {
    copies_wait();
    __syncthreads();
    load_tile<D, kN, kThreads>(sm.v, V, ks, j0, p.kv_len);
#pragma unroll
    for (int t = 0; t < 2; ++t) {
      // scores of rows 8 ty .. + 7 against keys tx + 16 j
      float s[kRows][kKeys] = {};
#pragma unroll 2
      for (int c = t * (D / 2); c < (t + 1) * (D / 2); c += 4) {
        float4 kk[kKeys];
#pragma unroll
        for (int j = 0; j < kKeys; ++j)
          kk[j] = *reinterpret_cast<const float4*>(&sm.k[tx + 16 * j][c]);
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const float4 x = *reinterpret_cast<const float4*>(&sm.q[ty * kRows + i][c]);
#pragma unroll
          for (int j = 0; j < kKeys; ++j) s[i][j] = dot4(x, kk[j], s[i][j]);
        }
      }
#pragma unroll
      for (int i = 0; i < kRows; ++i) {
        const int lo = sm.lo[ty * kRows + i], hi = sm.hi[ty * kRows + i];
        float mx = -INFINITY;
#pragma unroll
        for (int j = 0; j < kKeys; ++j) {
          const int key = j0 + tx + 16 * j;
          s[i][j] = key >= lo && key < hi ? s[i][j] * sl2 : -INFINITY;
          mx = fmaxf(mx, s[i][j]);
        }
#pragma unroll
        for (int w = 8; w > 0; w >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, w));
        const float mn = fmaxf(m[t][i], mx);
        const float mb = mn == -INFINITY ? 0.f : mn;
        const float corr = exp2f(m[t][i] - mb);
        m[t][i] = mn;
        l[t][i] *= corr;                           // this thread's key columns only
#pragma unroll
        for (int j = 0; j < kKeys; ++j) {
          s[i][j] = exp2f(s[i][j] - mb);
          l[t][i] += s[i][j];
        }
        float* const row = &sm.p[t][ty * kRows + i][kKeys * tx];
        if constexpr (kKeys == 4) st4(row, make_float4(s[i][0], s[i][1], s[i][2], s[i][3]));
        else *reinterpret_cast<float2*>(row) = make_float2(s[i][0], s[i][1]);
#pragma unroll
        for (int c = 0; c < kCols; ++c) o[t][i][c] = scaled(corr, o[t][i][c]);
      }
    }
    copies_wait();
    __syncthreads();                                // V is there, K and P's rows are done with
    if (j0 + kN < key_hi) load_tile<D, kN, kThreads>(sm.k, K, ks, j0 + kN, p.kv_len);
#pragma unroll (D == 64 ? 4 : 2)
    for (int j = 0; j < kN; j += 4) {
      float4 v[4][kCols];
#pragma unroll
      for (int jj = 0; jj < 4; ++jj)
#pragma unroll
        for (int c = 0; c < kCols; ++c)
          v[jj][c] = *reinterpret_cast<const float4*>(&sm.v[key_row<kKeys>(j + jj)][c * 64 + tx * 4]);
#pragma unroll
      for (int t = 0; t < 2; ++t)
#pragma unroll
        for (int i = 0; i < kRows; ++i) {
          const float4 w = *reinterpret_cast<const float4*>(&sm.p[t][ty * kRows + i][j]);
#pragma unroll
          for (int c = 0; c < kCols; ++c)
            o[t][i][c] = fma4(w.w, v[3][c], fma4(w.z, v[2][c], fma4(w.y, v[1][c],
                              fma4(w.x, v[0][c], o[t][i][c]))));
        }
    }
  }
  copies_wait();                                // a tile that sees no key has copies in flight

  float* O = reinterpret_cast<float*>(p.out);
  float* O2 = reinterpret_cast<float*>(a.out2);
#pragma unroll
  for (int i = 0; i < kRows; ++i) {
    const int64_t row = row0 + ty * kRows + i;
    float inv[2];
#pragma unroll
    for (int t = 0; t < 2; ++t) {
#pragma unroll
      for (int w = 8; w > 0; w >>= 1) l[t][i] += __shfl_xor_sync(0xffffffffu, l[t][i], w);
      inv[t] = l[t][i] > 0.f ? 1.f / l[t][i] : 0.f;
      if (row < T && tx == 0 && p.lse != nullptr)
        p.lse[((int64_t)h * 2 + t) * T + row] = (m[t][i] + log2f(l[t][i])) * kLn2;
    }
    if (row >= T) continue;
    const float lam = lambda_of(a, h, row);
#pragma unroll
    for (int c = 0; c < kCols; ++c) {
      const int64_t off = row * qs + (int64_t)h * D + c * 64 + tx * 4;
      const float4 x = o[0][i][c], y = o[1][i][c];
      const float4 o2 = make_float4(y.x * inv[1], y.y * inv[1], y.z * inv[1], y.w * inv[1]);
      st4(O + off, make_float4(x.x * inv[0] - lam * o2.x, x.y * inv[0] - lam * o2.y,
                               x.z * inv[0] - lam * o2.z, x.w * inv[0] - lam * o2.w));
      if (O2 != nullptr) st4(O2 + off, o2);
    }
  }
}

// ---------------------------------------------------------------- backward

template <int D>
constexpr int kBwdRows = D == 64 ? 8 : 4;          // rows of a thread, by 4 keys
template <int D>
constexpr int kBwdThreads = 1024 / kBwdRows<D>;
constexpr int kBwdTile = 64;          // query rows and keys of a tile

template <int D>
struct BwdSmem {
  float q[kBwdTile][D + 4], dout[kBwdTile][D + 4];
  float k[kBwdTile][D + 4], v[kBwdTile][D + 4];
  float ds[2][kBwdTile][kBwdTile + 4];            // [map][row of the output][summed index]
  float nlse2[2][kBwdTile], ndelta[2][kBwdTile], coef[kBwdTile];
  int lo[kBwdTile], hi[kBwdTile];
};

// dS of a tile, written for the product that follows: KEY puts it in rows of
// keys (dK), otherwise in rows of queries (dQ); pc: P_1 - lambda P_2 of the thread's
// rows (kBwdRows ty + i) and keys tx + 16 j.  A row of queries holds a thread's
// keys beside each other, as key_row tells.
template <int D, bool KEY>
__device__ __forceinline__ void tile_ds(BwdSmem<D>& sm, int64_t key0, float sl2, float (&pc)[4][kBwdRows<D>]) {
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  float s[2][kBwdRows<D>][4] = {}, dp[kBwdRows<D>][4] = {};
#pragma unroll
  for (int t = 0; t < 2; ++t)
#pragma unroll 1
    for (int c = t * (D / 2); c < (t + 1) * (D / 2); c += 4) {
      float4 kk[4], vv[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        kk[j] = *reinterpret_cast<const float4*>(&sm.k[tx + 16 * j][c]);
        vv[j] = *reinterpret_cast<const float4*>(&sm.v[tx + 16 * j][c]);
      }
#pragma unroll
      for (int i = 0; i < kBwdRows<D>; ++i) {
        const float4 x = *reinterpret_cast<const float4*>(&sm.q[ty * kBwdRows<D> + i][c]);
        const float4 y = *reinterpret_cast<const float4*>(&sm.dout[ty * kBwdRows<D> + i][c]);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
          s[t][i][j] = dot4(x, kk[j], s[t][i][j]);
          dp[i][j] = dot4(y, vv[j], dp[i][j]);
        }
      }
    }
#pragma unroll
  for (int i = 0; i < kBwdRows<D>; ++i) {
    const int r = ty * kBwdRows<D> + i;
    const int lo = sm.lo[r], hi = sm.hi[r];
    const float n0 = sm.nlse2[0][r], n1 = sm.nlse2[1][r], co = sm.coef[r];
    const float e0 = sm.ndelta[0][r], e1 = sm.ndelta[1][r];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const int64_t key = key0 + tx + 16 * j;
      const bool vis = key >= lo && key < hi;
      const float p1 = vis ? exp2f(fmaf(s[0][i][j], sl2, n0)) : 0.f;
      const float p2 = vis ? co * exp2f(fmaf(s[1][i][j], sl2, n1)) : 0.f;
      s[0][i][j] = vis ? p1 * (dp[i][j] + e0) : 0.f;
      s[1][i][j] = vis ? p2 * (dp[i][j] + e1) : 0.f;
      pc[j][i] = p1 + p2;
    }
  }
#pragma unroll
  for (int t = 0; t < 2; ++t)
    if constexpr (KEY) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        const int kk = tx + 16 * j;
#pragma unroll
        for (int i = 0; i < kBwdRows<D>; i += 4)
          st4(&sm.ds[t][kk][ty * kBwdRows<D> + i],
              make_float4(s[t][i][j], s[t][i + 1][j], s[t][i + 2][j], s[t][i + 3][j]));
      }
    } else {
#pragma unroll
      for (int i = 0; i < kBwdRows<D>; ++i)
        st4(&sm.ds[t][ty * kBwdRows<D> + i][4 * tx], make_float4(s[t][i][0], s[t][i][1], s[t][i][2], s[t][i][3]));
    }
}

// acc[i][c] += sum_j w[kBwdRows ty + i][j] x[j][col + 64 c]: a kBwdTile x D product of
// a square tile in shared memory; w_of picks the tile of the column's map.
template <int D, bool KEY, typename W>
__device__ __forceinline__ void tile_product(float4 (&acc)[kBwdRows<D>][D / 64], W&& w_of, float (*x)[D + 4]) {
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
#pragma unroll 4
  for (int j = 0; j < kBwdTile; j += 4) {
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      const int col = c * 64 + tx * 4;
      float4 b[4];
#pragma unroll
      for (int jj = 0; jj < 4; ++jj)
        b[jj] = *reinterpret_cast<const float4*>(&x[KEY ? j + jj : key_row<4>(j + jj)][col]);
#pragma unroll
      for (int i = 0; i < kBwdRows<D>; ++i) {
        const float4 w = *reinterpret_cast<const float4*>(w_of(col) + (ty * kBwdRows<D> + i) * (kBwdTile + 4) + j);
        acc[i][c] = fma4(w.w, b[3], fma4(w.z, b[2], fma4(w.y, b[1], fma4(w.x, b[0], acc[i][c]))));
      }
    }
  }
}

template <int D>
__device__ __forceinline__ void load_rows(BwdSmem<D>& sm, const DiffProblem& a, int h, int64_t row0) {
  const AttnProblem& p = a.p;
  const int r = threadIdx.x;
  if (r >= kBwdTile) return;
  const int64_t t = row0 + r;
  int lo = 0, hi = 0;
  if (t < p.q_len) {
    visible(p, t, lo, hi);
#pragma unroll
    for (int m = 0; m < 2; ++m) {
      sm.nlse2[m][r] = a.nlse2[((int64_t)h * 2 + m) * a.Tp + t];
      sm.ndelta[m][r] = a.ndelta[((int64_t)h * 2 + m) * a.Tp + t];
    }
    sm.coef[r] = a.coef[(int64_t)h * a.Tp + t];
  }
  sm.lo[r] = lo;
  sm.hi[r] = hi;
}

// One query head's share of dK and dV for a key tile: summed over the group's
// heads by diff_group_sum_kernel (one block a head, so that few key tiles still
// fill the GPU), or written at once when the group is one head.
template <int D>
__global__ void __launch_bounds__(kBwdThreads<D>, D == 64 ? 2 : 1) diff_bwd_dkdv_simt_kernel(const DiffProblem a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  BwdSmem<D>& sm = *reinterpret_cast<BwdSmem<D>*>(smem_raw);
  const AttnProblem& p = a.p;
  if (status_bad(p.hdr)) return;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int h = blockIdx.y, G = p.Hq / p.Hkv, g = h / G;
  const int64_t T = p.q_len, key0 = (int64_t)blockIdx.x * kBwdTile;
  const int64_t qs = (int64_t)p.Hq * D, ks = (int64_t)p.Hkv * D;
  load_tile<D, kBwdTile, kBwdThreads<D>>(sm.k, reinterpret_cast<const float*>(p.k) + (int64_t)g * D, ks, key0, T);
  load_tile<D, kBwdTile, kBwdThreads<D>>(sm.v, reinterpret_cast<const float*>(p.v) + (int64_t)g * D, ks, key0, T);
  const int64_t key1 = min(key0 + kBwdTile, T) - 1;
  const int b0 = doc_of(p.cu, p.ndoc, key0), b1 = doc_of(p.cu, p.ndoc, key1);
  const int64_t r_lo = p.causal ? key0 : (int64_t)__ldg(p.cu + b0);
  const int64_t r_hi = min((int64_t)__ldg(p.cu + b1 + 1), T);
  float4 dk[kBwdRows<D>][D / 64] = {}, dv[kBwdRows<D>][D / 64] = {};
  const float* const Q = reinterpret_cast<const float*>(p.q) + (int64_t)h * D;
  load_tile<D, kBwdTile, kBwdThreads<D>>(sm.q, Q, qs, r_lo, T);
  for (int64_t r0 = r_lo; r0 < r_hi; r0 += kBwdTile) {
    __syncthreads();
    load_tile<D, kBwdTile, kBwdThreads<D>>(sm.dout, reinterpret_cast<const float*>(a.dout) + (int64_t)h * D, qs, r0, T);
    load_rows<D>(sm, a, h, r0);
    copies_wait();
    __syncthreads();
    float pc[4][kBwdRows<D>];
    tile_ds<D, true>(sm, key0, p.scale * kLog2e, pc);
    __syncthreads();
    tile_product<D, true>(dk, [&](int col) { return &sm.ds[col >= D / 2][0][0]; }, sm.q);
    __syncthreads();
    // the next tile's queries arrive while dV's product runs
    if (r0 + kBwdTile < r_hi) load_tile<D, kBwdTile, kBwdThreads<D>>(sm.q, Q, qs, r0 + kBwdTile, T);
    // P over dS (a buffer of its own would leave room for one block of an SM only)
#pragma unroll
    for (int j = 0; j < 4; ++j)
#pragma unroll
      for (int i = 0; i < kBwdRows<D>; i += 4)
        st4(&sm.ds[0][tx + 16 * j][ty * kBwdRows<D> + i],
            make_float4(pc[j][i], pc[j][i + 1], pc[j][i + 2], pc[j][i + 3]));
    __syncthreads();
    tile_product<D, true>(dv, [&](int) { return &sm.ds[0][0][0]; }, sm.dout);
  }
  copies_wait();
  float* const DK = G > 1 ? a.dk_heads : reinterpret_cast<float*>(a.dk);
  float* const DV = G > 1 ? a.dv_heads : reinterpret_cast<float*>(a.dv);
#pragma unroll
  for (int i = 0; i < kBwdRows<D>; ++i) {
    const int64_t key = key0 + ty * kBwdRows<D> + i;
    if (key >= T) continue;
#pragma unroll
    for (int c = 0; c < D / 64; ++c) {
      const int64_t off = key * qs + (int64_t)h * D + c * 64 + tx * 4;
      st4(DK + off, scaled(p.scale, dk[i][c]));
      st4(DV + off, dv[i][c]);
    }
  }
}

// dk, dv [T, Hkv, d] = sums over each group's G heads of [T, Hq, d], in order.
__global__ void __launch_bounds__(kThreads) diff_group_sum_kernel(const DiffProblem a) {
  const AttnProblem& p = a.p;
  if (status_bad(p.hdr)) return;
  const int G = p.Hq / p.Hkv, d4 = p.d / 4;
  const int64_t n = p.q_len * p.Hkv * d4;
  for (int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x; e < 2 * n;
       e += (int64_t)gridDim.x * kThreads) {
    const bool is_v = e >= n;
    const int64_t i = is_v ? e - n : e, tg = i / d4;
    const float* src = (is_v ? a.dv_heads : a.dk_heads) + (tg * G * d4 + (i - tg * d4)) * 4;
    float4 x = ld4(src);
    for (int h = 1; h < G; ++h) x = fma4(1.f, ld4(src + (int64_t)h * p.d), x);
    st4(reinterpret_cast<float*>(is_v ? a.dv : a.dk) + i * 4, x);
  }
}

template <int D>
__global__ void __launch_bounds__(kBwdThreads<D>, D == 64 ? 2 : 1) diff_bwd_dq_simt_kernel(const DiffProblem a) {
  extern __shared__ __align__(16) unsigned char smem_raw[];
  BwdSmem<D>& sm = *reinterpret_cast<BwdSmem<D>*>(smem_raw);
  const AttnProblem& p = a.p;
  if (status_bad(p.hdr)) return;
  const int ty = threadIdx.x >> 4, tx = threadIdx.x & 15;
  const int h = blockIdx.y, g = h / (p.Hq / p.Hkv);
  const int64_t T = p.q_len, row0 = (int64_t)(gridDim.x - 1 - blockIdx.x) * kBwdTile;
  const int64_t qs = (int64_t)p.Hq * D, ks = (int64_t)p.Hkv * D;
  load_tile<D, kBwdTile, kBwdThreads<D>>(sm.q, reinterpret_cast<const float*>(p.q) + (int64_t)h * D, qs, row0, T);
  load_tile<D, kBwdTile, kBwdThreads<D>>(sm.dout, reinterpret_cast<const float*>(a.dout) + (int64_t)h * D, qs, row0, T);
  load_rows<D>(sm, a, h, row0);
  __syncthreads();
  const int last = (int)min((int64_t)kBwdTile, T - row0) - 1;
  const int key_lo = sm.lo[0] / kBwdTile * kBwdTile, key_hi = sm.hi[last];
  float4 dq[kBwdRows<D>][D / 64] = {};
  const float* const V = reinterpret_cast<const float*>(p.v) + (int64_t)g * D;
  load_tile<D, kBwdTile, kBwdThreads<D>>(sm.v, V, ks, key_lo, T);
  for (int j0 = key_lo; j0 < key_hi; j0 += kBwdTile) {
    __syncthreads();
    load_tile<D, kBwdTile, kBwdThreads<D>>(sm.k, reinterpret_cast<const float*>(p.k) + (int64_t)g * D, ks, j0, T);
    copies_wait();
    __syncthreads();
    float pc[4][kBwdRows<D>];
    tile_ds<D, false>(sm, j0, p.scale * kLog2e, pc);
    __syncthreads();
    // the next tile's values arrive while the product runs
    if (j0 + kBwdTile < key_hi) load_tile<D, kBwdTile, kBwdThreads<D>>(sm.v, V, ks, j0 + kBwdTile, T);
    tile_product<D, false>(dq, [&](int col) { return &sm.ds[col >= D / 2][0][0]; }, sm.k);
  }
  copies_wait();                                   // of a tile that sees no key
#pragma unroll
  for (int i = 0; i < kBwdRows<D>; ++i) {
    const int64_t row = row0 + ty * kBwdRows<D> + i;
    if (row >= T) continue;
#pragma unroll
    for (int c = 0; c < D / 64; ++c)
      st4(reinterpret_cast<float*>(a.dq) + row * qs + (int64_t)h * D + c * 64 + tx * 4,
          scaled(p.scale, dq[i][c]));
  }
}

template <typename K>
cudaError_t launch(K kern, dim3 grid, int threads, size_t smem, const DiffProblem& a, cudaStream_t s) {
  cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
  if (e != cudaSuccess) return e;
  kern<<<grid, threads, smem, s>>>(a);
  count_launches(1);
  count_path(false);
  return cudaGetLastError();
}

template <int D>
cudaError_t fwd(const DiffProblem& a, cudaStream_t s) {
  const dim3 grid((unsigned)ceil_div(a.p.q_len, kFwdM), a.p.Hq);
  return launch(diff_fwd_simt_kernel<D>, grid, kThreads, sizeof(FwdSmem<D>), a, s);
}

template <int D>
cudaError_t bwd(const DiffProblem& a, cudaStream_t s) {
  const dim3 grid((unsigned)ceil_div(a.p.q_len, kBwdTile), a.p.Hq);
  cudaError_t e = launch(diff_bwd_dkdv_simt_kernel<D>, grid, kBwdThreads<D>, sizeof(BwdSmem<D>), a, s);
  if (e != cudaSuccess) return e;
  if (a.p.Hq > a.p.Hkv) {
    const int64_t n = 2 * a.p.q_len * a.p.Hkv * (D / 4);
    const int64_t blocks = ceil_div(n, kThreads), most = (int64_t)num_sms() * 8;
    diff_group_sum_kernel<<<(unsigned)(blocks < most ? blocks : most), kThreads, 0, s>>>(a);
    count_launches(1);
    e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return launch(diff_bwd_dq_simt_kernel<D>, grid, kBwdThreads<D>, sizeof(BwdSmem<D>), a, s);
}

}  // namespace

cudaError_t launch_diff_fwd_simt(const DiffProblem& a, cudaStream_t s) {
  return a.p.d == 128 ? fwd<128>(a, s) : fwd<64>(a, s);
}

cudaError_t launch_diff_bwd_simt(const DiffProblem& a, cudaStream_t s) {
  return a.p.d == 128 ? bwd<128>(a, s) : bwd<64>(a, s);
}

}  // namespace nsp
