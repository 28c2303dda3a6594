// Root-mean-square norm of every query and key head with the rotation by its
// token's position in the same pass:
//   r = 1 / sqrt(mean(x^2) + eps),  n = x r,  y = R(w n),
// R the rotation of rope.cu (its factor included), and the backward, with
// z = R^T dy and u = w z:
//   dx = r (u - n mean(u n)),  dw = sum over rows of n z.
//
// Bound: HBM, one read of x (and dy) and one write of y (dx).  A head's row lives in the
// registers of a team of lanes, two 16-byte vectors a lane, reduced by shuffles; a token's
// sines and cosines are computed once for all its heads, with the weights multiplied in.
// The forward gives a team a part of a token and has four heads in flight; the backward,
// with both weights' columns and their sums in registers as well, has its rows copied
// ahead into shared memory, and every warp takes as many rows as the others.  32768
// tokens, 32 + 4 heads of 128 bf16 columns out of a fused projection: 98 us a call, 6.2
// TB/s (three launches of norms and rotation move twice the bytes); backward 176 us, 5.1
// TB/s: its 15 instructions an element keep 44 % of the issue slots, and warps wait for
// shuffles and reciprocal roots more than for memory.
#include <algorithm>

#include "tc_ptx.cuh"
#include "train.cuh"

namespace nsp {
namespace {

using namespace tc;

constexpr int kThreads = 256;
constexpr int kVecThreads = 128;
constexpr int kWarps = kThreads / 32;
constexpr int64_t kL2Bytes = (int64_t)128 << 20;
constexpr int kBwdBlocks = 304;          // three blocks of an SM: 288 us of the backward above (spills)

__device__ __forceinline__ float warp_sum(float x) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
  return x;
}

// The blocks of a grid that a tensor's rows are given to, and the parts that a token's
// heads are split in there.
struct Share {
  int first[kRopeMaxTensors + 1];
  int hsplit[kRopeMaxTensors], per[kRopeMaxTensors];
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

// ---- whole 16-byte pieces
//
// A team of lanes owns a token's heads (or a part of them) and computes the sines and
// cosines of its pairs once; a lane holds U units of two 16-byte vectors of a head: both
// halves of its pairs, or any two.  The weights enter the turn's coefficients, so
// that a pair costs two products, two FMAs and the row's factor.

// The columns of a lane's unit; `second`: its second vector is there; turned: bit v, vector
// v's pairs are rotated.  (Neighbouring lanes' vectors are neighbours in memory: lanes 32
// bytes apart would take half of every sector they touch.)
template <int N, bool INTER>
__device__ __forceinline__ bool unit_of(int d, int rot, int u, int& c0, int& c1, bool& second, int& turned) {
  const int r = INTER ? 0 : rot / 2 / N;
  if (u >= r) {
    const int first = INTER ? 0 : rot, vecs = (d - first) / N, half = (vecs + 1) / 2, v = u - r;
    c0 = first + v * N;
    c1 = c0 + half * N;
    second = v + half < vecs;
    turned = INTER ? (c0 < rot ? 1 : 0) | (c1 < rot ? 2 : 0) : 0;
    return v < half;
  }
  c0 = u * N;
  c1 = c0 + rot / 2;
  second = true;
  turned = 3;
  return true;
}

// A lane's part of a head: its units' columns, and which of their vectors there are.
template <int N, bool INTER, int LANES, int U>
struct Units {
  int c0[U], c1[U], turned[U];
  bool first[U], second[U];

  __device__ __forceinline__ Units(const QkArgs& a, int lane) {
#pragma unroll
    for (int i = 0; i < U; ++i) {
      first[i] = unit_of<N, INTER>(a.d, a.rot, lane + i * LANES, c0[i], c1[i], second[i], turned[i]);
      second[i] = second[i] && first[i];
      if (!first[i]) turned[i] = 0;
    }
  }
};

// Sum over a team of LANES lanes, which meet here together.
template <int LANES>
__device__ __forceinline__ float team_sum(float x, uint32_t mask) {
#pragma unroll
  for (int o = LANES >> 1; o > 0; o >>= 1) x += __shfl_xor_sync(mask, x, o);
  return x;
}
template <int LANES>
__device__ __forceinline__ uint32_t team_mask() {
  return LANES == 32 ? 0xffffffffu : ((1u << (LANES & 31)) - 1) << (threadIdx.x & 31 & ~(LANES - 1));
}

// A vector's values as packed pairs.
template <typename T>
__device__ __forceinline__ void unpack2(const uint4& u, uint64_t* x) {
  float t[Vec<T>::N];
  Vec<T>::unpack(u, t);
#pragma unroll
  for (int i = 0; i < Vec<T>::N / 2; ++i) x[i] = f2_pack(t[2 * i], t[2 * i + 1]);
}
template <typename T>
__device__ __forceinline__ uint4 pack2(const uint64_t* x) {
  float t[Vec<T>::N];
#pragma unroll
  for (int i = 0; i < Vec<T>::N / 2; ++i) f2_unpack(x[i], t[2 * i], t[2 * i + 1]);
  return Vec<T>::pack(t);
}
__device__ __forceinline__ uint64_t swap2(uint64_t x) {
  float a, b;
  f2_unpack(x, a, b);
  return f2_pack(b, a);
}
__device__ __forceinline__ float sum2(uint64_t x) {
  float a, b;
  f2_unpack(x, a, b);
  return a + b;
}

// Cosines and sines of a unit's pairs: halves: pair j of both vectors; neighbours: pairs j
// of the first, N / 2 + j of the second.  Columns that are not rotated: 1 and 0.
template <int N, bool INTER>
__device__ __forceinline__ void turns(const QkArgs& a, const uint64_t* s_fx, int64_t pos, int c0, int c1,
                                      int turned, bool inverse, float (&c)[N], float (&s)[N]) {
#pragma unroll
  for (int j = 0; j < N; ++j) {
    c[j] = 1.f;
    s[j] = 0.f;
    const bool on = INTER ? (turned >> (j >= N / 2 ? 1 : 0)) & 1 : turned != 0;
    const int pair = INTER ? (j < N / 2 ? c0 / 2 + j : c1 / 2 + j - N / 2) : c0 + j;
    if (on) turn(pos, s_fx[pair], a.mscale, inverse, c[j], s[j]);
  }
}

template <typename T, int N>
__device__ __forceinline__ void load_weight(const void* w, int col, bool there, float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) x[i] = 1.f;
  if (w != nullptr && there) Vec<T>::unpack(__ldg(reinterpret_cast<const uint4*>(reinterpret_cast<const T*>(w) + col)), x);
}

// Where a team's part of a token's heads begins; the part lies in one head group.
struct Item {
  int64_t t;
  int h0, h1;
};
__device__ __forceinline__ Item item_of(const QkTensor& q, int64_t item, int hsplit, int per) {
  Item m;
  m.t = hsplit == 1 ? item : (int64_t)((uint32_t)item / (uint32_t)hsplit);
  m.h0 = (int)(item - m.t * hsplit) * per;
  m.h1 = min(m.h0 + per, q.heads);
  return m;
}

template <typename T, bool INTER, int LANES, int U>
__global__ void __launch_bounds__(kVecThreads, U == 1 ? 4 : 2) qk_vec_kernel(const __grid_constant__ QkArgs a,
                                                                             const Share share) {
  constexpr int N = Vec<T>::N, P = N / 2, kFlight = U == 1 ? 4 : 2, kTeams = kVecThreads / LANES;
  __shared__ uint64_t s_fx[kQkMaxDim / 2];
  for (int i = threadIdx.x; i < a.rot / 2; i += kVecThreads) s_fx[i] = fixed_turns(a.freqs[i]);
  __syncthreads();
  int k = 0;
  while ((int)blockIdx.x >= share.first[k + 1]) ++k;
  const QkTensor& q = a.t[k];
  const int lane = threadIdx.x % LANES, team = threadIdx.x / LANES;
  const uint32_t mask = team_mask<LANES>();
  const Units<N, INTER, LANES, U> un(a, lane);
  const int hsplit = share.hsplit[k], per = share.per[k];
  const int64_t items = a.len * hsplit;
  const float inv_d = 1.f / (float)a.d;
  const int64_t step = (int64_t)(share.first[k + 1] - share.first[k]) * kTeams;
  for (int64_t item = (int64_t)(blockIdx.x - share.first[k]) * kTeams + team; item < items; item += step) {
    const Item m = item_of(q, item, hsplit, per);
    const T* x = reinterpret_cast<const T*>(q.x) + m.t * q.x_stride + (int64_t)m.h0 * a.d;
    T* y = reinterpret_cast<T*>(q.y) + row_offset(m.t, m.h0, q.y_stride, q.heads, q.groups, a.len, a.d);
    bool ready = false;
    uint64_t ca[U][N], cb[U][N];             // [P] for the first output vector, [P] for the second
    for (int h = m.h0; h < m.h1; h += kFlight) {
      uint4 v[kFlight][U][2];
#pragma unroll
      for (int f = 0; f < kFlight; ++f) {
        const T* const row = x + f * a.d;
#pragma unroll
        for (int i = 0; i < U; ++i) {
          v[f][i][0] = v[f][i][1] = make_uint4(0, 0, 0, 0);
          if (h + f < m.h1 && un.first[i]) v[f][i][0] = ld_once(row + un.c0[i]);
          if (h + f < m.h1 && un.second[i]) v[f][i][1] = ld_once(row + un.c1[i]);
        }
      }
      if (!ready) {                          // under the first loads
        int64_t pos;
        if (!position_of(Positions{a.positions, a.cu, a.ndoc, a.start}, m.t, pos)) break;
        ready = true;
#pragma unroll
        for (int i = 0; i < U; ++i) {
          float c[N], s[N], w0[N], w1[N];
          turns<N, INTER>(a, s_fx, pos, un.c0[i], un.c1[i], un.turned[i], false, c, s);
          load_weight<T>(q.weight, un.c0[i], un.first[i], w0);
          load_weight<T>(q.weight, un.c1[i], un.second[i], w1);
#pragma unroll
          for (int j = 0; j < P; ++j) {
            if constexpr (INTER) {
              // out = (x_even, x_odd) ca + (x_odd, x_even) cb
              ca[i][j] = f2_pack(w0[2 * j] * c[j], w0[2 * j + 1] * c[j]);
              cb[i][j] = f2_pack(-w0[2 * j + 1] * s[j], w0[2 * j] * s[j]);
              ca[i][P + j] = f2_pack(w1[2 * j] * c[P + j], w1[2 * j + 1] * c[P + j]);
              cb[i][P + j] = f2_pack(-w1[2 * j + 1] * s[P + j], w1[2 * j] * s[P + j]);
            } else {
              // out0 = x0 ca + x1 cb, out1 = x1 ca' + x0 cb'
              ca[i][j] = f2_pack(w0[2 * j] * c[2 * j], w0[2 * j + 1] * c[2 * j + 1]);
              cb[i][j] = f2_pack(-w1[2 * j] * s[2 * j], -w1[2 * j + 1] * s[2 * j + 1]);
              ca[i][P + j] = f2_pack(w1[2 * j] * c[2 * j], w1[2 * j + 1] * c[2 * j + 1]);
              cb[i][P + j] = f2_pack(w0[2 * j] * s[2 * j], w0[2 * j + 1] * s[2 * j + 1]);
            }
          }
        }
      }
      float r[kFlight];
#pragma unroll
      for (int f = 0; f < kFlight; ++f) {
        uint64_t ss = 0;
#pragma unroll
        for (int i = 0; i < U; ++i) {
          uint64_t e[N];
          unpack2<T>(v[f][i][0], e);
          unpack2<T>(v[f][i][1], e + P);
#pragma unroll
          for (int j = 0; j < N; ++j) ss = f2_fma(e[j], e[j], ss);
        }
        r[f] = sum2(ss);
      }
#pragma unroll
      for (int f = 0; f < kFlight; ++f) r[f] = rsqrtf(fmaf(team_sum<LANES>(r[f], mask), inv_d, a.eps));
#pragma unroll
      for (int f = 0; f < kFlight; ++f) {
        if (h + f >= m.h1) break;
        const uint64_t r2 = f2_pack(r[f], r[f]);
        T* const row = y + f * a.d;
#pragma unroll
        for (int i = 0; i < U; ++i) {
          uint64_t e[N], o[N];
          unpack2<T>(v[f][i][0], e);
          unpack2<T>(v[f][i][1], e + P);
#pragma unroll
          for (int j = 0; j < N; ++j) {
            const uint64_t other = INTER ? swap2(e[j]) : e[j < P ? j + P : j - P];
            o[j] = f2_mul(f2_fma(other, cb[i][j], f2_mul(e[j], ca[i][j])), r2);
          }
          if (un.first[i]) st_once(row + un.c0[i], pack2<T>(o));
          if (un.second[i]) st_once(row + un.c1[i], pack2<T>(o + P));
        }
      }
      x += kFlight * a.d;
      y += kFlight * a.d;
    }
  }
}

// The backward's rows come through a ring in shared memory: a thread copies its own
// vectors of the heads ahead, kAhead of them at any time (4: the same), and reads only what
// it copied itself.  (The next head in registers: 183 us of the case above.)
constexpr int kAhead = 6;
template <int U> constexpr int bwd_ring_bytes() { return kAhead / U * U * 4 * 16 * kThreads; }

__device__ __forceinline__ void copy16(uint4* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}

// A warp's rows of a tensor, `row` to `end` of them: the heads of TOKENS tokens at a time,
// a team each, which turn to their next tokens together; all warps have as many, give or
// take one.  Rows behind the last document (at `live`) are nobody's.
template <int TOKENS>
struct WarpRows {
  int64_t live, row, end;

  __device__ __forceinline__ WarpRows(const QkArgs& a, const QkTensor& q, int64_t warp, int64_t warps) {
    live = a.len;
    if (a.positions == nullptr)
      live = max((int64_t)0, min(live, (int64_t)__ldg(a.cu + a.ndoc) - a.start));
    const int64_t rows = (live + TOKENS - 1) / TOKENS * q.heads, each = rows / warps;
    const int64_t more = rows - each * warps;
    row = warp * each + min(warp, more);
    end = row + each + (warp < more ? 1 : 0);
  }
};

// Positions of a team's tokens: a search where a document ends.
struct PositionWalk {
  int64_t start = 0, end = 0;
  __device__ __forceinline__ int64_t of(const QkArgs& a, int64_t t) {
    if (a.positions != nullptr) return __ldg(a.positions + t);
    const int64_t g = a.start + t;
    if (g >= end) {
      const int doc = doc_of(a.cu, a.ndoc, g);
      start = __ldg(a.cu + doc);
      end = __ldg(a.cu + doc + 1);
    }
    return g - start;
  }
};

template <typename T, int U, int TOKENS, typename UNITS>
struct HeadCopies {
  const QkArgs& a;
  const QkTensor& q;
  const UNITS& un;
  const int64_t live;
  int64_t left, t;                                 // rows that are not copied yet; token of the next
  int h;
  const T *x, *dy;

  __device__ __forceinline__ HeadCopies(const QkArgs& a, const QkTensor& q, const UNITS& un,
                                        const WarpRows<TOKENS>& rows, int64_t t, int h)
      : a(a), q(q), un(un), live(rows.live), left(t < live ? rows.end - rows.row : 0), t(t), h(h) {
    x = reinterpret_cast<const T*>(q.x) + t * q.x_stride + (int64_t)h * a.d;
    find();
  }
  __device__ __forceinline__ void find() {
    dy = reinterpret_cast<const T*>(q.dy) + row_offset(t, h, q.y_stride, q.heads, q.groups, a.len, a.d);
  }
  // the next head into the four places (of every unit) from `to` on
  __device__ __forceinline__ void copy(uint4* to) {
    if (left > 0) {
#pragma unroll
      for (int i = 0; i < U; ++i) {
        uint4* const p = to + i * 4 * kThreads;
        if (un.first[i]) {
          copy16(p, x + un.c0[i]);
          copy16(p + 2 * kThreads, dy + un.c0[i]);
        }
        if (un.second[i]) {
          copy16(p + kThreads, x + un.c1[i]);
          copy16(p + 3 * kThreads, dy + un.c1[i]);
        }
      }
      --left;
      x += a.d;
      dy += a.d;
      if (++h == q.heads) {
        h = 0;
        t += TOKENS;
        x += TOKENS * q.x_stride - (int64_t)q.heads * a.d;
        if (t >= live) left = 0;
        if (left > 0) find();
      } else if (q.groups > 1 && left > 0) {
        find();
      }
    }
    asm volatile("cp.async.commit_group;" ::: "memory");
  }
};

template <typename T, bool INTER, int LANES, int U>
__global__ void __launch_bounds__(kThreads, U == 1 ? 2 : 1) qk_vec_bwd_kernel(const __grid_constant__ QkArgs a,
                                                                              const Share share) {
  constexpr int N = Vec<T>::N, P = N / 2, kTeams = kThreads / LANES, kHeads = kAhead / U, kTokens = 32 / LANES;
  using UnitsOf = Units<N, INTER, LANES, U>;
  extern __shared__ __align__(16) uint4 s_ring[];  // [kHeads][U][4][kThreads]; in the end [kTeams][d] sums
  __shared__ uint64_t s_fx[kQkMaxDim / 2];
  grid_dep_trigger();
  int k = 0;
  while ((int)blockIdx.x >= share.first[k + 1]) ++k;
  const QkTensor& q = a.t[k];
  const int lane = threadIdx.x % LANES, team = threadIdx.x / LANES;
  const uint32_t mask = team_mask<LANES>();
  const UnitsOf un(a, lane);
  const float inv_d = 1.f / (float)a.d;
  const WarpRows<kTokens> rows(a, q, (int64_t)(blockIdx.x - share.first[k]) * kWarps + threadIdx.x / 32,
                               (int64_t)(share.first[k + 1] - share.first[k]) * kWarps);
  int64_t t = rows.row / q.heads;                  // (of the warp's groups of tokens)
  int h = (int)(rows.row - t * q.heads);
  t = t * kTokens + team % kTokens;
  uint4* const ring = s_ring + threadIdx.x;
  // (vectors that a lane does not have are never copied: zeros)
  for (int i = 0; i < kHeads * U * 4; ++i) ring[i * kThreads] = make_uint4(0, 0, 0, 0);
  HeadCopies<T, U, kTokens, UnitsOf> ahead(a, q, un, rows, t, h);
#pragma unroll
  for (int i = 0; i < kHeads; ++i) ahead.copy(ring + i * U * 4 * kThreads);
  for (int i = threadIdx.x; i < a.rot / 2; i += kThreads) s_fx[i] = fixed_turns(a.freqs[i]);
  __syncthreads();
  uint64_t w[U][N], dw[U][N];                      // [P] of the first vector, [P] of the second
#pragma unroll
  for (int i = 0; i < U; ++i) {
    float t[N];
    load_weight<T>(q.weight, un.c0[i], un.first[i], t);
#pragma unroll
    for (int j = 0; j < P; ++j) w[i][j] = f2_pack(t[2 * j], t[2 * j + 1]);
    load_weight<T>(q.weight, un.c1[i], un.second[i], t);
#pragma unroll
    for (int j = 0; j < P; ++j) w[i][P + j] = f2_pack(t[2 * j], t[2 * j + 1]);
#pragma unroll
    for (int j = 0; j < N; ++j) dw[i][j] = 0;
  }
  int slot = 0;
  PositionWalk at;
  for (int64_t row = rows.row; row < rows.end && t < rows.live; t += kTokens, h = 0) {
    const int h1 = (int)min((int64_t)q.heads, h + (rows.end - row));
    row += h1 - h;
    const int64_t pos = at.of(a, t);
    T* dx = reinterpret_cast<T*>(q.dx) + t * q.dx_stride + (int64_t)h * a.d;
    // halves: c and s of the pairs, packed; neighbours: (c, c) and (-s, s) of each
    uint64_t c2[U][INTER ? N : P], s2[U][INTER ? N : P];
#pragma unroll
    for (int i = 0; i < U; ++i) {
      float c[N], s[N];
      turns<N, INTER>(a, s_fx, pos, un.c0[i], un.c1[i], un.turned[i], true, c, s);
      if constexpr (INTER) {
#pragma unroll
        for (int j = 0; j < N; ++j) {
          c2[i][j] = f2_pack(c[j], c[j]);
          s2[i][j] = f2_pack(-s[j], s[j]);
        }
      } else {
#pragma unroll
        for (int j = 0; j < P; ++j) {
          c2[i][j] = f2_pack(c[2 * j], c[2 * j + 1]);
          s2[i][j] = f2_pack(s[2 * j], s[2 * j + 1]);
        }
      }
    }
    for (; h < h1; ++h) {
      uint64_t xs[U][N], z[U][N], ss = 0, su = 0;
      uint4* const place = ring + slot * U * 4 * kThreads;
      slot = slot + 1 == kHeads ? 0 : slot + 1;
      asm volatile("cp.async.wait_group %0;" ::"n"(kHeads - 1) : "memory");
#pragma unroll
      for (int i = 0; i < U; ++i) {
        uint64_t e[N];
        const uint4* const v = place + i * 4 * kThreads;
        unpack2<T>(v[0], xs[i]);
        unpack2<T>(v[kThreads], xs[i] + P);
        unpack2<T>(v[2 * kThreads], e);
        unpack2<T>(v[3 * kThreads], e + P);
        if constexpr (INTER) {
#pragma unroll
          for (int j = 0; j < N; ++j) z[i][j] = f2_fma(swap2(e[j]), s2[i][j], f2_mul(e[j], c2[i][j]));
        } else {
#pragma unroll
          for (int j = 0; j < P; ++j) {
            z[i][j] = f2_sub(f2_mul(e[j], c2[i][j]), f2_mul(e[P + j], s2[i][j]));
            z[i][P + j] = f2_fma(e[j], s2[i][j], f2_mul(e[P + j], c2[i][j]));
          }
        }
      }
#pragma unroll
      for (int i = 0; i < U; ++i)
#pragma unroll
        for (int j = 0; j < N; ++j) {
          ss = f2_fma(xs[i][j], xs[i][j], ss);
          su = f2_fma(xs[i][j], f2_mul(z[i][j], w[i][j]), su);
        }
      const float r = rsqrtf(fmaf(team_sum<LANES>(sum2(ss), mask), inv_d, a.eps));
      const float mean = team_sum<LANES>(sum2(su), mask) * r * inv_d;          // mean(u n)
      ahead.copy(place);                           // (the sums have used its last contents)
      const uint64_t r2 = f2_pack(r, r), nm2 = f2_pack(-r * mean * r, -r * mean * r);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        uint64_t o[N];
#pragma unroll
        for (int j = 0; j < N; ++j) {
          const uint64_t zr = f2_mul(z[i][j], r2);
          dw[i][j] = f2_fma(xs[i][j], zr, dw[i][j]);
          o[j] = f2_fma(zr, w[i][j], f2_mul(xs[i][j], nm2));
        }
        if (un.first[i]) st_once(dx + un.c0[i], pack2<T>(o));
        if (un.second[i]) st_once(dx + un.c1[i], pack2<T>(o + P));
      }
      dx += a.d;
    }
  }
  if (q.dweight == nullptr) return;
  asm volatile("cp.async.wait_all;" ::: "memory");
  __syncthreads();
  float* const s_dw = reinterpret_cast<float*>(s_ring);
#pragma unroll
  for (int i = 0; i < U; ++i) {
    float* const o = s_dw + team * a.d;
#pragma unroll
    for (int j = 0; j < P; ++j) {
      if (un.first[i]) f2_unpack(dw[i][j], o[un.c0[i] + 2 * j], o[un.c0[i] + 2 * j + 1]);
      if (un.second[i]) f2_unpack(dw[i][P + j], o[un.c1[i] + 2 * j], o[un.c1[i] + 2 * j + 1]);
    }
  }
  __syncthreads();
  for (int c = threadIdx.x; c < a.d; c += kThreads) {
    float x = 0.f;
    for (int m = 0; m < kTeams; ++m) x += s_dw[m * a.d + c];
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

// Whether rows are whole 16-byte pieces, and the lanes of a team and units of a lane then.
template <typename T>
bool vector_shape(const QkArgs& a, int& lanes, int& units) {
  constexpr int N = Vec<T>::N;
  if (a.d % N != 0 || (a.interleaved ? a.rot : a.rot / 2) % N != 0) return false;
  for (int i = 0; i < a.n; ++i) {
    const QkTensor& q = a.t[i];
    const void* const ptrs[] = {q.x, q.weight, q.y, q.dy, q.dx};
    for (const void* p : ptrs)
      if ((reinterpret_cast<uintptr_t>(p) & 15) != 0) return false;
    if (q.x_stride % N != 0 || q.y_stride % N != 0 || q.dx_stride % N != 0) return false;
  }
  const int vecs = a.d / N, turned = a.rot / N;
  const int n = a.interleaved ? (vecs + 1) / 2 : turned / 2 + (vecs - turned + 1) / 2;
  lanes = 4;
  while (lanes < 32 && lanes < n) lanes *= 2;
  units = (n + lanes - 1) / lanes;
  return units <= 2;
}

// Heads of a part when there are to be `hsplit` parts or more: a part lies in one group.
int part_heads(const QkTensor& q, int64_t hsplit) {
  const int hpg = q.heads / q.groups;
  int per = (int)ceil_div(q.heads, hsplit);
  if (q.groups == 1) return per;
  per = std::min(per, hpg);
  while (hpg % per != 0) --per;
  return per;
}

// The kernel of a shape, as a type: KERN is a template of <T, INTER, LANES, U>.
template <auto K> struct Kernel { static constexpr auto value = K; };
#define NSP_QK_KERNEL(KERN, T, lanes, units, inter, go)                                        \
  do {                                                                                         \
    if (units == 2) {                                                                          \
      if (inter) go(Kernel<KERN<T, true, 32, 2>>{}); else go(Kernel<KERN<T, false, 32, 2>>{}); \
    } else if (lanes == 4) {                                                                   \
      if (inter) go(Kernel<KERN<T, true, 4, 1>>{}); else go(Kernel<KERN<T, false, 4, 1>>{});   \
    } else if (lanes == 8) {                                                                   \
      if (inter) go(Kernel<KERN<T, true, 8, 1>>{}); else go(Kernel<KERN<T, false, 8, 1>>{});   \
    } else if (lanes == 16) {                                                                  \
      if (inter) go(Kernel<KERN<T, true, 16, 1>>{}); else go(Kernel<KERN<T, false, 16, 1>>{}); \
    } else {                                                                                   \
      if (inter) go(Kernel<KERN<T, true, 32, 1>>{}); else go(Kernel<KERN<T, false, 32, 1>>{}); \
    }                                                                                          \
  } while (0)

template <typename T>
cudaError_t fwd(const QkArgs& a, cudaStream_t s) {
  Share share = {};
  int lanes, units;
  const bool vec = vector_shape<T>(a, lanes, units);
  const int64_t nsm = num_sms();
  int total = 0;
  for (int i = 0; i < a.n; ++i) total += a.t[i].heads;
  for (int i = 0; i < a.n; ++i) {
    const int heads = a.t[i].heads;
    int64_t blocks;
    if (vec) {
      // A token's heads are split over several teams, each with its own search and angles,
      // until every SM has two blocks, and in parts of 12 heads or more of a stream that does
      // not fit in L2, whose rows in flight then lie closer together (as in rope.cu)
      const int teams = kVecThreads / lanes;
      const int64_t bytes = 2 * a.len * total * a.d * (int64_t)sizeof(T);
      int64_t hsplit = ceil_div(nsm * 2 * teams * heads, a.len * total);
      if (bytes > kL2Bytes) hsplit = std::max<int64_t>(hsplit, heads / 12);
      hsplit = std::max<int64_t>(1, std::min<int64_t>(hsplit, heads));
      if (a.len * hsplit > UINT32_MAX) hsplit = 1;     // the kernel divides split items in 32 bits
      share.per[i] = part_heads(a.t[i], hsplit);
      share.hsplit[i] = (int)ceil_div(heads, share.per[i]);
      blocks = std::min<int64_t>(ceil_div(a.len * share.hsplit[i], teams), nsm * 128);
    } else {
      blocks = std::min<int64_t>(ceil_div(a.len * heads, kWarps), nsm * 8);
    }
    share.first[i + 1] = share.first[i] + (int)blocks;
  }
  auto go = [&](auto tag) { decltype(tag)::value<<<share.first[a.n], kVecThreads, 0, s>>>(a, share); };
  if (!vec) qk_element_kernel<T, false><<<share.first[a.n], kThreads, 0, s>>>(a, share);
  else NSP_QK_KERNEL(qk_vec_kernel, T, lanes, units, a.interleaved, go);
  count_launches(1);
  return cudaGetLastError();
}

template <typename T>
cudaError_t bwd(const QkArgs& a, cudaStream_t s) {
  Share share = {};
  int lanes, units;
  const bool vec = vector_shape<T>(a, lanes, units);
  bool weights = false;
  for (int i = 0; i < a.n; ++i) {
    share.first[i + 1] = share.first[i] + qk_bwd_blocks(a.t, a.n, i, a.len);
    weights = weights || a.t[i].dweight != nullptr;
  }
  const int smem = units == 2 ? bwd_ring_bytes<2>() : bwd_ring_bytes<1>();
  cudaError_t e = cudaSuccess;
  auto go = [&](auto tag) {
    constexpr auto kern = decltype(tag)::value;
    static bool allowed[64] = {};
    int dev = 0;
    e = cudaGetDevice(&dev);
    if (e == cudaSuccess && (dev >= 64 || !allowed[dev])) {
      e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
      if (e == cudaSuccess && dev < 64) allowed[dev] = true;
    }
    if (e == cudaSuccess) kern<<<share.first[a.n], kThreads, smem, s>>>(a, share);
  };
  if (!vec) qk_element_kernel<T, true><<<share.first[a.n], kThreads, sizeof(float) * kWarps * a.d, s>>>(a, share);
  else NSP_QK_KERNEL(qk_vec_bwd_kernel, T, lanes, units, a.interleaved, go);
  count_launches(1);
  if (e == cudaSuccess) e = cudaGetLastError();
  if (e != cudaSuccess || !weights) return e;
  e = launch_dependent(qk_weight_grad_kernel<T>, dim3((a.d + 31) / 32, a.n), dim3(kSumThreads), 0, s,
                       a, share);
  count_launches(1);
  return e;
}

}  // namespace

// kBwdBlocks blocks, two on each of 152 SMs, shared by the tensors' heads and some for
// every tensor's searches and angles; fewer for few rows.  The same on every device: the
// workspace's size, and the order of the weights' sums, go by it.
template <typename Tensor>
static int bwd_blocks(const Tensor* t, int n, int i, int64_t len) {
  int64_t total = 0;
  for (int k = 0; k < n; ++k) total += t[k].heads + 4;
  const int64_t share = std::max<int64_t>(1, (int64_t)kBwdBlocks * (t[i].heads + 4) / total);
  return (int)std::max<int64_t>(1, std::min<int64_t>(share, ceil_div(len * t[i].heads, kWarps)));
}
int qk_bwd_blocks(const QkTensor* t, int n, int i, int64_t len) { return bwd_blocks(t, n, i, len); }
int qk_bwd_blocks(const nsp_qk_tensor_t* t, int n, int i, int64_t len) { return bwd_blocks(t, n, i, len); }

cudaError_t launch_qk_norm_rope(const QkArgs& a, int32_t io_dtype, cudaStream_t s) {
  return io_dtype == NSP_BF16 ? fwd<__nv_bfloat16>(a, s) : fwd<float>(a, s);
}

cudaError_t launch_qk_norm_rope_bwd(const QkArgs& a, int32_t io_dtype, cudaStream_t s) {
  return io_dtype == NSP_BF16 ? bwd<__nv_bfloat16>(a, s) : bwd<float>(a, s);
}

}  // namespace nsp
