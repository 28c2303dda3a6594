// Log-probability of a given token of every row of logits, and its gradient:
//   x_j = s logit_j,  lse = ln sum_j exp(x_j),  logp = x_y - lse,
//   d logit_j = s g ([j = y] - exp(x_j - lse)),
// g the gradient of logp: given (backward), or the policy loss's own, of the logp
// just computed (the row is then read once for both).  A row without a target
// (y < 0) is not read; its logp, lse and gradient are zero.
//
// All in base 2: with c = s log2(e), a range's state is M = c max x (rounded once)
// and S = sum 2^(c x - M), each term's argument one FMA of the unrounded c x; ranges
// join by S1 2^(M1 - M) + S2 2^(M2 - M).  The same M serves the sum, logp and the
// gradient, so that its rounding cancels.
//
// A row is split over the blocks of a cluster, and a block's slice lives in its
// threads' registers: one read of the logits, the sum, one exchange of (M, S)
// through the cluster's shared memory, and the gradient from the same registers.
#include <algorithm>
#include <cmath>

#include "policy.cuh"
#include "tc_ptx.cuh"

namespace nsp {
namespace {

using namespace tc;

constexpr int kMaxRanks = 8;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// The sum of both ranges, in the first.
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
  const float top = fmaxf(m, m2);
  const float ref = top == -INFINITY ? 0.f : top;
  s = s * ex2(m - ref) + s2 * ex2(m2 - ref);
  m = top;
}

template <typename T> struct Raw;
template <> struct Raw<float> {
  static constexpr uint32_t kNegInf = 0xff800000u;
  __device__ static __forceinline__ float top(const uint4& u) {
    return fmaxf(max3f(__uint_as_float(u.x), __uint_as_float(u.y), __uint_as_float(u.z)),
                 __uint_as_float(u.w));
  }
};
template <> struct Raw<__nv_bfloat16> {
  static constexpr uint32_t kNegInf = 0xff80ff80u;
  __device__ static __forceinline__ float top(const uint4& u) {
    uint32_t a, b;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(u.x), "r"(u.y));
    asm("max.bf16x2 %0, %1, %2;" : "=r"(b) : "r"(u.z), "r"(u.w));
    asm("max.bf16x2 %0, %1, %2;" : "=r"(a) : "r"(a), "r"(b));
    return fmaxf(__uint_as_float(a << 16), __uint_as_float(a & 0xffff0000u));
  }
};

// sum of 2^(c x + n) over a vector, added to acc pair by pair
template <typename T>
__device__ __forceinline__ uint64_t add_exps(const uint4& u, uint64_t c2, uint64_t n2, uint64_t acc) {
  float x[Vec<T>::N];
  Vec<T>::unpack(u, x);
#pragma unroll
  for (int i = 0; i < Vec<T>::N / 2; ++i) {
    float a, b;
    f2_unpack(f2_fma(f2_pack(x[2 * i], x[2 * i + 1]), c2, n2), a, b);
    acc = f2_add(acc, f2_pack(ex2(a), ex2(b)));
  }
  return acc;
}

__device__ __forceinline__ void cluster_arrive() { asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory"); }
__device__ __forceinline__ void cluster_wait() { asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory"); }
__device__ __forceinline__ void st_peer(const float2* p, int rank, float2 v) {
  uint32_t at;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(at) : "r"(smem_u32(p)), "r"(rank));
  asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(at), "f"(v.x), "f"(v.y) : "memory");
}

// VPT: vectors of a thread held in registers; what a slice has more is read again.
template <typename T, RowMode MODE, int THREADS, int VPT>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) row_kernel(const __grid_constant__ RowArgs a,
                                                                      const int ranks) {
  constexpr int N = Vec<T>::N, kWarps = THREADS / 32;
  __shared__ float2 s_part[kMaxRanks * kWarps];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t t = blockIdx.x / (unsigned)ranks;
  const int rank = (int)(blockIdx.x - (unsigned)t * ranks);
  if (MODE == kRowPolicy && status_bad(a.p.hdr)) return;
  const int y = __ldg(a.targets + t);
  const T* const x = reinterpret_cast<const T*>(a.logits) + t * a.row_stride;
  T* const dx = reinterpret_cast<T*>(a.dlogits) + t * a.out_stride;
  bool scored = y >= 0;
  if (MODE == kRowPolicy) scored = scored && t < (int64_t)__ldg(a.p.cu + a.p.ndoc);
  // The row's whole vectors start at its first 16-byte border; the elements before and
  // behind them are rank 0's first threads'.
  const int head = min((int)((16 - (reinterpret_cast<uintptr_t>(x) & 15)) & 15) / (int)sizeof(T), a.vocab);
  const int nvec = (a.vocab - head) / N, rest = a.vocab - nvec * N;
  const int per = (nvec + ranks - 1) / ranks, v0 = rank * per, v1 = min(v0 + per, nvec);
  const bool extra = rank == 0 && tid < rest;
  const int ecol = tid < head ? tid : nvec * N + tid;
  const uint4* const xv = reinterpret_cast<const uint4*>(x + head);
  const bool whole = ((reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(dx)) & 15) == 0;
  auto store = [&](int v, const float (&o)[N]) {
    if (whole) {
      st_once(dx + head + (int64_t)v * N, Vec<T>::pack(o));
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) st_out(dx + head + (int64_t)v * N + i, o[i]);
    }
  };
  if (!scored) {
    if (MODE != kRowForward) {
      const float zero[N] = {};
      for (int v = v0 + tid; v < v1; v += THREADS) store(v, zero);
      if (extra) st_out(dx + ecol, 0.f);
    }
    if (MODE != kRowBackward && rank == 0 && tid == 0) {
      if (a.logp) a.logp[t] = 0.f;
      if (a.lse) a.lse[t] = 0.f;
      if (MODE == kRowPolicy)
        for (int i = 0; i < 3; ++i) a.p.terms[i * a.rows + t] = 0.f;
    }
    return;
  }
  if (MODE != kRowBackward && ranks > 1) cluster_arrive();
  uint4 reg[VPT];
#pragma unroll
  for (int i = 0; i < VPT; ++i) {
    const int v = v0 + i * THREADS + tid;
    reg[i] = v < v1 ? ld_once(xv + v)
                    : make_uint4(Raw<T>::kNegInf, Raw<T>::kNegInf, Raw<T>::kNegInf, Raw<T>::kNegInf);
  }
  const float xe = extra ? to_f(x[ecol]) : -INFINITY;
  const float c = a.scale * kLog2e;
  const uint64_t c2 = f2_pack(c, c);
  float n, k, g;                     // p = 2^(c x + n) k;  d logit = s g ([j = y] - p)
  if constexpr (MODE == kRowBackward) {
    n = -__ldg(a.in_lse + t) * kLog2e;
    k = 1.f;
    g = __ldg(a.dlogp + t);
  } else {
    // (read before the barrier: a gradient in place is written behind it)
    const float xy = y < a.vocab ? to_f(x[y]) : NAN;
    const int doc = MODE == kRowPolicy ? doc_of(a.p.cu, a.p.ndoc, t) : 0;
    float top = xe;
#pragma unroll
    for (int i = 0; i < VPT; ++i) top = fmaxf(top, Raw<T>::top(reg[i]));
    float m = top * c;
    auto ref = [](float m) { return m == -INFINITY ? 0.f : -m; };
    const uint64_t n2 = f2_pack(ref(m), ref(m));
    uint64_t acc[2] = {f2_pack(ex2(fmaf(xe, c, ref(m))), 0.f), 0};
#pragma unroll
    for (int i = 0; i < VPT; ++i) acc[i & 1] = add_exps<T>(reg[i], c2, n2, acc[i & 1]);
    float s, s1;
    f2_unpack(f2_add(acc[0], acc[1]), s, s1);
    s += s1;
    for (int v = v0 + VPT * THREADS + tid; v < v1; v += THREADS) {
      const uint4 u = ld_once(xv + v);
      const float m1 = Raw<T>::top(u) * c;
      const uint64_t one = add_exps<T>(u, c2, f2_pack(ref(m1), ref(m1)), 0);
      float p0, p1;
      f2_unpack(one, p0, p1);
      join(m, s, m1, p0 + p1);
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      join(m, s, __shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, s, o));
    // every warp's state to every block of the cluster
    if (ranks > 1) {
      cluster_wait();
      if (lane < ranks) st_peer(&s_part[rank * kWarps + warp], lane, make_float2(m, s));
      __syncwarp();
      cluster_arrive();
      cluster_wait();
    } else {
      if (lane == 0) s_part[warp] = make_float2(m, s);
      __syncthreads();
    }
    m = -INFINITY;
    s = 0.f;
    for (int i = lane; i < ranks * kWarps; i += 32) join(m, s, s_part[i].x, s_part[i].y);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
      join(m, s, __shfl_xor_sync(0xffffffffu, m, o), __shfl_xor_sync(0xffffffffu, s, o));
    const float rest2 = log2f(s);
    float logp = (fmaf(xy, c, -m) - rest2) * kLn2;
    if (logp > 0.f) logp = 0.f;      // (by its rounding)
    const bool writes = rank == 0 && tid == 0;
    if (writes) {
      if (a.logp) a.logp[t] = logp;
      if (a.lse) a.lse[t] = (m + rest2) * kLn2;
    }
    if constexpr (MODE == kRowPolicy) {
      const PolicyRow r = policy_row(a.p, policy_scalars(a.p, t, doc), logp);
      g = r.grad;
      if (writes) {
        a.p.terms[t] = r.surrogate;
        a.p.terms[a.rows + t] = r.kl;
        a.p.terms[2 * a.rows + t] = r.clipped;
      }
      n = ref(m);
      k = 1.f / s;
    }
  }
  if constexpr (MODE != kRowForward) {
    if (y >= a.vocab) g = NAN;
    const float sg = a.scale * g, f = -sg * k;
    const uint64_t n2 = f2_pack(n, n), f2 = f2_pack(f, f);
    const int yv = y < head ? -1 : (y - head) / N, yi = y - head - yv * N;
    auto gradient = [&](int v, const uint4& u) {
      float o[N];
      Vec<T>::unpack(u, o);
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        float p, q;
        f2_unpack(f2_fma(f2_pack(o[2 * i], o[2 * i + 1]), c2, n2), p, q);
        f2_unpack(f2_mul(f2_pack(ex2(p), ex2(q)), f2), o[2 * i], o[2 * i + 1]);
      }
      if (v == yv) {
#pragma unroll
        for (int i = 0; i < N; ++i) o[i] += i == yi ? sg : 0.f;
      }
      store(v, o);
    };
#pragma unroll
    for (int i = 0; i < VPT; ++i) {
      const int v = v0 + i * THREADS + tid;
      if (v < v1) gradient(v, reg[i]);
    }
    for (int v = v0 + VPT * THREADS + tid; v < v1; v += THREADS) gradient(v, ld_once(xv + v));
    if (extra) st_out(dx + ecol, ex2(fmaf(xe, c, n)) * f + (ecol == y ? sg : 0.f));
  }
}

// ---- many long rows: persistent blocks behind a ring of asynchronous copies
//
// A block (a cluster of them, where a row is longer than 128 KB) walks its rows.  Every
// thread copies its own vectors of the rows ahead into shared memory, kRing chunks of
// kChunk vectors at any time, and reads only what it copied itself, so that the ring
// needs no barrier.  A scored row is read from there into registers, which the gradient
// is taken from.
constexpr int kRingThreads = 512, kRingWarps = kRingThreads / 32;
constexpr int kChunk = 4, kRing = 6;
constexpr int kRingBytes = kRing * kChunk * kRingThreads * 16;

__device__ __forceinline__ void copy16(uint32_t dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// The sum of a warp's 32 ranges, in every lane.
__device__ __forceinline__ void join_warp(float& m, float& s) {
  float top;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(top) : "f"(m));
  s *= ex2(m - (top == -INFINITY ? 0.f : top));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  m = top;
}

// NCH: chunks of a row (policy), held in registers; 0: any number, not held (forward).
template <typename T, RowMode MODE, int NCH>
__global__ void __launch_bounds__(kRingThreads, 1) ring_kernel(const __grid_constant__ RowArgs a,
                                                               const int ranks, const int chunks) {
  constexpr int N = Vec<T>::N;
  extern __shared__ __align__(16) uint4 s_ring[];
  __shared__ float2 s_part[2][kMaxRanks * kRingWarps];
  __shared__ float2 s_target[2];                     // x: the target's logit
  __shared__ int2 s_queue[kRingWarps][8];            // rows copied ahead, a warp's own copy
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int rank = ranks > 1 ? (int)(blockIdx.x % (unsigned)ranks) : 0;
  const int64_t first = blockIdx.x / (unsigned)ranks, step = gridDim.x / (unsigned)ranks;
  if (MODE == kRowPolicy) {
    grid_dep_wait();
    if (status_bad(a.p.hdr)) return;
  }
  const int64_t end = MODE == kRowPolicy ? min(a.rows, (int64_t)__ldg(a.p.cu + a.p.ndoc)) : a.rows;
  uint4* const ring = s_ring + tid;
  const float c = a.scale * kLog2e;
  const uint64_t c2 = f2_pack(c, c);

  // A row's whole vectors start at its first 16-byte border, the thread's own ones at
  // `first_vec` of them, kRingThreads apart, while `left` > 0 of the block's slice; the
  // elements before and behind the vectors are rank 0's first threads'.
  struct Row {
    const T* x;
    int head, nvec, first_vec, left;
  };
  auto row_of = [&](int64_t t) {
    Row r;
    r.x = reinterpret_cast<const T*>(a.logits) + t * a.row_stride;
    r.head = min((int)((16 - (reinterpret_cast<uintptr_t>(r.x) & 15)) & 15) / (int)sizeof(T), a.vocab);
    r.nvec = (a.vocab - r.head) / N;
    const int per = (r.nvec + ranks - 1) / ranks;
    r.first_vec = rank * per + tid;
    r.left = min(rank * per + per, r.nvec) - r.first_vec;
    return r;
  };
  auto store = [&](T* dx, bool whole, const float (&o)[N]) {
    if (whole) {
      st_once(dx, Vec<T>::pack(o));
    } else {
#pragma unroll
      for (int i = 0; i < N; ++i) st_out(dx + i, o[i]);
    }
  };
  auto gradient_row = [&](int64_t t, const T* x, bool& whole) {
    T* const dx = reinterpret_cast<T*>(a.dlogits) + t * a.out_stride;
    whole = ((reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(dx)) & 15) == 0;
    return dx;
  };
  // a row without a score: zeros
  auto skip = [&](int64_t t) {
    if constexpr (MODE == kRowPolicy) {
      const Row r = row_of(t);
      bool whole;
      T* const dx = gradient_row(t, r.x, whole);
      const float zero[N] = {};
      for (int i = 0; i < r.left; i += kRingThreads)
        store(dx + r.head + (int64_t)(r.first_vec + i) * N, whole, zero);
      if (rank == 0 && tid < a.vocab - r.nvec * N) st_out(dx + (tid < r.head ? tid : r.nvec * N + tid), 0.f);
    }
    if (rank == 0 && tid == 0) {
      if (a.logp) a.logp[t] = 0.f;
      if (a.lse) a.lse[t] = 0.f;
      if (MODE == kRowPolicy)
        for (int i = 0; i < 3; ++i) a.p.terms[i * a.rows + t] = 0.f;
    }
  };

  // The block's rows in order, 32 targets at a time in a warp's lanes, the next 32 on
  // their way.
  auto target = [&](int64_t i) {
    const int64_t t = first + i * step;
    return t < end ? __ldg(a.targets + t) : -1;
  };
  int64_t base = 0;
  int y32 = target(lane), y_next = target(32 + lane);
  uint32_t left = __ballot_sync(0xffffffffu, y32 >= 0);
  int at = 0;                                        // rows of the 32 that are done with
  auto next = [&](int64_t& t, int& y) {
    for (;;) {
      const int bit = left ? __ffs(left) - 1 : 32;
      for (; at < bit; ++at) {
        const int64_t u = first + (base + at) * step;
        if (u >= a.rows) return false;
        skip(u);
      }
      if (bit < 32) {
        left &= left - 1;
        at = bit + 1;
        t = first + (base + bit) * step;
        y = __shfl_sync(0xffffffffu, y32, bit);
        return true;
      }
      base += 32;
      y32 = y_next;
      y_next = target(base + 32 + lane);
      left = __ballot_sync(0xffffffffu, y32 >= 0);
      at = 0;
    }
  };
  int queued = 0, taken = 0, ahead_left = 0;
  const uint4* ahead = nullptr;                      // the thread's first vector of the row ahead
  bool more = true;
  auto next_row = [&] {
    int64_t t;
    int y;
    more = more && next(t, y);
    ahead_left = 0;
    if (!more) return;
    const Row r = row_of(t);
    ahead = reinterpret_cast<const uint4*>(r.x + r.head) + r.first_vec;
    ahead_left = r.left;
    if (lane == 0) s_queue[warp][queued & 7] = make_int2((int)t, y);
    ++queued;
  };
  // chunk ch of the row ahead; where the row has no vector the ring holds -infinity
  auto copy_chunk = [&](int slot, int ch) {
    if (more) {
#pragma unroll
      for (int i = 0; i < kChunk; ++i) {
        uint4* const to = ring + (slot * kChunk + i) * kRingThreads;
        const int v = (ch * kChunk + i) * kRingThreads;
        if (v < ahead_left) copy16(smem_u32(to), ahead + v);
        else *to = make_uint4(Raw<T>::kNegInf, Raw<T>::kNegInf, Raw<T>::kNegInf, Raw<T>::kNegInf);
      }
    }
    copy_commit();
  };
  int ch_ahead = 0;
  for (int i = 0; i < kRing; ++i) {
    if (ch_ahead == 0) next_row();
    copy_chunk(i, ch_ahead);
    ch_ahead = ch_ahead + 1 == chunks ? 0 : ch_ahead + 1;
  }
  if (ranks > 1) {                                   // (every block of the cluster runs)
    cluster_arrive();
    cluster_wait();
  }
  int slot = 0;
  for (; taken < queued; ++taken) {
    __syncwarp();
    const int2 item = s_queue[warp][taken & 7];
    __syncwarp();
    const int64_t t = item.x;
    const int y = item.y, par = taken & 1;
    const Row r = row_of(t);
    const int rest = a.vocab - r.nvec * N;
    const bool extra = rank == 0 && tid < rest;
    const int ecol = tid < r.head ? tid : r.nvec * N + tid;
    const float xe = extra ? to_f(r.x[ecol]) : -INFINITY;
    // the thread's vector with the target (its number in the thread's), and where in it
    const int ydist = (y < r.head ? -1 : (y - r.head) / N) - r.first_vec;
    const int mine = ydist >= 0 && ydist < r.left && ydist % kRingThreads == 0 ? ydist / kRingThreads : -1;
    const int yi = (y - r.head) & (N - 1);
    auto publish = [&](float x) {
      if (ranks > 1) {
        for (int k = 0; k < ranks; ++k) st_peer(&s_target[par], k, make_float2(x, 0.f));
      } else {
        s_target[par].x = x;
      }
    };
    uint4 reg[NCH > 0 ? NCH * kChunk : kChunk];
    float m = -INFINITY, s = 0.f;
    auto take = [&](int ch, uint4* u) {
      copy_wait<kRing - 1>();
      float top = -INFINITY;
#pragma unroll
      for (int i = 0; i < kChunk; ++i) {
        u[i] = ring[(slot * kChunk + i) * kRingThreads];
        top = fmaxf(top, Raw<T>::top(u[i]));
        if (mine == ch * kChunk + i) {
          float e[N], xy = 0.f;
          Vec<T>::unpack(u[i], e);
#pragma unroll
          for (int j = 0; j < N; ++j) xy = j == yi ? e[j] : xy;
          publish(xy);
        }
      }
      const float m1 = fmaxf(m, top * c), n1 = m1 == -INFINITY ? 0.f : -m1;
      const uint64_t n2 = f2_pack(n1, n1);
      uint64_t acc[2] = {f2_pack(s * ex2(m + n1), 0.f), 0};
      m = m1;
#pragma unroll
      for (int i = 0; i < kChunk; ++i) acc[i & 1] = add_exps<T>(u[i], c2, n2, acc[i & 1]);
      float s1;
      f2_unpack(f2_add(acc[0], acc[1]), s, s1);
      s += s1;
    };
    auto advance = [&] { slot = slot + 1 == kRing ? 0 : slot + 1; };
    if constexpr (NCH > 0) {
#pragma unroll
      for (int ch = 0; ch < NCH; ++ch) {
        take(ch, reg + ch * kChunk);
        if ((ch + kRing) % NCH == 0) next_row();
        copy_chunk(slot, (ch + kRing) % NCH);
        advance();
      }
    } else {
      for (int ch = 0; ch < chunks; ++ch) {
        take(ch, reg);
        if (ch_ahead == 0) next_row();
        copy_chunk(slot, ch_ahead);
        ch_ahead = ch_ahead + 1 == chunks ? 0 : ch_ahead + 1;
        advance();
      }
    }
    PolicyScalars sc = {};
    if constexpr (MODE == kRowPolicy) {
      const float2 w = __ldg(a.p.row_scalars + t);
      sc = {w.x, w.y, __ldg(a.p.old_logp + t), a.p.ref_logp != nullptr ? __ldg(a.p.ref_logp + t) : 0.f};
    }
    if (extra) {
      join(m, s, xe * c, isinf(xe) && xe < 0.f ? 0.f : 1.f);
      if (ecol == y) publish(xe);
    }
    if (tid == 0 && rank == 0 && y >= a.vocab) publish(NAN);
    join_warp(m, s);
    // (two sets of states in turn: a block that writes the next row's has seen every block
    // behind this row's barrier, and so behind reading the last row's)
    if (ranks > 1) {
      if (lane < ranks) st_peer(&s_part[par][rank * kRingWarps + warp], lane, make_float2(m, s));
      __syncwarp();
      cluster_arrive();
      cluster_wait();
    } else {
      if (lane == 0) s_part[par][warp] = make_float2(m, s);
      __syncthreads();
    }
    if (MODE == kRowForward && warp != 0) continue;
    m = -INFINITY;
    s = 0.f;
    if (lane < ranks * kRingWarps) {
      m = s_part[par][lane].x;
      s = s_part[par][lane].y;
    }
    for (int i = lane + 32; i < ranks * kRingWarps; i += 32) join(m, s, s_part[par][i].x, s_part[par][i].y);
    join_warp(m, s);
    const float rest2 = log2f(s);
    float logp = (fmaf(s_target[par].x, c, -m) - rest2) * kLn2;
    if (logp > 0.f) logp = 0.f;      // (by its rounding)
    const bool writes = rank == 0 && tid == 0;
    if (writes) {
      if (a.logp) a.logp[t] = logp;
      if (a.lse) a.lse[t] = (m + rest2) * kLn2;
    }
    if constexpr (MODE == kRowPolicy) {
      const PolicyRow pr = policy_row(a.p, sc, logp);
      if (writes) {
        a.p.terms[t] = pr.surrogate;
        a.p.terms[a.rows + t] = pr.kl;
        a.p.terms[2 * a.rows + t] = pr.clipped;
      }
      const float g = y < a.vocab ? pr.grad : NAN;
      const float sg = a.scale * g, f = -sg / s, n = m == -INFINITY ? 0.f : -m;
      const uint64_t n2 = f2_pack(n, n), ff = f2_pack(f, f);
      bool whole;
      T* const dx = gradient_row(t, r.x, whole);
      T* const out = dx + r.head + (int64_t)r.first_vec * N;
#pragma unroll
      for (int i = 0; i < NCH * kChunk; ++i) {
        if (i * kRingThreads >= r.left) break;
        float o[N];
        Vec<T>::unpack(reg[i], o);
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
          float p, q;
          f2_unpack(f2_fma(f2_pack(o[2 * j], o[2 * j + 1]), c2, n2), p, q);
          f2_unpack(f2_mul(f2_pack(ex2(p), ex2(q)), ff), o[2 * j], o[2 * j + 1]);
        }
        if (i == mine) {
#pragma unroll
          for (int j = 0; j < N; ++j) o[j] += j == yi ? sg : 0.f;
        }
        store(out + i * kRingThreads * N, whole, o);
      }
      if (extra) st_out(dx + ecol, ex2(fmaf(xe, c, n)) * f + (ecol == y ? sg : 0.f));
    }
  }
}

template <typename T, RowMode MODE, int NCH>
cudaError_t go_ring(const RowArgs& a, int ranks, int chunks, cudaStream_t s) {
  static bool allowed[64] = {};
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  auto kern = ring_kernel<T, MODE, NCH>;
  if (dev >= 64 || !allowed[dev]) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
    if (e != cudaSuccess) return e;
    if (dev < 64) allowed[dev] = true;
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(num_sms() / ranks * ranks));
  cfg.blockDim = dim3(kRingThreads);
  cfg.dynamicSmemBytes = kRingBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  int n = 0;
  if (ranks > 1) {
    attr[n].id = cudaLaunchAttributeClusterDimension;
    attr[n].val.clusterDim.x = (unsigned)ranks;
    attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
    ++n;
    // the clusters that run at once: one that had to wait for others would double the time
    static int resident[64][kMaxRanks + 1] = {};
    int fit = dev < 64 ? resident[dev][ranks] : 0;
    if (fit == 0) {
      cfg.attrs = attr;
      cfg.numAttrs = n;
      e = cudaOccupancyMaxActiveClusters(&fit, kern, &cfg);
      if (e != cudaSuccess) return e;
      if (fit < 1) return cudaErrorInvalidConfiguration;
      if (dev < 64) resident[dev][ranks] = fit;
    }
    cfg.gridDim.x = (unsigned)(std::min<int64_t>(fit, num_sms() / ranks) * ranks);
  }
  if (a.rows * ranks < cfg.gridDim.x) cfg.gridDim.x = (unsigned)(a.rows * ranks);
  if (MODE == kRowPolicy) {
    attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[n].val.programmaticStreamSerializationAllowed = 1;
    ++n;
  }
  cfg.attrs = attr;
  cfg.numAttrs = n;
  count_launches(1);
  return cudaLaunchKernelEx(&cfg, kern, a, ranks, chunks);
}

template <typename T, RowMode MODE, int THREADS, int VPT>
cudaError_t go(const RowArgs& a, int ranks, cudaStream_t s) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(a.rows * ranks));
  cfg.blockDim = dim3(THREADS);
  cfg.stream = s;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = MODE != kRowBackward && ranks > 1 ? 1 : 0;
  count_launches(1);
  return cudaLaunchKernelEx(&cfg, row_kernel<T, MODE, THREADS, VPT>, a, ranks);
}

template <typename T, RowMode MODE>
cudaError_t launch_mode(const RowArgs& a, cudaStream_t s) {
  const int64_t nvec = std::max(1, a.vocab / (16 / (int)sizeof(T)));
  if (nvec <= 128) return go<T, MODE, 128, 1>(a, 1, s);
  if (nvec <= 256) return go<T, MODE, 128, 2>(a, 1, s);
  if (nvec <= 512) return go<T, MODE, 128, 4>(a, 1, s);
  constexpr int kHeld = 4 * kChunk * kRingThreads;   // vectors of a block's registers
  if constexpr (MODE != kRowBackward) {
    int r = 1;
    if (MODE == kRowPolicy)
      while (r < kMaxRanks && nvec > (int64_t)r * kHeld) r *= 2;
    const int chunks = (int)ceil_div(ceil_div(nvec, r), kChunk * kRingThreads);
    if (a.rows * r >= (int64_t)num_sms() * 4 && (MODE == kRowForward || chunks <= 4)) {
      if constexpr (MODE == kRowForward) {
        return go_ring<T, MODE, 0>(a, 1, chunks, s);
      } else {
        const cudaError_t e = launch_loss_rows(a, s);
        if (e != cudaSuccess) return e;
        if (chunks == 1) return go_ring<T, MODE, 1>(a, r, chunks, s);
        if (chunks == 2) return go_ring<T, MODE, 2>(a, r, chunks, s);
        if (chunks == 3) return go_ring<T, MODE, 3>(a, r, chunks, s);
        return go_ring<T, MODE, 4>(a, r, chunks, s);
      }
    }
  }
  int ranks = 1;
  while (ranks < kMaxRanks && nvec > (int64_t)ranks * 4096) ranks *= 2;
  while (ranks < kMaxRanks && a.rows * ranks < (int64_t)num_sms() * 2 && nvec > (int64_t)ranks * 512) ranks *= 2;
  if (a.rows * ranks > INT32_MAX) ranks = 1;
  const int64_t per = ceil_div(nvec, ranks);
  if (per <= 512) return go<T, MODE, 512, 1>(a, ranks, s);
  if (per <= 1024) return go<T, MODE, 512, 2>(a, ranks, s);
  if (per <= 2048) return go<T, MODE, 512, 4>(a, ranks, s);
  return go<T, MODE, 512, 8>(a, ranks, s);
}

template <typename T>
cudaError_t launch_typed(const RowArgs& a, RowMode mode, cudaStream_t s) {
  if (mode == kRowForward) return launch_mode<T, kRowForward>(a, s);
  if (mode == kRowBackward) return launch_mode<T, kRowBackward>(a, s);
  return launch_mode<T, kRowPolicy>(a, s);
}

}  // namespace

cudaError_t launch_rows(const RowArgs& a, RowMode mode, int32_t io_dtype, cudaStream_t s) {
  return io_dtype == NSP_BF16 ? launch_typed<__nv_bfloat16>(a, mode, s) : launch_typed<float>(a, mode, s);
}

}  // namespace nsp
