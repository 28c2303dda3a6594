// Log-probability of a given token of every row of logits, and its gradient:
//   x_j = s logit_j,  lse = ln sum_j exp(x_j),  logp = x_y - lse,
//   d logit_j = s g ([j = y] - exp(x_j - lse)),
// g the gradient of logp: given (backward), or the policy loss's own, of the logp
// just computed (the row is then read once for both).  A row without a target
// (y < 0) is not read; its logp, lse and gradient are zero.
//
// All in base 2: with c = s log2(e) in two floats, a range's state is a whole number M
// just above c max x and S = sum 2^(c x - M), each term's argument two FMAs; ranges join
// by S1 2^(M1 - M) + S2 2^(M2 - M), whose powers are exact.  (c in one float and M = c max
// x: every logp of a document was off to the same side, by 2e-7 to 3e-7.)
//
// Bound: HBM; a scored row is read once, and where its gradient is wanted the gradient is
// taken from what is still on the chip.  Two ways there:
//   - few or short rows: a row over the registers of a block, or of the blocks of a cluster;
//     one exchange of (M, S) through the cluster's shared memory;
//   - many long rows: persistent blocks behind a ring of asynchronous copies (below).
// The backward alone has nothing to add up and streams: 149 us of 6000 rows of 49999 bf16
// logits (4180 scored), 6.8 TB/s.
#include <algorithm>
#include <cmath>

#include "policy.cuh"
#include "tc_ptx.cuh"

namespace nsp {
namespace {

using namespace tc;

constexpr int kMaxRanks = 8;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// 2^d of a whole d <= 0 (0 where it would be a denormal, and of -infinity).
__device__ __forceinline__ float pow2(float d) {
  return d >= -126.f ? __int_as_float(((int)d + 127) << 23) : 0.f;
}

// The sum of both ranges, in the first.
__device__ __forceinline__ void join(float& m, float& s, float m2, float s2) {
  const float top = fmaxf(m, m2);
  const float ref = top == -INFINITY ? 0.f : top;
  s = s * pow2(m - ref) + s2 * pow2(m2 - ref);
  m = top;
}

// logp and lse of a row whose sum is s 2^m.  Sums of a document's thousands of them are
// what they are wanted for, so that their errors must not lean to one side: ex2 is too
// small by 5.1e-8 of its value in the mean below zero (measured over [-30, 0]), and ln 2
// is taken in two floats.
constexpr float kBias = 5.1e-8f, kLn2Lo = (float)(0.69314718055994530942 - (double)kLn2);
__device__ __forceinline__ float finish(float xy, const RowArgs& a, float m, float s, float& lse) {
  const float l = log2f(s), d = fmaf(xy, a.c_lo, fmaf(xy, a.c, -m)) - l;
  const float logp = d == -INFINITY ? d : fmaf(d, kLn2, fmaf(d, kLn2Lo, -kBias));
  lse = fmaf(m + l, kLn2, fmaf(m + l, kLn2Lo, kBias));
  return logp > 0.f ? 0.f : logp;  // (by its rounding; NaN stays)
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

// c = s log2(e) in two floats, each twice.
struct Scale2 {
  uint64_t hi, lo;
  __device__ __forceinline__ explicit Scale2(const RowArgs& a)
      : hi(f2_pack(a.c, a.c)), lo(f2_pack(a.c_lo, a.c_lo)) {}
};

// sum of 2^(c x + n) over a vector, added to acc pair by pair
template <typename T>
__device__ __forceinline__ uint64_t add_exps(const uint4& u, const Scale2& c, uint64_t n2, uint64_t acc) {
  float x[Vec<T>::N];
  Vec<T>::unpack(u, x);
#pragma unroll
  for (int i = 0; i < Vec<T>::N / 2; ++i) {
    const uint64_t v = f2_pack(x[2 * i], x[2 * i + 1]);
    float a, b;
    f2_unpack(f2_fma(v, c.lo, f2_fma(v, c.hi, n2)), a, b);
    acc = f2_add(acc, f2_pack(ex2(a), ex2(b)));
  }
  return acc;
}

// c x + n for a gradient: bf16 ones need no more than c's first float.
template <typename T>
__device__ __forceinline__ uint64_t exponents(uint64_t v, const Scale2& c, uint64_t n2) {
  const uint64_t z = f2_fma(v, c.hi, n2);
  return sizeof(T) == 4 ? f2_fma(v, c.lo, z) : z;
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
  const float c = a.c;
  const Scale2 c2(a);
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
    float m = ceilf(top * c);
    auto ref = [](float m) { return m == -INFINITY ? 0.f : -m; };
    const uint64_t n2 = f2_pack(ref(m), ref(m));
    uint64_t acc[2] = {f2_pack(ex2(fmaf(xe, a.c_lo, fmaf(xe, c, ref(m)))), 0.f), 0};
#pragma unroll
    for (int i = 0; i < VPT; ++i) acc[i & 1] = add_exps<T>(reg[i], c2, n2, acc[i & 1]);
    float s, s1;
    f2_unpack(f2_add(acc[0], acc[1]), s, s1);
    s += s1;
    for (int v = v0 + VPT * THREADS + tid; v < v1; v += THREADS) {
      const uint4 u = ld_once(xv + v);
      const float m1 = ceilf(Raw<T>::top(u) * c);
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
    const bool writes = rank == 0 && tid == 0;
    float lse;
    const float logp = finish(xy, a, m, s, lse);
    if (writes) {
      if (a.logp) a.logp[t] = logp;
      if (a.lse) a.lse[t] = lse;
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
        f2_unpack(exponents<T>(f2_pack(o[2 * i], o[2 * i + 1]), c2, n2), p, q);
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
    if (extra) st_out(dx + ecol, ex2(fmaf(xe, a.c_lo, fmaf(xe, c, n))) * f + (ecol == y ? sg : 0.f));
  }
}

// ---- many long rows: persistent blocks behind a ring of asynchronous copies
//
// A block of every SM walks its rows (policy: a cluster of blocks a row, a slice of it
// each).  Every thread copies its own vectors of the rows ahead into its own places of
// shared memory, 192 KB of them at any time, and reads only what it copied itself, so
// that the ring needs no barrier and no wait but the copies' own.
// 8192 rows of 65536 bf16 logits (5730 scored): 127 us a call, 5.9 TB/s; a policy step on
// 8192 x 131072 of them, 30 % without a score: 656 us, 5.6 TB/s of logits read and
// gradients written (row by row from registers: 344 and 1491 us).  In the way of more:
// 10 instructions an element of the scores (80 % of the issue slots), twice that and two
// exponentials of the policy step (60 %), and a row's chain from
// its last vector over the cluster's exchange to the first gradient, under which a block
// only copies.  512 threads and clusters twice as large: 718 us of the step; a row held in
// registers in place of the ring: 867 us.
constexpr int kScoreThreads = 1024, kScoreSlots = 12;    // 16-byte places of a thread
constexpr int kPolicyThreads = 1024, kPolicySlots = 12, kMaxSlice = 8;   // vectors of a thread in a row
constexpr int kRingBytes = 12 * 1024 * 16;
static_assert(kScoreThreads * kScoreSlots * 16 == kRingBytes && kPolicyThreads * kPolicySlots * 16 == kRingBytes, "");

__device__ __forceinline__ void copy16(uint4* dst, const void* src) {
  asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(smem_u32(dst)), "l"(src) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait() { asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory"); }

// The sum of a warp's 32 ranges, in every lane.
__device__ __forceinline__ void join_warp(float& m, float& s) {
  float top;
  asm("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(top) : "f"(m));
  s *= pow2(m - (top == -INFINITY ? 0.f : top));
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) s += __shfl_xor_sync(0xffffffffu, s, o);
  m = top;
}

// A row's whole vectors start at its first 16-byte border, the thread's own ones at
// `vec` of them, the block's threads apart, while `left` > 0 of the block's slice; the elements
// before and behind the vectors are rank 0's first threads'.
template <typename T>
struct Row {
  const T* x;
  int head, nvec, vec, left;
};

template <typename T>
__device__ __forceinline__ Row<T> row_of(const RowArgs& a, int64_t t, int rank, int log_ranks) {
  constexpr int N = Vec<T>::N;
  Row<T> r;
  r.x = reinterpret_cast<const T*>(a.logits) + t * a.row_stride;
  r.head = min((int)((16 - (reinterpret_cast<uintptr_t>(r.x) & 15)) & 15) / (int)sizeof(T), a.vocab);
  r.nvec = (a.vocab - r.head) / N;
  const int per = (r.nvec + (1 << log_ranks) - 1) >> log_ranks;
  r.vec = rank * per + (int)threadIdx.x;
  r.left = min(rank * per + per, r.nvec) - r.vec;
  return r;
}

template <typename T>
__device__ __forceinline__ void store_vec(T* dx, bool whole, const float (&o)[Vec<T>::N]) {
  if (whole) {
    st_once(dx, Vec<T>::pack(o));
  } else {
#pragma unroll
    for (int i = 0; i < Vec<T>::N; ++i) st_out(dx + i, o[i]);
  }
}

// Where row t's gradient goes; whole: its vectors are vectors there as well.
template <typename T>
__device__ __forceinline__ T* gradient_row(const RowArgs& a, int64_t t, const T* x, bool& whole) {
  T* const dx = reinterpret_cast<T*>(a.dlogits) + t * a.out_stride;
  whole = ((reinterpret_cast<uintptr_t>(x) ^ reinterpret_cast<uintptr_t>(dx)) & 15) == 0;
  return dx;
}

// A block's share of the list of scored rows: entries first, first + step, ... of it, so
// that blocks differ by one row at most, wherever the scored ones lie in the stream.  A
// warp's lanes hold 32 entries, the next 32 on their way; all warps of a block walk alike.
struct RowWalk {
  const int2* const list;
  const int64_t first, step, count;
  int64_t base = 0;
  int2 now, then;
  int at = 0;

  __device__ __forceinline__ RowWalk(const RowArgs& a, int log_ranks)
      : list(a.list), first(blockIdx.x >> log_ranks), step(gridDim.x >> log_ranks),
        count(*(volatile const int32_t*)&a.hdr->n_items) {
    now = entry(threadIdx.x & 31);
    then = entry(32 + (threadIdx.x & 31));
  }
  __device__ __forceinline__ int2 entry(int64_t i) const {
    const int64_t k = first + i * step;
    return k < count ? __ldcg(list + k) : make_int2(-1, -1);
  }
  __device__ __forceinline__ bool next(int64_t& t, int& y) {
    if (at == 32) {
      base += 32;
      now = then;
      then = entry(base + 32 + (threadIdx.x & 31));
      at = 0;
    }
    t = __shfl_sync(0xffffffffu, now.x, at);
    y = __shfl_sync(0xffffffffu, now.y, at);
    if (t < 0) return false;
    ++at;
    return true;
  }
};

// The copies: `row` is the thread's first vector of the row ahead.  The rows on their way
// wait in a queue of every warp's own.
template <typename T, int THREADS>
struct RowCopies {
  const RowArgs& a;
  const int rank, log_ranks;
  RowWalk walk;
  uint4* const ring;                                 // the thread's first place
  int2* const queue;                                 // the warp's [16]
  const uint4* row = nullptr;
  int left = 0, queued = 0;
  bool more = true;

  __device__ __forceinline__ RowCopies(const RowArgs& a, int rank, int log_ranks, uint4* ring, int2* queue)
      : a(a), rank(rank), log_ranks(log_ranks), walk(a, log_ranks), ring(ring), queue(queue) {}
  __device__ __forceinline__ void next_row() {
    int64_t t;
    int y;
    more = more && walk.next(t, y);
    left = 0;
    if (!more) return;
    const Row<T> r = row_of<T>(a, t, rank, log_ranks);
    row = reinterpret_cast<const uint4*>(r.x + r.head) + r.vec;
    left = r.left;
    if ((threadIdx.x & 31) == 0) queue[queued & 15] = make_int2((int)t, y);
    ++queued;
  }
  // vector i of the row ahead; where it has none the place holds -infinity
  __device__ __forceinline__ void copy(int slot, int i) {
    if (!more) return;
    uint4* const to = ring + slot * THREADS;
    if (i * THREADS < left) copy16(to, row + i * THREADS);
    else *to = make_uint4(Raw<T>::kNegInf, Raw<T>::kNegInf, Raw<T>::kNegInf, Raw<T>::kNegInf);
  }
};

// One element more.
__device__ __forceinline__ void join_element(float& m, float& s, float x, const RowArgs& a) {
  const float m1 = ceilf(x * a.c);
  join(m, s, m1, m1 == -INFINITY ? 0.f : ex2(fmaf(x, a.c_lo, fmaf(x, a.c, -m1))));
}

// A thread's part of a row's sum, and the logit of the row's target if it is the thread's.
template <typename T>
struct RowSum {
  float m = -INFINITY, s = 0.f;

  // G vectors more
  template <int G>
  __device__ __forceinline__ void add(const uint4 (&u)[G], float c, const Scale2& c2) {
    float top = Raw<T>::top(u[0]);
#pragma unroll
    for (int i = 1; i < G; ++i) top = fmaxf(top, Raw<T>::top(u[i]));
    const float m1 = fmaxf(m, ceilf(top * c)), n1 = m1 == -INFINITY ? 0.f : -m1;
    const uint64_t n2 = f2_pack(n1, n1);
    uint64_t acc[2] = {f2_pack(s * pow2(m + n1), 0.f), 0};
    m = m1;
#pragma unroll
    for (int i = 0; i < G; ++i) acc[i & 1] = add_exps<T>(u[i], c2, n2, acc[i & 1]);
    float s1;
    f2_unpack(f2_add(acc[0], acc[1]), s, s1);
    s += s1;
  }
};

template <typename T>
__device__ __forceinline__ float element(const uint4& u, int k) {
  float e[Vec<T>::N], x = 0.f;
  Vec<T>::unpack(u, e);
#pragma unroll
  for (int j = 0; j < Vec<T>::N; ++j) x = j == k ? e[j] : x;
  return x;
}

// Scores alone: a row a block, in groups of kGroup vectors of a thread.  A warp leaves its
// part of a row in shared memory and goes on; one warp of the block, another for every
// row, waits for the others' parts at one of kOpen barriers and joins them.  Before a
// barrier and its places are used again the whole block meets.
constexpr int kOpen = 8;
__device__ __forceinline__ void arrive_at(int barrier, int threads) {
  asm volatile("barrier.cta.arrive.aligned %0, %1;" ::"r"(barrier), "r"(threads) : "memory");
}
__device__ __forceinline__ void wait_at(int barrier, int threads) {
  asm volatile("barrier.cta.sync.aligned %0, %1;" ::"r"(barrier), "r"(threads) : "memory");
}
constexpr int kGroup = 4, kGroups = kScoreSlots / kGroup;
template <typename T>
__global__ void __launch_bounds__(kScoreThreads, 1) score_ring_kernel(const __grid_constant__ RowArgs a,
                                                                     const int groups) {
  constexpr int N = Vec<T>::N, kLogN = N == 8 ? 3 : 2;
  extern __shared__ __align__(16) uint4 s_ring[];
  constexpr int kWarps = kScoreThreads / 32;
  __shared__ float2 s_part[kOpen][kWarps];
  __shared__ float s_target[kOpen];
  __shared__ int2 s_queue[kWarps][16];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const float c = a.c;
  const Scale2 c2(a);
  grid_dep_wait();
  RowCopies<T, kScoreThreads> ahead(a, 0, 0, s_ring + tid, s_queue[warp]);
  int g_ahead = 0;
  auto copy_group = [&](int slot) {
    if (g_ahead == 0) ahead.next_row();
#pragma unroll
    for (int i = 0; i < kGroup; ++i) ahead.copy(slot + i, g_ahead * kGroup + i);
    copy_commit();
    g_ahead = g_ahead + 1 == groups ? 0 : g_ahead + 1;
  };
  for (int i = 0; i < kGroups; ++i) copy_group(i * kGroup);
  int slot = 0;
  for (int taken = 0; taken < ahead.queued; ++taken) {
    if (taken > 0 && taken % kOpen == 0) __syncthreads();
    __syncwarp();
    const int2 item = s_queue[warp][taken & 15];
    __syncwarp();
    const int64_t t = item.x;
    const int y = item.y, par = taken % kOpen;
    const Row<T> r = row_of<T>(a, t, 0, 0);
    const bool extra = tid < a.vocab - r.nvec * N;
    const int ecol = tid < r.head ? tid : r.nvec * N + tid;
    const float xe = extra ? to_f(r.x[ecol]) : -INFINITY;
    // the target's vector among the thread's, if it is one of them, and where in it
    const unsigned dist = (unsigned)((y - r.head) >> kLogN) - (unsigned)tid;
    const int mine = y >= r.head && (int)dist < r.left && dist % kScoreThreads == 0 ? (int)(dist / kScoreThreads) : -1;
    RowSum<T> sum;
    for (int g = 0; g < groups; ++g) {
      copy_wait<kGroups - 1>();
      uint4 u[kGroup];
#pragma unroll
      for (int i = 0; i < kGroup; ++i) {
        u[i] = ahead.ring[(slot + i) * kScoreThreads];

      }
      if (mine >= g * kGroup && mine < (g + 1) * kGroup)
        s_target[par] = element<T>(ahead.ring[(slot + mine - g * kGroup) * kScoreThreads], (y - r.head) & (N - 1));
      sum.add(u, c, c2);
      copy_group(slot);
      slot = slot + kGroup == kScoreSlots ? 0 : slot + kGroup;
    }
    float m = sum.m, s = sum.s;
    if (extra) {
      join_element(m, s, xe, a);
      if (ecol == y) s_target[par] = xe;
    }
    if (tid == 0 && y >= a.vocab) s_target[par] = NAN;
    join_warp(m, s);
    if (lane == 0) s_part[par][warp] = make_float2(m, s);
    __syncwarp();
    if (warp != taken % kWarps) {
      arrive_at(1 + par, kScoreThreads);
      continue;
    }
    wait_at(1 + par, kScoreThreads);
    m = -INFINITY;
    s = 0.f;
    if (lane < kWarps) {
      m = s_part[par][lane].x;
      s = s_part[par][lane].y;
    }
    join_warp(m, s);
    if (lane == 0) {
      float row_lse;
      a.logp[t] = finish(s_target[par], a, m, s, row_lse);
      if (a.lse) a.lse[t] = row_lse;
    }
  }
}

// The policy loss: a cluster of blocks a row, SLICE vectors of a thread, which stay in
// their places of the ring until the gradient has been taken from them.
template <typename T, int SLICE>
__global__ void __launch_bounds__(kPolicyThreads, 1) policy_ring_kernel(const __grid_constant__ RowArgs a,
                                                                      const int log_ranks) {
  constexpr int N = Vec<T>::N, kLogN = N == 8 ? 3 : 2;
  extern __shared__ __align__(16) uint4 s_ring[];
  __shared__ float2 s_part[2][kMaxRanks * (kPolicyThreads / 32)];
  __shared__ float2 s_target[2];                     // x: the target's logit
  __shared__ float4 s_coef;                          // p = 2^(c x + .x), gradient .y p, .z at the target
  __shared__ int2 s_queue[(kPolicyThreads / 32)][16];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, ranks = 1 << log_ranks;
  const int rank = (int)(blockIdx.x & (unsigned)(ranks - 1));
  grid_dep_wait();
  if (status_bad(a.p.hdr)) return;
  const float c = a.c;
  const Scale2 c2(a);
  RowCopies<T, kPolicyThreads> ahead(a, rank, log_ranks, s_ring + tid, s_queue[warp]);
#pragma unroll
  for (int i = 0; i < kPolicySlots; ++i) {
    if (i % SLICE == 0) ahead.next_row();
    ahead.copy(i, i % SLICE);
    copy_commit();
  }
  if (ranks > 1) {                                   // (every block of the cluster runs)
    cluster_arrive();
    cluster_wait();
  }
  // The rows without a score get their zeros between the others, evenly.
  const int64_t others = a.rows - ahead.walk.count;
  int64_t zeroed = ahead.walk.first;
  auto zero_rows = [&](int64_t upto) {
    for (; zeroed < upto; zeroed += ahead.walk.step) {
      const int64_t t = __ldcg(a.list + a.rows - 1 - zeroed).x;
      const Row<T> r = row_of<T>(a, t, rank, log_ranks);
      bool whole;
      T* const dx = gradient_row<T>(a, t, r.x, whole);
      const float zero[N] = {};
      for (int i = 0; i < r.left; i += kPolicyThreads)
        store_vec<T>(dx + r.head + (int64_t)(r.vec + i) * N, whole, zero);
      if (rank == 0 && tid < a.vocab - r.nvec * N) st_out(dx + (tid < r.head ? tid : r.nvec * N + tid), 0.f);
    }
  };
  // (others / count of them a scored row, as the entries of both kinds are spread alike)
  const float share = ahead.walk.count > 0 ? (float)others / (float)ahead.walk.count : 0.f;
  int slot0 = 0;                                     // the row's first place
  for (int taken = 0; taken < ahead.queued; ++taken) {
    __syncwarp();
    const int2 item = s_queue[warp][taken & 15];
    __syncwarp();
    const int64_t t = item.x;
    const int y = item.y, par = taken & 1;
    const Row<T> r = row_of<T>(a, t, rank, log_ranks);
    const bool extra = rank == 0 && tid < a.vocab - r.nvec * N;
    const int ecol = tid < r.head ? tid : r.nvec * N + tid;
    const float xe = extra ? to_f(r.x[ecol]) : -INFINITY;
    const unsigned dist = (unsigned)((y - r.head) >> kLogN) - (unsigned)r.vec;
    const int mine = y >= r.head && (int)dist < r.left && dist % kPolicyThreads == 0 ? (int)(dist / kPolicyThreads) : -1;
    const int yi = (y - r.head) & (N - 1);
    PolicyScalars sc = {};
    if (warp == 0) {
      const float2 w = __ldg(a.p.row_scalars + t);
      sc = {w.x, w.y, __ldg(a.p.old_logp + t), a.p.ref_logp != nullptr ? __ldg(a.p.ref_logp + t) : 0.f};
    }
    auto publish = [&](float x) {
      if (ranks > 1) {
        for (int k = 0; k < ranks; ++k) st_peer(&s_target[par], k, make_float2(x, 0.f));
      } else {
        s_target[par].x = x;
      }
    };
    auto place = [&](int i) {
      const int p = slot0 + i;
      return p >= kPolicySlots ? p - kPolicySlots : p;
    };
    RowSum<T> sum;
    constexpr int G = SLICE % 2 == 0 ? 2 : 1;
    // (kPolicySlots - 1 - i groups are behind vector i of the row)
    auto add = [&](int i) {
      uint4 u[G];
#pragma unroll
      for (int j = 0; j < G; ++j) {
        u[j] = ahead.ring[place(i + j) * kPolicyThreads];
        if (mine == i + j) publish(element<T>(u[j], yi));
      }
      sum.add(u, c, c2);
    };
#define NSP_WAIT_ADD(i)                          \
  if constexpr ((i) < SLICE) {                   \
    copy_wait<kPolicySlots - (i) - G>();               \
    add(i);                                      \
  }
    if constexpr (G == 2) {
      NSP_WAIT_ADD(0) NSP_WAIT_ADD(2) NSP_WAIT_ADD(4) NSP_WAIT_ADD(6)
    } else {
      NSP_WAIT_ADD(0) NSP_WAIT_ADD(1) NSP_WAIT_ADD(2) NSP_WAIT_ADD(3)
      NSP_WAIT_ADD(4) NSP_WAIT_ADD(5) NSP_WAIT_ADD(6) NSP_WAIT_ADD(7)
    }
#undef NSP_WAIT_ADD
    float m = sum.m, s = sum.s;
    if (extra) {
      join_element(m, s, xe, a);
      if (ecol == y) publish(xe);
    }
    if (tid == 0 && rank == 0 && y >= a.vocab) publish(NAN);
    join_warp(m, s);
    // (two sets of states in turn: a block that writes the next row's but one has passed the
    // next row's barrier, and so has every block of the cluster, behind reading this row's)
    if (ranks > 1) {
      if (lane < ranks) st_peer(&s_part[par][rank * (kPolicyThreads / 32) + warp], lane, make_float2(m, s));
      __syncwarp();
      cluster_arrive();
      cluster_wait();
    } else {
      if (lane == 0) s_part[par][warp] = make_float2(m, s);
      __syncthreads();
    }
    if (warp == 0) {                  // one warp for all: the others' issue slots are dear
      m = -INFINITY;
      s = 0.f;
      for (int i = lane; i < ranks * (kPolicyThreads / 32); i += 32) join(m, s, s_part[par][i].x, s_part[par][i].y);
      join_warp(m, s);
      float row_lse;
      const float logp = finish(s_target[par].x, a, m, s, row_lse);
      const PolicyRow pr = policy_row(a.p, sc, logp);
      if (lane == 0) {
        const float sg = y < a.vocab ? a.scale * pr.grad : NAN;
        s_coef = make_float4(m == -INFINITY ? 0.f : -m, -sg / s, sg, 0.f);
        if (rank == 0) {
          if (a.logp) a.logp[t] = logp;
          a.p.terms[t] = pr.surrogate;
          a.p.terms[a.rows + t] = pr.kl;
          a.p.terms[2 * a.rows + t] = pr.clipped;
        }
      }
    }
    __syncthreads();
    const float4 coef = s_coef;        // (written again behind the next row's barrier)
    const float n = coef.x, f = coef.y, sg = coef.z;
    const uint64_t n2 = f2_pack(n, n), ff = f2_pack(f, f);
    bool whole;
    T* const dx = gradient_row<T>(a, t, r.x, whole);
    T* const out = dx + r.head + (int64_t)r.vec * N;
#pragma unroll
    for (int i = 0; i < SLICE; ++i) {
      if (i * kPolicyThreads < r.left) {
        const uint4 u = ahead.ring[place(i) * kPolicyThreads];
        float o[N];
        Vec<T>::unpack(u, o);
#pragma unroll
        for (int j = 0; j < N / 2; ++j) {
          float p, q;
          f2_unpack(exponents<T>(f2_pack(o[2 * j], o[2 * j + 1]), c2, n2), p, q);
          f2_unpack(f2_mul(f2_pack(ex2(p), ex2(q)), ff), o[2 * j], o[2 * j + 1]);
        }
        if (i == mine) {
#pragma unroll
          for (int j = 0; j < N; ++j) o[j] += j == yi ? sg : 0.f;
        }
        store_vec<T>(out + i * kPolicyThreads * N, whole, o);
      }
      // the place takes the vector kPolicySlots further on
      if ((kPolicySlots + i) % SLICE == 0) ahead.next_row();
      ahead.copy(place(i), (kPolicySlots + i) % SLICE);
      copy_commit();
    }
    if (extra) st_out(dx + ecol, ex2(fmaf(xe, a.c_lo, fmaf(xe, c, n))) * f + (ecol == y ? sg : 0.f));
    slot0 = place(SLICE);
    zero_rows(min(others, (int64_t)(share * (float)(taken + 1) * (float)ahead.walk.step)));
  }
  zero_rows(others);
}

// Dynamic shared memory of a ring kernel, allowed once a device.
template <typename K>
cudaError_t allow_ring(K kern, bool (&allowed)[64], int& dev) {
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess || (dev < 64 && allowed[dev])) return e;
  e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingBytes);
  if (e == cudaSuccess && dev < 64) allowed[dev] = true;
  return e;
}

template <typename T>
cudaError_t go_score_ring(const RowArgs& a, cudaStream_t s) {
  static bool allowed[64] = {};
  int dev = 0;
  cudaError_t e = allow_ring(score_ring_kernel<T>, allowed, dev);
  if (e == cudaSuccess) e = launch_row_list(a, s);
  if (e != cudaSuccess) return e;
  const int64_t nvec = std::max(1, a.vocab / Vec<T>::N);
  const int64_t blocks = std::min<int64_t>(a.rows, num_sms());
  count_launches(1);
  return launch_dependent(score_ring_kernel<T>, dim3((unsigned)blocks), dim3(kScoreThreads), kRingBytes, s, a,
                          (int)ceil_div(nvec, kGroup * kScoreThreads));
}

template <typename T, int SLICE>
cudaError_t go_policy_ring(const RowArgs& a, int log_ranks, cudaStream_t s) {
  static bool allowed[64] = {};
  static int resident[64][4] = {};
  auto kern = policy_ring_kernel<T, SLICE>;
  int dev = 0;
  cudaError_t e = allow_ring(kern, allowed, dev);
  if (e != cudaSuccess) return e;
  const int ranks = 1 << log_ranks;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)(num_sms() / ranks * ranks));
  cfg.blockDim = dim3(kPolicyThreads);
  cfg.dynamicSmemBytes = kRingBytes;
  cfg.stream = s;
  cudaLaunchAttribute attr[2];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)ranks;
  attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
  attr[1].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[1].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  // the clusters that run at once: one that had to wait for others would double the time
  int fit = dev < 64 ? resident[dev][log_ranks] : 0;
  if (fit == 0) {
    cfg.numAttrs = 1;
    e = cudaOccupancyMaxActiveClusters(&fit, kern, &cfg);
    if (e != cudaSuccess) return e;
    if (fit < 1) return cudaErrorInvalidConfiguration;
    if (dev < 64) resident[dev][log_ranks] = fit;
  }
  cfg.gridDim.x = (unsigned)(std::min<int64_t>(std::min<int64_t>(fit, num_sms() / ranks), a.rows) * ranks);
  cfg.numAttrs = 2;
  count_launches(1);
  return cudaLaunchKernelEx(&cfg, kern, a, log_ranks);
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

// Blocks of a policy row's cluster, as a power of two, and vectors of a thread; false
// where the ring has no room for the row.
bool policy_slice(int64_t nvec, int& log_ranks, int64_t& slice) {
  log_ranks = 0;
  while (log_ranks < 3 && nvec > ((int64_t)kMaxSlice * kPolicyThreads << log_ranks)) ++log_ranks;
  slice = ceil_div(ceil_div(nvec, 1 << log_ranks), kPolicyThreads);
  return slice <= kMaxSlice;
}

// Many rows of more than 64 KB go through the ring.  Scores and policy step of rows 30 %
// unscored, in us, ring against registers: 8000 rows of 1024 vectors 85 and 132 against 25
// and 55; 4000 of 4096 50 and 115 against 44 and 99; 4000 of 5000 69 and 131 against 87 and
// 161; 2000 of 16384 76 and 181 against 101 and 214 (bf16; float32 alike).
constexpr int64_t kRingVectors = 4096;
bool listed(const RowArgs& a, RowMode mode, int64_t nvec) {
  if (mode == kRowBackward || nvec <= kRingVectors) return false;
  int log_ranks = 0;
  int64_t slice;
  if (mode == kRowPolicy && !policy_slice(nvec, log_ranks, slice)) return false;
  return (a.rows << log_ranks) >= (int64_t)num_sms() * 4;
}

template <typename T, RowMode MODE>
cudaError_t launch_mode(const RowArgs& a, cudaStream_t s) {
  const int64_t nvec = std::max(1, a.vocab / Vec<T>::N);
  if (listed(a, MODE, nvec)) {
    if constexpr (MODE == kRowForward) {
      return go_score_ring<T>(a, s);
    } else if constexpr (MODE == kRowPolicy) {
      int log_ranks;
      int64_t slice;
      policy_slice(nvec, log_ranks, slice);
      const cudaError_t e = launch_loss_rows(a, s);
      if (e != cudaSuccess) return e;
      // (a ring's row is longer than four vectors of a thread)
      if (slice <= 6) return go_policy_ring<T, 6>(a, log_ranks, s);
      return go_policy_ring<T, 8>(a, log_ranks, s);
    }
  }
  // Many rows: as few threads a row as hold it in eight vectors each, so that many rows are
  // on an SM at once; a row longer than 64 KB over a cluster.
  if (a.rows >= (int64_t)num_sms() * 4) {
    if (nvec <= 64) return go<T, MODE, 32, 2>(a, 1, s);
    if (nvec <= 128) return go<T, MODE, 32, 4>(a, 1, s);
    if (nvec <= 256) return go<T, MODE, 64, 4>(a, 1, s);
    if (nvec <= 512) return go<T, MODE, 128, 4>(a, 1, s);
    if (nvec <= 768) return go<T, MODE, 128, 6>(a, 1, s);
    if (nvec <= 1024) return go<T, MODE, 128, 8>(a, 1, s);
    if (nvec <= 1536) return go<T, MODE, 256, 6>(a, 1, s);
    if (nvec <= 2048) return go<T, MODE, 256, 8>(a, 1, s);
  }
  if (nvec <= 128) return go<T, MODE, 128, 1>(a, 1, s);
  // Few: every SM a part of them.
  int ranks = 1;
  while (ranks < kMaxRanks && nvec > (int64_t)ranks * 4096) ranks *= 2;
  while (ranks < kMaxRanks && a.rows * ranks < (int64_t)num_sms() * 2 && nvec > (int64_t)ranks * 512) ranks *= 2;
  if (a.rows * ranks > INT32_MAX) ranks = 1;
  const int64_t per = ceil_div(nvec, ranks);
  if (per <= 512) return go<T, MODE, 512, 1>(a, ranks, s);
  if (per <= 1024) return go<T, MODE, 512, 2>(a, ranks, s);
  if (per <= 2048) return go<T, MODE, 512, 4>(a, ranks, s);
  if (per <= 512 * 6) return go<T, MODE, 512, 6>(a, ranks, s);
  return go<T, MODE, 512, 8>(a, ranks, s);
}

template <typename T>
cudaError_t launch_typed(const RowArgs& a, RowMode mode, cudaStream_t s) {
  if (mode == kRowForward) return launch_mode<T, kRowForward>(a, s);
  if (mode == kRowBackward) return launch_mode<T, kRowBackward>(a, s);
  return launch_mode<T, kRowPolicy>(a, s);
}

}  // namespace

bool rows_listed(const RowArgs& a, RowMode mode, int32_t io_dtype) {
  return listed(a, mode, std::max(1, a.vocab / (io_dtype == NSP_BF16 ? 8 : 4)));
}

cudaError_t launch_rows(const RowArgs& a, RowMode mode, int32_t io_dtype, cudaStream_t s) {
  return io_dtype == NSP_BF16 ? launch_typed<__nv_bfloat16>(a, mode, s) : launch_typed<float>(a, mode, s);
}

}  // namespace nsp
