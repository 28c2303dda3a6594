// Rotary positions of a packed stream: every token's heads rotated by angles
// that grow with the token's position inside its own document.
//
// With f_i the frequency of pair i (radians per position) and a = pos f_i,
//   u = m (x_a cos a - x_b sin a),  w = m (x_a sin a + x_b cos a),
// and, inverse, the transpose (a -> -a): the backward of the rotation.
//
// Angles.  A far position times a frequency near 1 needs more bits than
// float32 has (position 400000: an angle error of 0.03).  The frequency is
// converted once per block to a fixed-point fraction of a turn, 2^-64 turns
// per unit, so that position x frequency is one integer product whose wrap
// modulo 2^64 is the reduction modulo whole turns, exactly; its top 32 bits,
// signed, are the angle in [-1/2, 1/2) turns, cut off by at most 2^-32 turns.  Two
// errors are larger: the frequency as a fraction of a turn is a float64 product,
// 2^-52 of the whole angle (2^-36 turns at position 400000 and frequency 1), and the 32
// bits are rounded to float32 for the sine, 2^-26 turns at most.
//
// Bound: HBM, one read and one write of every element.  A team of threads
// owns one token and a 16-byte piece of a head each (both pieces of the pair
// with halves), computes the sines and cosines of its pairs once and walks
// the token's heads with four heads' loads in flight.  With few tokens the
// heads of one token are split over several teams, so that a single token
// still spreads over the GPU.  32768 tokens, 32 + 4 heads of 128 bf16 columns read
// from the fused projection: 91 us, 6.6 TB/s; 8191 tokens, 16 + 4 heads of 64 float32
// columns, half of them rotated in interleaved pairs: 10.4 us when its 84 MB are in L2,
// and a call takes the host 21 us.
#include <algorithm>

#include "rotary.cuh"

namespace nsp {
namespace {

constexpr int kThreads = 256;
constexpr int kHeadsInFlight = 4;
constexpr int64_t kL2Bytes = (int64_t)128 << 20;

__device__ __forceinline__ bool position_of(const RopeArgs& a, int64_t t, int64_t& pos) {
  return position_of(Positions{a.positions, a.cu, a.ndoc, a.start}, t, pos);
}

// Where a team's piece of the current head is read and written: heads of one
// tensor (and head group) follow one another, d elements apart.
template <typename T>
struct Cursor {
  const T* src;
  T* dst;
  int k, h, left;                     // tensor, head in it, heads until the next jump

  __device__ __forceinline__ void place(const RopeArgs& a, int64_t t, int col) {
    const RopeTensor& r = a.t[k];
    src = reinterpret_cast<const T*>(r.in) + col +
          row_offset(t, h, r.in_stride, r.heads, r.in_groups, a.len, a.d);
    dst = reinterpret_cast<T*>(r.out) + col +
          row_offset(t, h, r.out_stride, r.heads, r.out_groups, a.len, a.d);
    left = r.hpg - h % r.hpg;
  }
  __device__ __forceinline__ void start(const RopeArgs& a, int64_t t, int head, int col) {
    k = 0;
    while (head >= a.t[k].heads) head -= a.t[k++].heads;
    h = head;
    place(a, t, col);
  }
  __device__ __forceinline__ void next(const RopeArgs& a, int64_t t, int col) {
    ++h;
    src += a.d;
    dst += a.d;
    if (--left > 0) return;
    const RopeTensor& r = a.t[k];
    if (h < r.heads) {                // the next head group of the same tensor
      left = r.hpg;
      src += r.in_jump;
      dst += r.out_jump;
      return;
    }
    h = 0;
    if (++k < a.n) place(a, t, col);  // (else past the last head)
  }
};

// Pieces of one head: INTERLEAVED: rot / N rotated vectors of whole pairs;
// halves: rot / 2 / N pairs of vectors; then the (d - rot) / N unrotated
// vectors, copied.
template <typename T, bool INTERLEAVED>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ RopeArgs a,
                                                        int pieces, int rotated, int total_heads,
                                                        int hsplit) {
  constexpr int N = Vec<T>::N;
  constexpr int kPairs = INTERLEAVED ? N / 2 : N;    // pairs of one rotated piece
  __shared__ uint64_t s_fx[kRopeMaxDim / 2];
  for (int i = threadIdx.x; i < a.rot / 2; i += blockDim.x) s_fx[i] = fixed_turns(a.freqs[i]);
  __syncthreads();
  const int teams = blockDim.x / pieces;
  const int team = threadIdx.x / pieces, u = threadIdx.x - team * pieces;
  if (team >= teams) return;
  const int64_t items = a.len * hsplit;
  const int per = (total_heads + hsplit - 1) / hsplit;
  const int half = a.rot / 2;
  for (int64_t item = (int64_t)blockIdx.x * teams + team; item < items;
       item += (int64_t)gridDim.x * teams) {
    const int64_t t = hsplit == 1 ? item : (int64_t)((uint32_t)item / (uint32_t)hsplit);
    const int part = (int)(item - t * hsplit);
    const bool rot = u < rotated;
    float c[kPairs], s[kPairs];
    // column of the piece's first vector
    const int col = rot ? u * N : a.rot + (u - rotated) * N;
    bool turned = false;                     // the token's angles are there
    const int h_end = min((part + 1) * per, total_heads);
    if (part * per >= total_heads) continue;
    Cursor<T> at;
    at.start(a, t, part * per, col);
    for (int h0 = part * per; h0 < h_end; h0 += kHeadsInFlight) {
      uint4 x[kHeadsInFlight], y[kHeadsInFlight];
      T* dst[kHeadsInFlight];
#pragma unroll
      for (int i = 0; i < kHeadsInFlight; ++i) {
        if (h0 + i >= h_end) break;
        x[i] = ld_once(at.src);
        if (!INTERLEAVED && rot) y[i] = ld_once(at.src + half);
        dst[i] = at.dst;
        at.next(a, t, col);
      }
      if (!turned) {                         // under the first loads
        int64_t pos;
        if (!position_of(a, t, pos)) break;
        turned = true;
        if (rot) {
#pragma unroll
          for (int i = 0; i < kPairs; ++i)
            turn(pos, s_fx[u * kPairs + i], a.mscale, a.inverse != 0, c[i], s[i]);
        }
      }
#pragma unroll
      for (int i = 0; i < kHeadsInFlight; ++i) {
        if (h0 + i >= h_end) break;
        if (!rot) {
          st_once(dst[i], x[i]);
          continue;
        }
        float p[N], q[N];
        Vec<T>::unpack(x[i], p);
        if constexpr (INTERLEAVED) {
#pragma unroll
          for (int j = 0; j < N / 2; ++j) {
            q[2 * j] = p[2 * j] * c[j] - p[2 * j + 1] * s[j];
            q[2 * j + 1] = p[2 * j] * s[j] + p[2 * j + 1] * c[j];
          }
          st_once(dst[i], Vec<T>::pack(q));
        } else {
          Vec<T>::unpack(y[i], q);
#pragma unroll
          for (int j = 0; j < N; ++j) {
            const float b = q[j];
            q[j] = p[j] * s[j] + b * c[j];
            p[j] = p[j] * c[j] - b * s[j];
          }
          st_once(dst[i], Vec<T>::pack(p));
          st_once(dst[i] + half, Vec<T>::pack(q));
        }
      }
    }
  }
}

// Sizes, strides or addresses that do not allow 16-byte pieces: one pair (or
// one unrotated element) per thread.
template <typename T>
__global__ void __launch_bounds__(kThreads) rope_element_kernel(const __grid_constant__ RopeArgs a,
                                                                int total_heads) {
  const int half = a.rot / 2, units = half + a.d - a.rot;
  const int64_t n = a.len * total_heads * units;
  for (int64_t e = (int64_t)blockIdx.x * kThreads + threadIdx.x; e < n;
       e += (int64_t)gridDim.x * kThreads) {
    const int64_t th = e / units, t = th / total_heads;
    const int u = (int)(e - th * units);
    int h = (int)(th - t * total_heads), k = 0;
    int64_t pos;
    if (!position_of(a, t, pos)) continue;
    while (h >= a.t[k].heads) h -= a.t[k++].heads;
    const RopeTensor& r = a.t[k];
    const T* src = reinterpret_cast<const T*>(r.in) +
                   row_offset(t, h, r.in_stride, r.heads, r.in_groups, a.len, a.d);
    T* dst = reinterpret_cast<T*>(r.out) +
             row_offset(t, h, r.out_stride, r.heads, r.out_groups, a.len, a.d);
    if (u >= half) {
      dst[a.rot + u - half] = src[a.rot + u - half];
      continue;
    }
    const int ia = a.interleaved ? 2 * u : u, ib = a.interleaved ? 2 * u + 1 : u + half;
    float c, s;
    turn(pos, fixed_turns(a.freqs[u]), a.mscale, a.inverse != 0, c, s);
    const float xa = to_f(src[ia]), xb = to_f(src[ib]);
    st_out(dst + ia, xa * c - xb * s);
    st_out(dst + ib, xa * s + xb * c);
  }
}

template <typename T>
bool vector_ok(const RopeArgs& a) {
  constexpr int N = 16 / (int)sizeof(T);
  if (a.d % N != 0 || (a.interleaved ? a.rot : a.rot / 2) % N != 0) return false;
  for (int i = 0; i < a.n; ++i) {
    const RopeTensor& r = a.t[i];
    if (((reinterpret_cast<uintptr_t>(r.in) | reinterpret_cast<uintptr_t>(r.out)) & 15) != 0)
      return false;
    if (r.in_stride % N != 0 || r.out_stride % N != 0) return false;
  }
  return true;
}

template <typename T>
cudaError_t launch_typed(const RopeArgs& a, cudaStream_t s) {
  int heads = 0;
  for (int i = 0; i < a.n; ++i) heads += a.t[i].heads;
  const int64_t nsm = num_sms();
  if (!vector_ok<T>(a)) {
    const int64_t n = a.len * heads * (a.d - a.rot / 2);
    const int64_t blocks = std::min<int64_t>(ceil_div(n, kThreads), nsm * 16);
    rope_element_kernel<T><<<(unsigned)blocks, kThreads, 0, s>>>(a, heads);
  } else {
    constexpr int N = 16 / (int)sizeof(T);
    const int rotated = (a.interleaved ? a.rot : a.rot / 2) / N;
    const int pieces = rotated + (a.d - a.rot) / N;
    // 128 threads, or as many pieces as a head has: with 256 a stream of few blocks
    // waits longer for its last ones (8191 tokens, 20 heads of 64 float32: 13.6 us against
    // 10.4; 32768 tokens, 36 heads of 128 bf16: 94.0 against 93.0)
    const int threads = pieces > kThreads / 2 ? kThreads : kThreads / 2;
    const int teams = threads / pieces;
    // A token's heads are split over several teams, each with its own search and angles,
    // for two blocks of an SM only (16 blocks: 14.6 us of the first stream above), and
    // in parts of 12 heads or more for a stream that does not fit in L2, whose rows in flight
    // then lie closer together (the second one: 90.4 us in three parts, 93.0 in one)
    const int64_t bytes = 2 * a.len * heads * a.d * (int64_t)sizeof(T);
    int64_t hsplit = ceil_div(nsm * 2 * teams, a.len);
    if (bytes > kL2Bytes) hsplit = std::max<int64_t>(hsplit, heads / 12);
    hsplit = std::min<int64_t>(hsplit, heads);
    if (a.len * hsplit > UINT32_MAX) hsplit = 1;     // the kernel divides split items in 32 bits
    // (one item a team where 128 blocks of an SM allow it: no block is left with one
    // more item than the others at the end)
    const int64_t blocks = std::min<int64_t>(ceil_div(a.len * hsplit, teams), nsm * 128);
    if (a.interleaved)
      rope_kernel<T, true><<<(unsigned)blocks, threads, 0, s>>>(a, pieces, rotated, heads, (int)hsplit);
    else
      rope_kernel<T, false><<<(unsigned)blocks, threads, 0, s>>>(a, pieces, rotated, heads, (int)hsplit);
  }
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_rope(const RopeArgs& a, int32_t io_dtype, cudaStream_t s) {
  return io_dtype == NSP_BF16 ? launch_typed<__nv_bfloat16>(a, s) : launch_typed<float>(a, s);
}

}  // namespace nsp
