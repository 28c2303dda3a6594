// What the tensor-core kernels of differential attention share.
#pragma once

#include <limits.h>

#include <atomic>

#include "layer.cuh"
#include "tc_ptx.cuh"

namespace nsp {
namespace tc {

constexpr uint32_t kBlk = 128 * 64 * 2;               // 128 rows x 64 bf16 column block
constexpr uint32_t kTile = 2 * kBlk;                   // 128 x 128 bf16
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr size_t kSmemLimit = 232448;

// One arrival of the warp, by lane 0, without a branch.  The caller's
// __syncwarp orders the other lanes' accesses before it.
__device__ __forceinline__ void mbar_arrive_warp(uint64_t* bar, int lane) {
  __syncwarp();
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "setp.eq.s32 p, %1, 0;\n\t"
      "@p mbarrier.arrive.shared::cta.b64 _, [%0];\n\t}" ::"r"(smem_u32(bar)), "r"(lane)
      : "memory");
}

__device__ __forceinline__ bool mbar_test(uint64_t* bar, uint32_t parity) {
  uint32_t ok;
  asm volatile(
      "{\n\t.reg .pred p;\n\t"
      "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
      "selp.u32 %0, 1, 0, p;\n\t}"
      : "=r"(ok)
      : "r"(smem_u32(bar)), "r"(parity)
      : "memory");
  return ok != 0;
}

// mbar_wait and mbar_wait_warp with a first look that neither suspends the
// thread nor reads the wait's bound: many phases are complete by then.
// (Polling for longer costs more than the wake-up of a suspended thread: 10 %
// of the forward's time, as the polls take issue slots from the softmax.)
__device__ __forceinline__ bool wait_one(uint64_t* bar, uint32_t parity, WaitCtl* wc, WsHeader* hdr) {
  return mbar_test(bar, parity) || mbar_wait(bar, parity, wc, hdr);
}
__device__ __forceinline__ bool wait_warp(uint64_t* bar, uint32_t parity, WaitCtl* wc, WsHeader* hdr) {
  if (__all_sync(0xffffffffu, mbar_test(bar, parity))) return true;
  return mbar_wait_warp(bar, parity, wc, hdr);
}

// Document [first, last) of stream row t0 + (lane >> shift), for a whole warp (rows at or
// past `rows` get the document of the last row below): the warp narrows the
// search 32-fold with each load, then reads the next documents' starts in one:
// three dependent loads for a thousand documents instead of ten.
struct Span32 {
  int first, last;
};
__device__ __forceinline__ Span32 document_of_rows(const int32_t* __restrict__ cu, int ndoc, int64_t t0,
                                                   int64_t rows, int lane, int shift = 0) {
  int lo = 0, m = ndoc;                              // the first row's document is in [lo, lo + m)
  while (m > 1) {
    const int step = (m + 31) >> 5, at = lo + lane * step;
    const bool below = lane * step < m && (int64_t)__ldg(cu + at) <= t0;
    const int top = 31 - __clz(__ballot_sync(0xffffffffu, below) | 1u);
    lo += top * step;
    m = min(step, m - top * step);
  }
  const int64_t t = min(t0 + (lane >> shift), rows - 1);
  const int at = lo + lane;
  const int start = at <= ndoc ? __ldg(cu + at) : INT_MAX;
  int n = 0;                                         // starts passed by row t
  for (; n < 31; ++n)
    if (!__any_sync(0xffffffffu, __shfl_sync(0xffffffffu, start, n + 1) <= (int)t)) break;
  // at most n of the window's starts are passed: count this row's
  int b = 0;
  for (int j = 1; j <= n; ++j) b += __shfl_sync(0xffffffffu, start, j) <= (int)t;
  Span32 d;
  d.first = __shfl_sync(0xffffffffu, start, b);
  d.last = __shfl_sync(0xffffffffu, start, min(b + 1, 31));
  if (n == 31 && b == 31) {                          // more documents than the window holds
    const int x = doc_of(cu, ndoc, t);
    d.first = __ldg(cu + x);
    d.last = __ldg(cu + x + 1);
  }
  return d;
}

// Work item of the query-stationary kernels: 128 query rows, 2^shift heads of one
// group at 128 >> shift consecutive tokens (row r is token t0 + (r >> shift), head
// h0 + r % 2^shift), against n_kv 128-key tiles from key lo, the start of the first
// token's document; n_kv = -1 stops.
struct QueryItem {
  int t0, h0, g, lo, n_kv;
  int pad[3];
};

// Item idx (128-token tiles in `order`, Hq items each); false when its tokens lie past
// the stream (the last tile may be short).
__device__ __forceinline__ bool query_item(QueryItem& it, const AttnProblem& p, const int* order, int idx,
                                           int shift) {
  const int rest = idx % p.Hq, part = rest & ((1 << shift) - 1), tokens = 128 >> shift;
  it.t0 = order[idx / p.Hq] * 128 + part * tokens;
  if (it.t0 >= p.q_len) return false;
  it.h0 = rest - part;
  it.g = it.h0 / (p.Hq / p.Hkv);
  const int end = (int)min((int64_t)it.t0 + tokens, p.q_len);
  it.lo = __ldg(p.cu + doc_of(p.cu, p.ndoc, it.t0));
  const int hi = p.causal ? end : (int)min((int64_t)__ldg(p.cu + doc_of(p.cu, p.ndoc, end - 1) + 1), p.kv_len);
  it.n_kv = (hi - it.lo + 127) / 128;
  return true;
}

// D = A B^T over columns [m HK, (m + 1) HK) of K-major 128-row tiles (128-byte
// swizzle: 16 columns are 32 bytes of a row, 64 columns one column block).
template <int HK>
__device__ __forceinline__ void mma_kk(int m, uint32_t d_tmem, uint32_t a_saddr, uint32_t b_saddr) {
  constexpr uint32_t idesc = idesc_bf16_f32(128, 128, false, false);
  const uint64_t ad = smem_desc_sw128(a_saddr, 16, 1024);
  const uint64_t bd = smem_desc_sw128(b_saddr, 16, 1024);
#pragma unroll
  for (int i = 0; i < HK / 16; ++i) {
    const int kk = m * (HK / 16) + i;
    const uint32_t off = ((kk >> 2) * kBlk + (kk & 3) * 32) >> 4;
    mma_ss(d_tmem, ad + off, bd + off, idesc, i > 0 ? 1u : 0u);
  }
}

// Address of column n0 (a multiple of 32) of an MN-major tile's first rows.
__device__ __forceinline__ uint32_t mn_offset(int n0) {
  return (uint32_t)(n0 >> 6) * kBlk + (uint32_t)(n0 & 63) * 2;
}

// D (+)= A B, A (128 x 128) from TMEM in groups of QPG K-columns (group j at
// columns a_tmem + j QPG + [0, QPG / 2), bf16 pairs), B MN-major columns
// [n0, n0 + N) of a 128-row tile (16 rows are 2048 bytes).
template <int QPG, int N>
__device__ __forceinline__ void mma_ts_mn(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_saddr, int n0,
                                          bool accumulate) {
  constexpr int kSteps = QPG / 16;
  const uint64_t bd = smem_desc_sw128(b_saddr + mn_offset(n0), kBlk, 1024);
#pragma unroll
  for (int kk = 0; kk < 8; ++kk)
    mma_ts(d_tmem, a_tmem + (kk / kSteps) * QPG + (kk % kSteps) * 8, bd + ((kk * 2048) >> 4),
           idesc_bf16_f32(128, N, true, false), (accumulate || kk > 0) ? 1u : 0u);
}

// The same with A K-major in shared memory.
template <int N>
__device__ __forceinline__ void mma_ss_mn(uint32_t d_tmem, uint32_t a_saddr, uint32_t b_saddr, int n0,
                                          bool accumulate) {
  const uint64_t ad = smem_desc_sw128(a_saddr, 16, 1024);
  const uint64_t bd = smem_desc_sw128(b_saddr + mn_offset(n0), kBlk, 1024);
#pragma unroll
  for (int kk = 0; kk < 8; ++kk)
    mma_ss(d_tmem, ad + (((kk >> 2) * kBlk + (kk & 3) * 32) >> 4), bd + ((kk * 2048) >> 4),
           idesc_bf16_f32(128, N, true, false), (accumulate || kk > 0) ? 1u : 0u);
}

// Bits [lo, hi) of 32 columns (bounds relative to the first one, any value).
__device__ __forceinline__ uint32_t column_bits(int lo, int hi) {
  lo = min(max(lo, 0), 32);
  hi = min(max(hi, 0), 32);
  return hi <= lo ? 0u : (0xffffffffu >> (32 - hi)) & (0xffffffffu << lo);
}

// Masks of 16-bit pairs from column bits: pair j of the result covers bits
// 8 j and 8 j + 1 of `bits`, 0xffff or 0 in each half.  A masked pair of
// results is cleared whatever it holds (infinities and NaN included).
__device__ __forceinline__ void pair_masks(uint32_t bits, uint32_t (&mask)[4]) {
  const uint32_t even = bits << 7, odd = bits << 6;       // the bit at each byte's sign
  asm("prmt.b32 %0, %1, %2, 0xcc88;" : "=r"(mask[0]) : "r"(even), "r"(odd));
  asm("prmt.b32 %0, %1, %2, 0xdd99;" : "=r"(mask[1]) : "r"(even), "r"(odd));
  asm("prmt.b32 %0, %1, %2, 0xeeaa;" : "=r"(mask[2]) : "r"(even), "r"(odd));
  asm("prmt.b32 %0, %1, %2, 0xffbb;" : "=r"(mask[3]) : "r"(even), "r"(odd));
}

// dst[0..31] = scale * v (raw float32 bits) in bf16.
__device__ __forceinline__ void store_row32(__nv_bfloat16* dst, const uint32_t (&v)[32], float scale) {
  uint32_t w[16];
#pragma unroll
  for (int i = 0; i < 16; ++i)
    w[i] = pack_bf16x2(__uint_as_float(v[2 * i]) * scale, __uint_as_float(v[2 * i + 1]) * scale);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    st_global_v8(dst + 16 * i, w[8 * i], w[8 * i + 1], w[8 * i + 2], w[8 * i + 3], w[8 * i + 4],
                 w[8 * i + 5], w[8 * i + 6], w[8 * i + 7]);
}

// 1024-aligned view of dynamic shared memory, or nullptr (error recorded)
// when the aligned structure would not fit in the launch's allocation.
template <typename S>
__device__ __forceinline__ S* smem_view(uint8_t* raw, WsHeader* hdr) {
  uint32_t dyn_bytes;
  asm("mov.u32 %0, %%dynamic_smem_size;" : "=r"(dyn_bytes));
  const uint32_t base = smem_u32(raw);
  if (((base + 1023u) & ~1023u) - base + sizeof(S) > dyn_bytes) {
    if (threadIdx.x == 0) atomicExch(&hdr->status, (int)NSP_ERR_UNSUPPORTED);
    return nullptr;
  }
  return reinterpret_cast<S*>((reinterpret_cast<uintptr_t>(raw) + 1023) &
                              ~static_cast<uintptr_t>(1023));
}

template <typename S>
constexpr size_t smem_bytes() {
  return sizeof(S) + 1024 <= kSmemLimit ? sizeof(S) + 1024 : kSmemLimit;
}

__device__ __forceinline__ void tma_load_3d(void* smem_dst, const CUtensorMap* map, uint64_t* bar, int x,
                                            int y, int z) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes"
      " [%0], [%1, {%3, %4, %5}], [%2];" ::"r"(smem_u32(smem_dst)),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(x), "r"(y), "r"(z)
      : "memory");
}

// Tiled store of one box from shared memory (rows past the map's end are
// not written), tracked by the issuing thread's bulk groups.
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* map, const void* smem_src, int x, int y,
                                             int z) {
  asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.tile.bulk_group [%0, {%2, %3, %4}], [%1];" ::"l"(
                   reinterpret_cast<uint64_t>(map)),
               "r"(smem_u32(smem_src)), "r"(x), "r"(y), "r"(z)
               : "memory");
}

// Launches a persistent kernel behind the one before it, with `smem` bytes of
// dynamic shared memory (allowed once for each device and kernel; ID tells the
// file's kernels of one signature apart).
template <int ID, typename K, typename... Args>
static cudaError_t launch_persistent(K kern, int threads, size_t smem, cudaStream_t s, Args... args) {
  static std::atomic<uint64_t> allowed{0};           // one bit a device
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  if (e != cudaSuccess) return e;
  const uint64_t bit = dev < 64 ? (uint64_t)1 << dev : 0;
  if ((allowed.load(std::memory_order_relaxed) & bit) == 0) {
    e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e != cudaSuccess) return e;
    allowed.fetch_or(bit, std::memory_order_relaxed);
  }
  e = launch_dependent(kern, dim3(persistent_grid()), dim3(threads), smem, s, args...);
  count_launches(1);
  count_path(true);
  return e;
}

}  // namespace tc
}  // namespace nsp
