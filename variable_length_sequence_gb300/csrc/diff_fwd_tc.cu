// Differential attention forward on the 5th-generation tensor cores (tcgen05,
// TMEM accumulators, TMA loads): bf16 inputs, float32 scores, softmax and
// accumulation, head dimension D = 128 or 64 (two maps of D / 2 columns).
//
//   P_m = softmax(scale q_m k_m^T) over a row's visible keys,  O_m = P_m V,
//   out = O_1 - lambda O_2,  with the online softmax of Milakov and Gimelshein.
//
// Work item: 128 query rows, the 2^k heads of one group at 128 / 2^k consecutive
// tokens (k as large as the group's head count and kMaxItemHeads allow), against the
// 128-key tiles from the start of the first token's document on.  Fewer tokens of an
// item see fewer keys of other documents, and tiles that begin with a document waste
// less: 10800 tiles in place of 18400 for 454 documents of 32 to 256 tokens and 8 heads
// of a group, 14400 in place of 15900 for 19 documents around 1024 and 4 heads (whole
// calls: 300 us of one head in an item, 280 of 4, 265 of 8; 191 and 178; one long
// document: 921 and 909).  Items are taken from an atomic counter by a persistent grid of
// one CTA per SM, 128-token tiles in the schedule kernel's order (most keys first).  Both
// maps read the same Q, K and V tiles: map m is the m-th half of the columns of Q and K
// (an offset into the same shared-memory tile), V is shared whole, and the difference is
// formed in the epilogue, so no map's output goes to memory (out2 only when a backward
// follows).
//
// CTA roles (384 threads, three warpgroups):
//   warps 0-3   softmax of map 1 (one query row a thread, TMEM lanes 0-127)
//   warps 4-7   softmax of map 2
//   warp 8      TMA producer and work fetch
//   warp 9      TMEM allocation and the single MMA-issuing thread
//   warp 10     stores finished tiles (TMA, from a staging buffer)
//   warp 11     idle (completes the control warpgroup)
// Registers are moved from the control warpgroup to the softmax warpgroups
// (launched at 168: 384 x 168 = 64512 = 256 x 200 + 128 x 104; with 192 and 112
// a long document takes 909 us, not 900, with 208 and 88 short ones 292, not 265),
// enough to hold a 128-column row of S.
// TMEM (512 columns): S_1 [0,128) S_2 [128,256) O_1 [256,384) O_2 [384,512);
// P (bf16 pairs) over the first 64 columns of its S, read from there by P V.
// The tensor core alternates between the maps, so that one map's softmax
// runs under the other's products.
//
// Bound: the tensor core's issue, 24 instructions of a 128 x 128 tile of pairs and
// both maps at about 115 cycles each.  One causal document of 20001 tokens, 8 heads
// on 4, D = 128: 900 us, 1365 TFLOP/s of the visible pairs' 6 D; D = 64 has the same
// number of instructions of P V at half the columns and reaches 729.  16384 tokens
// in 19 documents, 16 heads: 178 us, 917 TFLOP/s.  454 documents of 32 to 256 tokens
// (65536 tokens, 16 heads on 2): 265 us, 2.3 TB/s; an item has 1.3 tiles of keys there,
// and the chain of its scores, softmax, product and epilogue, some 9000 cycles, has
// nothing of its own CTA beside it: TMEM holds no second item's accumulators.
//
// Rounding: P is rounded to bf16 as the product's operand; the row sums use
// the unrounded float32 values.  The running output is rescaled only when a
// row's maximum has grown by more than 2^8 (exact either way: numerator and
// denominator share the reference).  lse takes the short logarithm, 2^-22 or 2 ulp of it.
#include <cudaTypedefs.h>

#include "diff_tc.cuh"

namespace nsp {
namespace {

using namespace tc;

constexpr int BM = 128, BN = 128;
constexpr int NSTAGE = 2;
constexpr int kThreads = 384;
constexpr int kRegsSoftmax = 200, kRegsControl = 104;
constexpr int kWarpProducer = 8, kWarpMma = 9, kWarpStore = 10;
__host__ __device__ constexpr uint32_t col_s(int m) { return m == 0 ? 0u : 128u; }
__host__ __device__ constexpr uint32_t col_o(int m) { return m == 0 ? 256u : 384u; }
constexpr float kRescaleThreshold = 8.0f;                 // log2 units

struct __align__(1024) Smem {
  uint8_t q[2][kTile];                 // this item's and the next one's; then out2's tile
  uint8_t k[NSTAGE][kTile];
  uint8_t v[NSTAGE][kTile];
  uint8_t out[kTile];                  // the finished tile, 128-byte swizzled, on its way out
  float inv[2][2][BM];                 // [item parity][map][row]: 1 / row sum
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[NSTAGE], k_empty[NSTAGE], v_full[NSTAGE], v_empty[NSTAGE];
  uint64_t s_full[2], p_full[2], o_full, o_free, inv_full, out_full, out_free;
  uint64_t item_full[2], item_empty[2];
  QueryItem items[2];
  uint64_t mma_drain_bar;
  uint32_t tmem_base;
  WaitCtl wait;
};
static_assert(sizeof(Smem) <= kSmemLimit, "forward tile set exceeds shared memory");

struct FwdArgs {
  AttnProblem p;
  const __nv_bfloat16* lambda;
  int64_t n_lambda;
  const int* order;                    // 128-token tiles, most keys first
  int shift;                           // log2 of the heads of an item
};

__device__ __forceinline__ float max32(const uint32_t (&s)[32]) {
  float a = max3f(__uint_as_float(s[0]), __uint_as_float(s[1]), __uint_as_float(s[2]));
  float b = max3f(__uint_as_float(s[16]), __uint_as_float(s[17]), __uint_as_float(s[18]));
#pragma unroll
  for (int i = 3; i < 15; i += 2) {
    a = max3f(a, __uint_as_float(s[i]), __uint_as_float(s[i + 1]));
    b = max3f(b, __uint_as_float(s[16 + i]), __uint_as_float(s[17 + i]));
  }
  return max3f(fmaxf(a, b), __uint_as_float(s[15]), __uint_as_float(s[31]));
}

// Columns whose bit is not set become -inf.
__device__ __forceinline__ void mask32(uint32_t (&s)[32], uint32_t bits) {
#pragma unroll
  for (int i = 0; i < 32; ++i)
    if ((bits & (1u << i)) == 0) s[i] = 0xff800000u;
}

// p = 2^(s scale log2 e - m) of 32 columns in bf16 pairs; their float32 values
// are added to the four pairs of sums.
__device__ __forceinline__ void exps32(const uint32_t (&s)[32], uint64_t sl2x2, uint64_t nm2,
                                       uint64_t (&sum)[4], uint32_t (&p)[16]) {
#pragma unroll
  for (int i = 0; i < 16; ++i) {
    float p0, p1;
    f2_unpack(f2_fma(f2_pack(__uint_as_float(s[2 * i]), __uint_as_float(s[2 * i + 1])), sl2x2, nm2), p0,
              p1);
    p0 = ex2(p0);
    p1 = ex2(p1);
    sum[i & 3] = f2_add(sum[i & 3], f2_pack(p0, p1));
    p[i] = pack_bf16x2(p0, p1);
  }
}

// SAVE: out2 is stored too.
template <int D, bool SAVE>
__global__ void __launch_bounds__(kThreads, 1)
    diff_fwd_tc_kernel(const __grid_constant__ CUtensorMap tm_q,
                       const __grid_constant__ CUtensorMap tm_k,
                       const __grid_constant__ CUtensorMap tm_v,
                       const __grid_constant__ CUtensorMap tm_out,
                       const __grid_constant__ CUtensorMap tm_out2, const __grid_constant__ FwdArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const AttnProblem& p = a.p;
  WsHeader* hdr = p.hdr;
  grid_dep_wait();                          // the schedule kernel's lists and status
  if (block_leaves(status_bad(hdr))) return;
  Smem* smp = smem_view<Smem>(smem_raw, hdr);
  if (smp == nullptr) return;
  Smem& sm = *smp;

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.q_full[s], 1);
      mbar_init(&sm.q_empty[s], 1);
      mbar_init(&sm.s_full[s], 1);
      mbar_init(&sm.p_full[s], 128);
      mbar_init(&sm.item_full[s], 1);
      mbar_init(&sm.item_empty[s], 2 + 8);
    }
    for (int s = 0; s < NSTAGE; ++s) {
      mbar_init(&sm.k_full[s], 1);
      mbar_init(&sm.k_empty[s], 1);
      mbar_init(&sm.v_full[s], 1);
      mbar_init(&sm.v_empty[s], 1);
    }
    mbar_init(&sm.o_full, 1);
    mbar_init(&sm.o_free, 8);
    mbar_init(&sm.inv_full, 8);
    mbar_init(&sm.out_full, 8);
    mbar_init(&sm.out_free, 1);
    mbar_init(&sm.mma_drain_bar, 1);
    wait_ctl_init(&sm.wait, p.wait_budget);
    fence_mbar_init();
  }
  if (warp == kWarpMma) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  if (warp == kWarpProducer && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
    tma_prefetch_desc(&tm_out);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  const uint32_t tmem = sm.tmem_base;
  WaitCtl* const wc = &sm.wait;
  const int n_items = hdr->n_items * p.Hq;
  constexpr int kBlocks = D / 64;                               // 64-column blocks of a row
  constexpr uint32_t kLoadBytes = kBlocks * kBlk;          // one Q, K or V tile

  if (warp >= 8) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kRegsControl));
    if (warp == kWarpProducer && lane == 0) {
      // ------------------------------------------------------------ producer
      uint32_t it_count = 0, kv_count = 0;
      bool ok = true;
      while (ok) {
        const int idx = atomicAdd(&hdr->counter, 1);
        QueryItem it = {};
        it.n_kv = -1;
        if (idx < n_items && !query_item(it, p, a.order, idx, a.shift)) continue;
        // items alternate over two slots of the queue and of Q
        const uint32_t slot = it_count & 1, use = it_count >> 1;
        if (use >= 1 && !mbar_wait(&sm.item_empty[slot], (use - 1) & 1, wc, hdr)) break;
        sm.items[slot] = it;
        mbar_arrive(&sm.item_full[slot]);
        if (it.n_kv < 0) break;
        if (use >= 1 && !mbar_wait(&sm.q_empty[slot], (use - 1) & 1, wc, hdr)) break;
        mbar_arrive_expect_tx(&sm.q_full[slot], kLoadBytes);
#pragma unroll
        for (int cb = 0; cb < kBlocks; ++cb)
          tma_load_3d(sm.q[slot] + cb * kBlk, &tm_q, &sm.q_full[slot], cb * 64, it.h0, it.t0);
        ++it_count;
        for (int jj = 0; jj < it.n_kv; ++jj) {
          const uint32_t st = kv_count % NSTAGE, n = kv_count / NSTAGE;
          const int key0 = it.lo + jj * BN;
          if (n >= 1 && !mbar_wait(&sm.k_empty[st], (n - 1) & 1, wc, hdr)) { ok = false; break; }
          mbar_arrive_expect_tx(&sm.k_full[st], kLoadBytes);
#pragma unroll
          for (int cb = 0; cb < kBlocks; ++cb)
            tma_load_2d(sm.k[st] + cb * kBlk, &tm_k, &sm.k_full[st], it.g * D + cb * 64, key0);
          if (n >= 1 && !mbar_wait(&sm.v_empty[st], (n - 1) & 1, wc, hdr)) {
            drain_wait(&sm.k_full[st], n & 1);      // the K copy just issued is in flight
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&sm.v_full[st], kLoadBytes);
#pragma unroll
          for (int cb = 0; cb < kBlocks; ++cb)
            tma_load_2d(sm.v[st] + cb * kBlk, &tm_v, &sm.v_full[st], it.g * D + cb * 64, key0);
          ++kv_count;
        }
      }
      // leaving, normally or on an abort: every issued copy lands first
      for (uint32_t j = it_count > 2 ? it_count - 2 : 0; j < it_count; ++j)
        drain_wait(&sm.q_full[j & 1], (j >> 1) & 1);
      for (uint32_t j = kv_count > NSTAGE ? kv_count - NSTAGE : 0; j < kv_count; ++j) {
        drain_wait(&sm.k_full[j % NSTAGE], (j / NSTAGE) & 1);
        drain_wait(&sm.v_full[j % NSTAGE], (j / NSTAGE) & 1);
      }
    } else if (warp == kWarpMma && lane == 0) {
      // ------------------------------------------------------------ MMA issuer
      uint32_t it_count = 0, kv_count = 0, p_count = 0;
      while (true) {
        const uint32_t slot = it_count & 1, use = it_count >> 1;
        if (!wait_one(&sm.item_full[slot], use & 1, wc, hdr)) break;
        const QueryItem it = sm.items[slot];
        mbar_arrive(&sm.item_empty[slot]);
        if (it.n_kv < 0) break;
        if (!wait_one(&sm.q_full[slot], use & 1, wc, hdr)) break;
        const uint32_t qs = smem_u32(sm.q[slot]);
        bool ok = true;
        {
          const uint32_t st = kv_count % NSTAGE, n = kv_count / NSTAGE;
          if (!wait_one(&sm.k_full[st], n & 1, wc, hdr)) break;
          tc_fence_after();
          const uint32_t ks = smem_u32(sm.k[st]);
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            mma_kk<D / 2>(m, tmem + col_s(m), qs, ks);              // S_m = Q_m K_m^T
            mma_commit(&sm.s_full[m]);
          }
          mma_commit(&sm.k_empty[st]);
        }
        for (int jj = 0; jj < it.n_kv && ok; ++jj) {
          const uint32_t st = (kv_count + jj) % NSTAGE, n = (kv_count + jj) / NSTAGE;
          const bool has_next = jj + 1 < it.n_kv;
          const uint32_t stn = (kv_count + jj + 1) % NSTAGE, nn = (kv_count + jj + 1) / NSTAGE;
          if (!wait_one(&sm.v_full[st], n & 1, wc, hdr)) { ok = false; break; }
          // the first product overwrites O: read by the previous item's epilogue
          if (jj == 0 && it_count >= 1 && !wait_one(&sm.o_free, (it_count - 1) & 1, wc, hdr)) {
            ok = false;
            break;
          }
          const uint32_t vs = smem_u32(sm.v[st]);
#pragma unroll
          for (int m = 0; m < 2; ++m) {
            if (!ok) continue;
            if (!wait_one(&sm.p_full[m], p_count & 1, wc, hdr)) { ok = false; continue; }
            tc_fence_after();
            mma_ts_mn<128, D>(tmem + col_o(m), tmem + col_s(m), vs, 0, jj > 0);   // O_m += P_m V
            if (m == 1) mma_commit(&sm.v_empty[st]);
            if (!has_next) {
              if (m == 1) mma_commit(&sm.o_full);
              continue;
            }
            if (m == 0) {
              if (!wait_one(&sm.k_full[stn], nn & 1, wc, hdr)) { ok = false; continue; }
              tc_fence_after();
            }
            mma_kk<D / 2>(m, tmem + col_s(m), qs, smem_u32(sm.k[stn]));
            mma_commit(&sm.s_full[m]);
            if (m == 1) mma_commit(&sm.k_empty[stn]);
          }
          ++p_count;
        }
        if (!ok) break;
        kv_count += it.n_kv;
        ++it_count;
      }
      mma_drain(&sm.mma_drain_bar);        // every product done before TMEM is freed
    } else if (warp == kWarpStore && lane == 0) {
      // ------------------------------------------------------------ store of finished tiles
      uint32_t it_count = 0;
      while (true) {
        const uint32_t slot = it_count & 1;
        if (!mbar_wait(&sm.item_full[slot], (it_count >> 1) & 1, wc, hdr)) break;
        const QueryItem it = sm.items[slot];
        mbar_arrive(&sm.item_empty[slot]);
        if (it.n_kv < 0) break;
        if (!mbar_wait(&sm.out_full, it_count & 1, wc, hdr)) break;
#pragma unroll
        for (int cb = 0; cb < kBlocks; ++cb) {
          tma_store_3d(&tm_out, sm.out + cb * kBlk, cb * 64, it.h0, it.t0);
          if constexpr (SAVE)
            tma_store_3d(&tm_out2, sm.q[slot] + cb * kBlk, cb * 64, it.h0, it.t0);
        }
        bulk_commit();
        bulk_wait_read_all();
        mbar_arrive(&sm.out_free);
        // (freed by the last product of scores instead, a long document takes 940 us, not 912)
        mbar_arrive(&sm.q_empty[slot]);
        ++it_count;
      }
      bulk_wait_all();                     // every tile is in memory before the CTA exits
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kRegsSoftmax));
    // ------------------------------------------------------------ softmax
    const int m_ = warp >> 2;              // map
    const int wq = warp & 3;
    const int r = wq * 32 + lane;
    const uint32_t lane_base = (uint32_t)(wq * 32) << 16;
    const uint32_t s_tm = tmem + lane_base + col_s(m_);
    const uint32_t o_tm = tmem + lane_base + col_o(m_);
    const float sl2 = p.scale * kLog2e;
    const uint64_t sl2x2 = f2_pack(sl2, sl2);
    uint32_t it_count = 0, s_count = 0;
    // An item's rows are found (a search of some 1400 cycles) while the item before
    // it waits for its last product.
    QueryItem it;
    Span32 doc = {0, 0};
    auto next_item = [&](uint32_t n) {
      if (!wait_warp(&sm.item_full[n & 1], (n >> 1) & 1, wc, hdr)) return false;
      it = sm.items[n & 1];
      mbar_arrive_warp(&sm.item_empty[n & 1], lane);
      if (it.n_kv >= 0)
        doc = document_of_rows(p.cu, p.ndoc, (int64_t)it.t0 + ((wq * 32) >> a.shift), p.q_len, lane, a.shift);
      return true;
    };
    if (!next_item(0)) it.n_kv = -1;
    while (it.n_kv >= 0) {
      const uint32_t slot = it_count & 1;
      const int h = it.h0 + (r & ((1 << a.shift) - 1));
      const int64_t row = (int64_t)it.t0 + (r >> a.shift);
      const bool valid = row < p.q_len;
      int lo = 0, hi = 0;                                      // visible keys [lo, hi)
      float lam = 0.f;
      if (valid) {
        lo = doc.first;
        hi = p.causal ? (int)row + 1 : (int)min((int64_t)doc.last, p.kv_len);
        lam = __bfloat162float(a.lambda[(int64_t)h * a.n_lambda + (a.n_lambda > 1 ? row : 0)]);
      }
      float m = -INFINITY, l = 0.f;
      bool ok = true;
      for (int jj = 0; jj < it.n_kv; ++jj) {
        if (!wait_warp(&sm.s_full[m_], s_count & 1, wc, hdr)) { ok = false; break; }
        ++s_count;
        tc_fence_after();
        const int key0 = it.lo + jj * BN;
        uint32_t sr[4][32];
#pragma unroll
        for (int c = 0; c < 4; ++c) tmem_ld32(s_tm + c * 32, sr[c]);
        tmem_wait_ld();
        // a warp whose rows all see the whole tile skips the masks (skipping single
        // chunks that nothing sees instead costs more in branches than it saves)
        if (!__all_sync(0xffffffffu, lo <= key0 && key0 + BN <= hi)) {
#pragma unroll
          for (int c = 0; c < 4; ++c)
            mask32(sr[c], column_bits(lo - key0 - 32 * c, hi - key0 - 32 * c));
        }
        float mx[4];
#pragma unroll
        for (int c = 0; c < 4; ++c) mx[c] = max32(sr[c]);
        const float m_new = fmaxf(m, fmaxf(fmaxf(mx[0], mx[1]), fmaxf(mx[2], mx[3])) * sl2);
        // the running output is rescaled only when the maximum grew a lot
        const bool need = (m != -INFINITY) && (m_new > m + kRescaleThreshold);
        const float corr = need ? ex2(m - m_new) : 1.f;
        if (need || m == -INFINITY) m = m_new;
        const float mb = (m == -INFINITY) ? 0.f : m;
        const uint64_t nm2 = f2_pack(-mb, -mb);
        uint64_t ls[4] = {0, 0, 0, 0};
#pragma unroll
        for (int c = 0; c < 4; ++c) {
          uint32_t pk[16];
          exps32(sr[c], sl2x2, nm2, ls, pk);
          tmem_st16(s_tm + c * 16, pk);
        }
        float l0, l1;
        f2_unpack(f2_add(f2_add(ls[0], ls[1]), f2_add(ls[2], ls[3])), l0, l1);
        l = l * corr + (l0 + l1);
        if (__any_sync(0xffffffffu, need)) {
#pragma unroll
          for (int c = 0; c < D / 32; ++c) {
            uint32_t orow[32];
            tmem_ld32(o_tm + c * 32, orow);
            tmem_wait_ld();
#pragma unroll
            for (int i = 0; i < 32; ++i) orow[i] = __float_as_uint(__uint_as_float(orow[i]) * corr);
            tmem_st32(o_tm + c * 32, orow);
          }
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&sm.p_full[m_]);
      }
      if (!ok) break;
      // ---- epilogue: out = O_1 / l_1 - lambda O_2 / l_2; the warpgroups swap
      // their row sums and take half of the columns of both accumulators each
      sm.inv[slot][m_][r] = l > 0.f ? 1.f / l : 0.f;
      if (valid && p.lse != nullptr)
        p.lse[((int64_t)h * 2 + m_) * p.q_len + row] = (m + __log2f(l)) * kLn2;
      mbar_arrive_warp(&sm.inv_full, lane);
      if (!next_item(it_count + 1)) break;
      if (!mbar_wait_warp(&sm.inv_full, it_count & 1, wc, hdr)) break;
      if (!mbar_wait_warp(&sm.o_full, it_count & 1, wc, hdr)) break;
      tc_fence_after();
      const float i0 = sm.inv[slot][0][r], i1 = sm.inv[slot][1][r];
      // the previous tile has left the staging buffer
      if (it_count >= 1 && !wait_warp(&sm.out_free, (it_count - 1) & 1, wc, hdr)) break;
#pragma unroll
      for (int c = 0; c < D / 64; ++c) {
        uint32_t x[32], y[32];
        tmem_ld32(tmem + lane_base + col_o(0) + m_ * (D / 2) + c * 32, x);
        tmem_ld32(tmem + lane_base + col_o(1) + m_ * (D / 2) + c * 32, y);
        tmem_wait_ld();
        if (c == D / 64 - 1) {             // both accumulators read: the next item may start
          tc_fence_before();
          mbar_arrive_warp(&sm.o_free, lane);
        }
        uint32_t w[16], w2[16];
#pragma unroll
        for (int i = 0; i < 16; ++i) {
          const float a0 = __uint_as_float(y[2 * i]) * i1, a1 = __uint_as_float(y[2 * i + 1]) * i1;
          w[i] = pack_bf16x2(fmaf(__uint_as_float(x[2 * i]), i0, -lam * a0),
                             fmaf(__uint_as_float(x[2 * i + 1]), i0, -lam * a1));
          w2[i] = pack_bf16x2(a0, a1);
        }
        // columns m D/2 + 32 c + 0..31 of the row: four 16-byte chunks of its swizzle span
        const int col = m_ * (D / 2) + c * 32;
        const uint32_t base = smem_u32(sm.out) + (col >> 6) * kBlk + r * 128;
#pragma unroll
        for (int i = 0; i < 4; ++i)
          st_shared_v4(base + (((((col & 63) >> 3) + i) ^ (r & 7)) << 4), w[4 * i], w[4 * i + 1],
                       w[4 * i + 2], w[4 * i + 3]);
        if constexpr (SAVE) {
          // (every product of the item is done: its Q tile is free until it is stored)
          const uint32_t base2 = smem_u32(sm.q[slot]) + (col >> 6) * kBlk + r * 128;
#pragma unroll
          for (int i = 0; i < 4; ++i)
            st_shared_v4(base2 + (((((col & 63) >> 3) + i) ^ (r & 7)) << 4), w2[4 * i], w2[4 * i + 1],
                         w2[4 * i + 2], w2[4 * i + 3]);
        }
      }
      fence_proxy_async_smem();
      mbar_arrive_warp(&sm.out_full, lane);
      ++it_count;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

template <int D, bool SAVE>
cudaError_t launch_fwd(const CUtensorMap& mq, const CUtensorMap& mk, const CUtensorMap& mv,
                       const CUtensorMap& mo, const CUtensorMap& mo2, const FwdArgs& a,
                       cudaStream_t s) {
  return launch_persistent<2 * D + SAVE>(diff_fwd_tc_kernel<D, SAVE>, kThreads, smem_bytes<Smem>(), s,
                                         mq, mk, mv, mo, mo2, a);
}

}  // namespace

static bool encode_map(CUtensorMap* m, const void* base, int rank, const cuuint64_t* dims,
                const cuuint64_t* strides, const cuuint32_t* box) {
  static const PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) != cudaSuccess || q != cudaDriverEntryPointSuccess)
      ptr = nullptr;
    return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }();
  const cuuint32_t estr[3] = {1, 1, 1};
  return fn && fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, rank, const_cast<void*>(base), dims, strides, box,
                  estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
                  CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// [T, H, d] bf16, box = 64 columns x `heads` heads x 128 / heads tokens, 128-byte swizzle:
// row r of the tile is token r / heads, head r % heads.
bool diff_heads_map(CUtensorMap* m, const void* base, int64_t T, int64_t H, int64_t d, int heads) {
  const cuuint64_t dims[3] = {(cuuint64_t)d, (cuuint64_t)H, (cuuint64_t)T};
  const cuuint64_t strides[2] = {(cuuint64_t)(d * 2), (cuuint64_t)(H * d * 2)};
  const cuuint32_t box[3] = {64, (cuuint32_t)heads, (cuuint32_t)(BM / heads)};
  return encode_map(m, base, 3, dims, strides, box);
}

// [rows, cols] bf16 row-major, box = 64 columns x 128 rows, 128-byte swizzle.
bool diff_tile_map(CUtensorMap* m, const void* base, int64_t rows, int64_t cols) {
  const cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  const cuuint64_t strides[1] = {(cuuint64_t)(cols * 2)};
  const cuuint32_t box[2] = {64, 128};
  return encode_map(m, base, 2, dims, strides, box);
}

cudaError_t launch_diff_fwd_tc(const DiffProblem& d, const FwdWsLayout& L, char* ws, cudaStream_t s) {
  const AttnProblem& p = d.p;
  CUtensorMap mq, mk, mv, mo, mo2;
  const int shift = d.shift;
  if (!diff_heads_map(&mq, p.q, p.q_len, p.Hq, p.d, 1 << shift) ||
      !diff_tile_map(&mk, p.k, p.kv_len, (int64_t)p.Hkv * p.d) ||
      !diff_tile_map(&mv, p.v, p.kv_len, (int64_t)p.Hkv * p.d) ||
      !diff_heads_map(&mo, p.out, p.q_len, p.Hq, p.d, 1 << shift) ||
      !diff_heads_map(&mo2, d.out2 ? d.out2 : p.out, p.q_len, p.Hq, p.d, 1 << shift))
    return cudaErrorNotSupported;
  FwdArgs a;
  a.p = p;
  a.lambda = reinterpret_cast<const __nv_bfloat16*>(d.lambda);
  a.n_lambda = d.n_lambda;
  a.order = reinterpret_cast<const int*>(ws + L.order);
  a.shift = shift;
  if (d.out2 != nullptr)
    return p.d == 128 ? launch_fwd<128, true>(mq, mk, mv, mo, mo2, a, s)
                      : launch_fwd<64, true>(mq, mk, mv, mo, mo2, a, s);
  return p.d == 128 ? launch_fwd<128, false>(mq, mk, mv, mo, mo2, a, s)
                    : launch_fwd<64, false>(mq, mk, mv, mo, mo2, a, s);
}

}  // namespace nsp
