// Differential attention backward on the tcgen05 tensor cores: bf16 inputs,
// float32 scores and accumulation, head dimension D = 128 or 64 (two maps of
// D / 2 columns), two persistent kernels without atomics.
//
// With P_m recomputed from the forward's lse, delta_m = <dout, O_m>, c = -lambda
// (per query row; delta, -lse log2 e and c are prepared by diff_prep_kernel in
// padded rows):
//   dP = dOut V^T (one product for both maps),
//   dS_1 = P_1 (dP - delta_1),  dS_2 = c P_2 (dP - delta_2),
//   dV = (P_1 + c P_2)^T dOut,  dK_m = scale dS_m^T Q_m,  dQ_m = scale dS_m K_m.
//
// dK/dV kernel (key-stationary).  Work item: one 128-key tile of one KV head;
// it walks every pair (2^shift query heads of the group, tile of 128 >> shift
// tokens of them that can see the keys).  With few key tiles an item is some of a tile's
// pairs, and the join kernel sums the parts' float32 shares in order (key_parts).  A pair
// costs four 128 x 128 x 128 products' worth: S_1 and S_2 (half the columns each), dP,
// dV (both maps in one product, their combination is its operand), dK_1 and dK_2 (half the columns each); treating
// the maps as two heads would cost six.  TMEM: two 128-column regions [0,256),
// dV [256,256+D), dK_1 | dK_2 [384,384+D).  Pair n puts S_1^T in region A = n & 1,
// dP^T in the other one, B; S_2^T follows into A when the softmax warps have
// read S_1.  dS_1^T (bf16) goes to shared memory; P^T = (P_1 + c P_2)^T and dS_2^T
// (bf16) over S_2, 16 columns each of every 32: both are operands read from
// TMEM, which spares shared memory's bandwidth (the operands of S, dP and dK_1, the
// tiles' copies and dS_1 take about 2900 cycles of it a pair).  The next pair swaps
// the regions, so its S_1 is computed into B, while the softmax is on this pair's
// second map.  A pair's 40 instructions take the tensor core 2560 cycles at least
// (64 for 128 columns, 62 for the 64 of a dK_m); it measures some 5200: dS_1 waits for
// S_1 and dP, dK_2 and dV for both, and the two regions hold no third pair.  393 us for
// 16384 tokens in 19 causal documents, 16 heads on 4, d = 128 (555 TFLOP/s of the
// visible pairs' 8 d).
//
// dQ kernel (query-stationary).  Work item: 128 query rows, several heads of a group
// at fewer tokens (QueryItem).
// TMEM: S_1 [0,128), S_2 [128,256), dP [256,384), dQ_1 | dQ_2 [384,384+D).  dS_m
// (bf16) goes over S_m and is read from TMEM.  The softmax keeps dP of a tile
// in registers for both maps; while it is on one map the tensor core does the
// other map's dQ, the next S, and the next dP.  The issuing thread always has a
// product to issue: 32 instructions of a tile take 3500 cycles, 110 each, against
// 68 to 76 of independent ones back to back (dP of the next tile between dQ_1's or
// dQ_2's, instruction by instruction or half by half, is 2 to 4 % slower: 600 us
// for both kernels against 581, with 128-token tiles of one head).
// The gradient of lambda comes from here too, -sum_j P_2 dP of each row, from the
// float32 values before any of them is rounded: its terms cancel over the tokens, and
// <dout, out2> with the saved bf16 out2 is off by 1 % and more where they do.  236 us for
// the same documents (693 TFLOP/s of their 6 d), 213 without that sum: its 32 packed
// instructions a warp and tile, 128 with a mask, stand in the issue slots of the softmax
// (behind the arrival that the products wait for they cost the same, or registers: 834 us
// of the step against 761).
//
// Roles, dK/dV: 16 softmax warps (four column groups of four lane quadrants;
// with 8 warps of 64 columns the loop is 18 KB of instructions and waits for
// them), warp 16 producer of tiles, warps 17 and 18 one MMA stream each (S and dP;
// dK and dV: products of one thread run in order, so those that wait for the
// softmax must not hold up the others), warp 19 producer of the row vectors.
// dQ: 8 softmax warps, warp 8 producer, warp 9 MMA.  All waits are bounded.
//
// Rounding: P_1 + c P_2 and dS_m are rounded to bf16, as the tensor core's operands
// next to bf16 inputs; delta_m are float32 sums over the bf16 out and out2 of the
// forward; scores, exponentials, sums and shares are float32.
// Against exact arithmetic dQ and dK are off by 0.0025 (relative norm) and dV by 0.0024,
// where outputs rounded to bf16 alone leave 0.0017; dlambda by its rounding.
#include "diff_tc.cuh"

namespace nsp {
namespace {

using namespace tc;

struct BwdArgs {
  AttnProblem p;
  const float *nlse2, *ndelta;      // [Hq / P][2][Tp][P], P = 2^shift
  const float *coef, *cndelta;      // [Hq / P][Tp][P]: c, -c delta_2
  int64_t Tp;
  __nv_bfloat16 *dq, *dk, *dv;
  float* dlam_rows;                 // ndelta's second map: -sum_j P_2 dP of each row, or
  __nv_bfloat16* dlam;              // (one lambda a token) written as its gradient [Hq][T]
  float* parts;                     // n_parts > 1: [part][dV, dK][T, Hkv, d] of the key tiles' parts
  int n_parts;
  const int* qorder;                // 128-token tiles of queries, most keys first
  int shift;                        // log2 of the heads of a query item
  const int* korder;
};

// ================================================================ dK / dV

constexpr int kKvThreads = 640;
constexpr int kKvSoftmaxWarps = 16;
constexpr int kKvWarpTiles = 16, kKvWarpMma1 = 17, kKvWarpMma2 = 18, kKvWarpRows = 19;
constexpr int kKvRegsControl = 64, kKvRegsSoftmax = 104;   // 128 x 64 + 512 x 104 = 640 x 96

struct KvItem {
  // n_q query tiles (128 >> shift tokens of 2^shift heads) from row q_lo = token << shift on;
  // pairs n0 .. n0 + pairs - 1 of the key tile's (head group, query tile) are this item's; -1 stops
  int ktile, g, q_lo, n_q, n0, pairs, part, whole;
};

// The query rows that a key tile sees, and its pairs.
__device__ __forceinline__ int key_tile_pairs(const AttnProblem& p, int ktile, int shift, int& q_lo, int& n_q) {
  const int key0 = ktile * 128;
  const int64_t last = min((int64_t)key0 + 128, p.kv_len) - 1;
  const int first = p.causal ? key0 : __ldg(p.cu + doc_of(p.cu, p.ndoc, key0));
  // (the stream may end inside a document: no row vectors are past its rows)
  const int end = (int)min((int64_t)__ldg(p.cu + doc_of(p.cu, p.ndoc, last) + 1), p.q_len);
  // (a multiple of a tile's tokens: the row vectors are read in whole tiles)
  q_lo = (first << shift) & ~127;
  n_q = ((end << shift) - q_lo + 127) >> 7;
  return (p.Hq / p.Hkv >> shift) * n_q;
}

// Parts of a key tile of so many pairs, four at least in each: a tile of few pairs is written
// whole (2000 tokens in short documents, 64 key tiles: 76 us; split in 8 parts each, 97; one
// document of 2000: 103 us, with 16 pairs at least 133).
constexpr int kPartPairs = 4;
__device__ __forceinline__ int parts_of(const BwdArgs& a, int pairs) {
  return min(a.n_parts, max(1, pairs / kPartPairs));
}

struct __align__(1024) SmemKV {
  uint8_t k[kTile];
  uint8_t v[kTile];
  // Q of pair j in slot j % 4, dOut in slot (j + 2) % 4, the (j / 2)-th fill
  // of their slots: Q of pair j + 2 takes the slot that dOut of pair j frees
  uint8_t qd[4][kTile];
  uint8_t ds[kTile];                         // dS_1^T, [q-block][key][64 q], 128-byte swizzle
  float first[2][128];                       // map 1: -lse log2 e, -delta
  float second[3][128];                      // map 2: -lse log2 e, -c delta, c
  uint64_t kv_full, kv_empty;
  uint64_t slot_full[4], slot_empty[4];
  uint64_t first_full, second_full;
  uint64_t s1_full, s1_free, s2_full, dp_full, dp_free, ds_ready, p_ready, p_done;
  uint64_t dkv_full, dkv_empty;
  uint64_t item_full[2], item_empty[2];
  KvItem items[2];
  uint64_t drain1, drain2;
  uint32_t tmem_base;
  WaitCtl wait;
};
static_assert(sizeof(SmemKV) <= kSmemLimit, "dK/dV tile set exceeds shared memory");

// Clears the masked pairs of a 16-lane fragment: rows e = 0 and 1 (pairs 2 j + e)
// keep columns [lo_e, hi_e).
__device__ __forceinline__ void mask_rows(uint32_t (&w)[8], int lo0, int hi0, int lo1, int hi1, int tc2) {
  uint32_t mask[4];
  pair_masks(column_bits(lo0, hi0) >> tc2, mask);
#pragma unroll
  for (int j = 0; j < 4; ++j) w[2 * j] &= mask[j];
  pair_masks(column_bits(lo1, hi1) >> tc2, mask);
#pragma unroll
  for (int j = 0; j < 4; ++j) w[2 * j + 1] &= mask[j];
}

template <int D>
__global__ void __launch_bounds__(kKvThreads, 1)
    diff_bwd_dkdv_tc_kernel(const __grid_constant__ CUtensorMap tm_q,
                            const __grid_constant__ CUtensorMap tm_do,
                            const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v,
                            const __grid_constant__ BwdArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const AttnProblem& p = a.p;
  WsHeader* hdr = p.hdr;
  grid_dep_wait();                          // the prepared row vectors
  grid_dep_trigger();                       // the dQ kernel may launch on SMs this one frees
  if (block_leaves(status_bad(hdr))) return;
  SmemKV* smp = smem_view<SmemKV>(smem_raw, hdr);
  if (smp == nullptr) return;
  SmemKV& sm = *smp;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    mbar_init(&sm.kv_full, 1);
    mbar_init(&sm.kv_empty, 1);
    for (int s = 0; s < 4; ++s) {
      mbar_init(&sm.slot_full[s], 1);
      mbar_init(&sm.slot_empty[s], 2);       // one commit of each stream
    }
    mbar_init(&sm.first_full, 1);
    mbar_init(&sm.second_full, 1);
    mbar_init(&sm.s1_full, 1);
    mbar_init(&sm.s1_free, kKvSoftmaxWarps);
    mbar_init(&sm.s2_full, 1);
    mbar_init(&sm.dp_full, 1);
    mbar_init(&sm.dp_free, kKvSoftmaxWarps);
    mbar_init(&sm.p_ready, kKvSoftmaxWarps);
    mbar_init(&sm.ds_ready, kKvSoftmaxWarps);
    mbar_init(&sm.p_done, 1);
    mbar_init(&sm.dkv_full, 1);
    mbar_init(&sm.dkv_empty, kKvSoftmaxWarps);
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.item_full[s], 1);
      mbar_init(&sm.item_empty[s], 3 + kKvSoftmaxWarps);
    }
    mbar_init(&sm.drain1, 1);
    mbar_init(&sm.drain2, 1);
    wait_ctl_init(&sm.wait, p.wait_budget);
    fence_mbar_init();
  }
  if (warp == kKvWarpMma1) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  if (warp == kKvWarpTiles && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_do);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  const uint32_t tmem = sm.tmem_base;
  WaitCtl* const wc = &sm.wait;
  const int G = p.Hq / p.Hkv;
  const int n_items = hdr->n_items2 * p.Hkv * a.n_parts;
  constexpr int kBlocks = D / 64;                        // 64-column blocks of a row
  constexpr uint32_t kLoad = kBlocks * kBlk;             // one Q, dOut, K or V tile

  if (warp >= kKvSoftmaxWarps) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kKvRegsControl));
    if (warp == kKvWarpTiles && lane == 0) {
      // ------------------------------------------------------------ producer: items, tiles
      uint32_t it_count = 0, kv_count = 0, qc = 0, loads = 0;
      bool ok = true;
      while (ok) {
        const int idx = atomicAdd(&hdr->counter2, 1);
        KvItem it = {};
        it.pairs = -1;
        if (idx < n_items) {
          const int rest = idx % (p.Hkv * a.n_parts);
          it.ktile = a.korder[idx / (p.Hkv * a.n_parts)];
          it.g = rest % p.Hkv;
          it.part = rest / p.Hkv;
          const int all = key_tile_pairs(p, it.ktile, a.shift, it.q_lo, it.n_q);
          const int parts = parts_of(a, all);
          if (it.part >= parts) continue;
          it.whole = parts == 1;
          it.n0 = (int)((int64_t)all * it.part / parts);
          it.pairs = (int)((int64_t)all * (it.part + 1) / parts) - it.n0;
        }
        const uint32_t slot = it_count & 1;
        if (it_count >= 2 && !mbar_wait(&sm.item_empty[slot], ((it_count >> 1) - 1) & 1, wc, hdr))
          break;
        sm.items[slot] = it;
        mbar_arrive(&sm.item_full[slot]);
        ++it_count;
        if (it.pairs < 0) break;
        if (kv_count >= 1 && !mbar_wait(&sm.kv_empty, (kv_count - 1) & 1, wc, hdr)) break;
        mbar_arrive_expect_tx(&sm.kv_full, 2 * kLoad);
#pragma unroll
        for (int cb = 0; cb < kBlocks; ++cb) {
          tma_load_2d(sm.k + cb * kBlk, &tm_k, &sm.kv_full, it.g * D + cb * 64, it.ktile * 128);
          tma_load_2d(sm.v + cb * kBlk, &tm_v, &sm.kv_full, it.g * D + cb * 64, it.ktile * 128);
        }
        ++kv_count;
        int h = it.g * G + ((it.n0 / it.n_q) << a.shift), i = it.n0 % it.n_q;
        for (int n = 0; n < it.pairs && ok; ++n) {
          const uint32_t fill = qc >> 1;
#pragma unroll
          for (int t = 0; t < 2; ++t) {                  // Q, then dOut
            const uint32_t s = (qc + 2 * t) & 3;
            if (!ok) continue;
            if (fill >= 1 && !mbar_wait(&sm.slot_empty[s], (fill - 1) & 1, wc, hdr)) {
              ok = false;
              continue;
            }
            mbar_arrive_expect_tx(&sm.slot_full[s], kLoad);
#pragma unroll
            for (int cb = 0; cb < kBlocks; ++cb)
              tma_load_3d(sm.qd[s] + cb * kBlk, t == 0 ? &tm_q : &tm_do, &sm.slot_full[s], cb * 64, h,
                          (it.q_lo + i * 128) >> a.shift);
            ++loads;
          }
          ++qc;
          if (++i == it.n_q) { i = 0; h += 1 << a.shift; }
        }
      }
      // leaving, normally or on an abort: every issued copy lands first
      if (kv_count >= 1) drain_wait(&sm.kv_full, (kv_count - 1) & 1);
      for (uint32_t l = (loads > 4 ? loads - 4 : 0); l < loads; ++l) {
        const uint32_t j = l >> 1;                        // load l: pair l / 2, Q or dOut
        drain_wait(&sm.slot_full[(l & 1) ? ((j + 2) & 3) : (j & 3)], (j >> 1) & 1);
      }
    } else if (warp == kKvWarpRows && lane == 0) {
      // ------------------------------------------------------------ producer: row vectors
      // One buffer for each map: the first map's is free in the middle of a pair
      // (all of dS_1 written) and wanted at the start of the next one, the
      // second's the other way round.
      uint32_t it_count = 0, n1 = 0, n2 = 0;
      bool ok = true;
      while (ok) {
        const uint32_t slot = it_count & 1;
        if (!mbar_wait(&sm.item_full[slot], (it_count >> 1) & 1, wc, hdr)) break;
        const KvItem it = sm.items[slot];
        mbar_arrive(&sm.item_empty[slot]);
        ++it_count;
        if (it.pairs < 0) break;
        int h = it.g * G + ((it.n0 / it.n_q) << a.shift), i = it.n0 % it.n_q;
        for (int n = 0; n < it.pairs; ++n) {
          const int64_t hg = h >> a.shift, np = a.Tp << a.shift, q0 = it.q_lo + (int64_t)i * 128;
          const int64_t r1 = 2 * hg * np + q0, r2 = r1 + np;
          if (n1 >= 1 && !mbar_wait(&sm.ds_ready, (n1 - 1) & 1, wc, hdr)) { ok = false; break; }
          mbar_arrive_expect_tx(&sm.first_full, 2 * 512);
          bulk_load(sm.first[0], a.nlse2 + r1, 512, &sm.first_full);
          bulk_load(sm.first[1], a.ndelta + r1, 512, &sm.first_full);
          ++n1;
          if (n2 >= 1 && !mbar_wait(&sm.p_ready, (n2 - 1) & 1, wc, hdr)) { ok = false; break; }
          mbar_arrive_expect_tx(&sm.second_full, 3 * 512);
          bulk_load(sm.second[0], a.nlse2 + r2, 512, &sm.second_full);
          const int64_t rc = hg * np + q0;
          bulk_load(sm.second[1], a.cndelta + rc, 512, &sm.second_full);
          bulk_load(sm.second[2], a.coef + rc, 512, &sm.second_full);
          ++n2;
          if (++i == it.n_q) { i = 0; h += 1 << a.shift; }
        }
      }
      if (n1 >= 1) drain_wait(&sm.first_full, (n1 - 1) & 1);
      if (n2 >= 1) drain_wait(&sm.second_full, (n2 - 1) & 1);
    } else if (warp == kKvWarpMma1 && lane == 0) {
      // ------------------------------------------------------------ stream 1: S_1, dP, S_2
      const uint32_t k_s = smem_u32(sm.k), v_s = smem_u32(sm.v);
      uint32_t it_count = 0, items_done = 0, qc = 0;
      bool ok = true;
      while (ok) {
        const uint32_t slot = it_count & 1;
        if (!wait_one(&sm.item_full[slot], (it_count >> 1) & 1, wc, hdr)) break;
        const KvItem it = sm.items[slot];
        mbar_arrive(&sm.item_empty[slot]);
        ++it_count;
        if (it.pairs < 0) break;
        if (!wait_one(&sm.kv_full, items_done & 1, wc, hdr)) break;
        for (int n = 0; n < it.pairs; ++n) {
          const uint32_t sq = qc & 3, sd = (qc + 2) & 3, fp = (qc >> 1) & 1, rb = qc & 1;
          const uint32_t ra = tmem + 128 * rb, rbb = tmem + 128 * (rb ^ 1);
          if (!wait_one(&sm.slot_full[sq], fp, wc, hdr)) { ok = false; break; }
          // A held the previous pair's dP: free once the softmax has read it twice
          if (qc >= 1 && !wait_one(&sm.dp_free, (qc - 1) & 1, wc, hdr)) { ok = false; break; }
          tc_fence_after();
          mma_kk<D / 2>(0, ra, k_s, smem_u32(sm.qd[sq]));                 // S_1^T = K_1 Q_1^T
          mma_commit(&sm.s1_full);
          if (!wait_one(&sm.slot_full[sd], fp, wc, hdr)) { ok = false; break; }
          // B held the previous pair's P and dS_2: free once dV and dK_2 have read them
          if (qc >= 1 && !wait_one(&sm.p_done, (qc - 1) & 1, wc, hdr)) { ok = false; break; }
          tc_fence_after();
          mma_kk<D>(0, rbb, v_s, smem_u32(sm.qd[sd]));                    // dP^T = V dOut^T
          mma_commit(&sm.dp_full);
          mma_commit(&sm.slot_empty[sd]);
          if (!wait_one(&sm.s1_free, qc & 1, wc, hdr)) { ok = false; break; }
          tc_fence_after();
          mma_kk<D / 2>(1, ra, k_s, smem_u32(sm.qd[sq]));                 // S_2^T = K_2 Q_2^T
          mma_commit(&sm.s2_full);
          mma_commit(&sm.slot_empty[sq]);
          ++qc;
        }
        if (!ok) break;
        mma_commit(&sm.kv_empty);
        ++items_done;
      }
      mma_drain(&sm.drain1);              // every product done before TMEM is freed
    } else if (warp == kKvWarpMma2 && lane == 0) {
      // ------------------------------------------------------------ stream 2: dK_1, dV, dK_2
      const uint32_t ds_s = smem_u32(sm.ds);
      uint32_t it_count = 0, items_done = 0, qc = 0;
      bool ok = true;
      while (ok) {
        const uint32_t slot = it_count & 1;
        if (!wait_one(&sm.item_full[slot], (it_count >> 1) & 1, wc, hdr)) break;
        const KvItem it = sm.items[slot];
        mbar_arrive(&sm.item_empty[slot]);
        ++it_count;
        if (it.pairs < 0) break;
        for (int n = 0; n < it.pairs; ++n) {
          const uint32_t sq = qc & 3, sd = (qc + 2) & 3, fp = (qc >> 1) & 1, rb = qc & 1;
          const uint32_t q_s = smem_u32(sm.qd[sq]);
          if (!wait_one(&sm.slot_full[sq], fp, wc, hdr)) { ok = false; break; }
          if (!wait_one(&sm.ds_ready, qc & 1, wc, hdr)) { ok = false; break; }
          // the accumulators hold the previous item until its epilogue has read them
          if (n == 0 && items_done > 0 &&
              !wait_one(&sm.dkv_empty, (items_done - 1) & 1, wc, hdr)) {
            ok = false;
            break;
          }
          tc_fence_after();
          mma_ss_mn<D / 2>(tmem + 384, ds_s, q_s, 0, n > 0);              // dK_1 += dS_1^T Q_1
          if (!wait_one(&sm.slot_full[sd], fp, wc, hdr)) { ok = false; break; }
          if (!wait_one(&sm.p_ready, qc & 1, wc, hdr)) { ok = false; break; }
          tc_fence_after();
          const uint32_t a_tm = tmem + 128 * rb;
          mma_ts_mn<32, D>(tmem + 256, a_tm, smem_u32(sm.qd[sd]), 0, n > 0);       // dV += P^T dOut
          mma_commit(&sm.slot_empty[sd]);
          mma_ts_mn<32, D / 2>(tmem + 384 + D / 2, a_tm + 16, q_s, D / 2, n > 0);  // dK_2 += dS_2^T Q_2
          mma_commit(&sm.p_done);
          mma_commit(&sm.slot_empty[sq]);
          ++qc;
        }
        if (!ok) break;
        mma_commit(&sm.dkv_full);
        ++items_done;
      }
      mma_drain(&sm.drain2);
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kKvRegsSoftmax));
    // ------------------------------------------------------------ softmax + dK/dV epilogue
    // Warp (cg, wq) covers TMEM lane quadrant wq (32 keys) and query columns
    // 32 cg .. 32 cg + 31, as 16-lane fragments: thread t holds key rows wq 32 +
    // t/4 + 8 i (i = 0..3) at columns 8 j + 2 (t % 4) + {0, 1} (j = 0..3).
    // Register pair k = 8 h + 2 j + e is row i = 2 h + e, columns of j.
    const int cg = warp >> 2, wq = warp & 3;
    const int r = wq * 32 + lane;                          // epilogue: TMEM lane = key row
    const int tr = lane >> 2, tc2 = 2 * (lane & 3);
    const uint32_t lane_base = (uint32_t)(wq * 32) << 16;
    const float sl2 = p.scale * kLog2e;
    const uint64_t sl2x2 = f2_pack(sl2, sl2);
    // dS^T tile: query block cg / 2, 16-byte chunks 4 (cg & 1) + j, swizzled
    // by key & 7 (= tr for every fragment row)
    const uint32_t ds_base = smem_u32(sm.ds) + (cg >> 1) * kBlk + (wq * 32 + tr) * 128 +
                             ((((cg & 1) * 4) ^ tr) << 4) + 2 * tc2;
    const float* const vec1 = sm.first[0] + cg * 32 + tc2;
    const float* const vec2 = sm.second[0] + cg * 32 + tc2;
    uint32_t it_count = 0, items_done = 0, qc = 0;
    bool ok = true;
    while (ok) {
      const uint32_t slot = it_count & 1;
      if (!mbar_wait_warp(&sm.item_full[slot], (it_count >> 1) & 1, wc, hdr)) break;
      const KvItem it = sm.items[slot];
      mbar_arrive_warp(&sm.item_empty[slot], lane);
      ++it_count;
      if (it.pairs < 0) break;
      int qlo[4], qhi[4];                                  // query rows that see fragment row i
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t key = (int64_t)it.ktile * 128 + wq * 32 + tr + 8 * i;
        qlo[i] = qhi[i] = 0;
        if (key < p.kv_len) {
          const int b = doc_of(p.cu, p.ndoc, key);
          qlo[i] = (p.causal ? (int)key : __ldg(p.cu + b)) << a.shift;
          qhi[i] = (int)min((int64_t)__ldg(p.cu + b + 1), p.q_len) << a.shift;
        }
      }
      // queries that see every row of the thread
      const int all_lo = max(max(qlo[0], qlo[1]), max(qlo[2], qlo[3]));
      const int all_hi = min(min(qhi[0], qhi[1]), min(qhi[2], qhi[3]));
      int n_in = it.n0 % it.n_q;                           // query tile of the pair, 0 .. n_q - 1
      for (int n = 0; n < it.pairs; ++n) {
        const int q0 = it.q_lo + n_in * 128 + cg * 32;
        if (++n_in == it.n_q) n_in = 0;
        const uint32_t rb = qc & 1;
        const uint32_t s_tm = tmem + lane_base + 128 * rb + cg * 32;
        const uint32_t dp_tm = tmem + lane_base + 128 * (rb ^ 1) + cg * 32;
        const bool full_w = __all_sync(0xffffffffu, all_lo <= q0 && q0 + 32 <= all_hi);
        // ---- first map: P_1 (kept for the second) and dS_1
        if (!wait_warp(&sm.first_full, qc & 1, wc, hdr)) { ok = false; break; }
        if (!wait_warp(&sm.s1_full, qc & 1, wc, hdr)) { ok = false; break; }
        tc_fence_after();
        uint64_t pp[16];
        {
          uint32_t x[32];
          tmem_ld16x256_x4(s_tm, x);
          tmem_ld16x256_x4(s_tm + (16u << 16), x + 16);
          tmem_wait_ld();
          tc_fence_before();
          mbar_arrive_warp(&sm.s1_free, lane);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint64_t nl = *reinterpret_cast<const uint64_t*>(vec1 + 8 * j);
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const int k = 8 * (i >> 1) + 2 * j + (i & 1);
              float u0, u1;
              f2_unpack(f2_fma(f2_pack(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])), sl2x2,
                               nl), u0, u1);
              pp[k] = f2_pack(ex2(u0), ex2(u1));
            }
          }
        }
        if (!wait_warp(&sm.dp_full, qc & 1, wc, hdr)) { ok = false; break; }
        tc_fence_after();
        // (dP of this pair follows dK_1 of the previous one, so dS_1's buffer is free)
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t y[16], ds[8];
          tmem_ld16x256_x4(dp_tm + ((uint32_t)(16 * h) << 16), y);
          tmem_wait_ld();
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint64_t nd = *reinterpret_cast<const uint64_t*>(vec1 + 128 + 8 * j);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int kk = 2 * j + e;
              float u0, u1;
              f2_unpack(f2_mul(pp[8 * h + kk], f2_add(f2_pack(__uint_as_float(y[2 * kk]),
                                                              __uint_as_float(y[2 * kk + 1])), nd)),
                        u0, u1);
              ds[kk] = pack_bf16x2(u0, u1);
            }
          }
          if (!full_w) mask_rows(ds, qlo[2 * h] - q0, qhi[2 * h] - q0, qlo[2 * h + 1] - q0,
                                 qhi[2 * h + 1] - q0, tc2);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk) {
            // (8 query columns per 16 bytes; j is two bits of the chunk number)
            st_shared_u32((ds_base ^ ((kk >> 1) << 4)) + (16 * h + 8 * (kk & 1)) * 128, ds[kk]);
          }
        }
        fence_proxy_async_smem();
        mbar_arrive_warp(&sm.ds_ready, lane);
        // ---- second map: P = P_1 + c P_2 and dS_2, the operands of dV and dK_2
        if (!wait_warp(&sm.second_full, qc & 1, wc, hdr)) { ok = false; break; }
        if (!wait_warp(&sm.s2_full, qc & 1, wc, hdr)) { ok = false; break; }
        tc_fence_after();
#pragma unroll
        for (int h = 0; h < 2; ++h) {
          uint32_t x[16], y[16], pk[8], ds[8];
          tmem_ld16x256_x4(s_tm + ((uint32_t)(16 * h) << 16), x);
          tmem_ld16x256_x4(dp_tm + ((uint32_t)(16 * h) << 16), y);
          tmem_wait_ld();
          if (h == 1) {
            tc_fence_before();
            mbar_arrive_warp(&sm.dp_free, lane);
          }
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const uint64_t nl = *reinterpret_cast<const uint64_t*>(vec2 + 8 * j);
            const uint64_t nd = *reinterpret_cast<const uint64_t*>(vec2 + 128 + 8 * j);
            const uint64_t cc = *reinterpret_cast<const uint64_t*>(vec2 + 256 + 8 * j);
#pragma unroll
            for (int e = 0; e < 2; ++e) {
              const int kk = 2 * j + e;
              float u0, u1;
              f2_unpack(f2_fma(f2_pack(__uint_as_float(x[2 * kk]), __uint_as_float(x[2 * kk + 1])),
                               sl2x2, nl), u0, u1);
              const uint64_t p2 = f2_pack(ex2(u0), ex2(u1));
              f2_unpack(f2_fma(p2, cc, pp[8 * h + kk]), u0, u1);
              pk[kk] = pack_bf16x2(u0, u1);
              f2_unpack(f2_mul(p2, f2_fma(f2_pack(__uint_as_float(y[2 * kk]),
                                                  __uint_as_float(y[2 * kk + 1])), cc, nd)), u0, u1);
              ds[kk] = pack_bf16x2(u0, u1);
            }
          }
          if (!full_w) {
            mask_rows(pk, qlo[2 * h] - q0, qhi[2 * h] - q0, qlo[2 * h + 1] - q0, qhi[2 * h + 1] - q0, tc2);
            mask_rows(ds, qlo[2 * h] - q0, qhi[2 * h] - q0, qlo[2 * h + 1] - q0, qhi[2 * h + 1] - q0, tc2);
          }
          // pair 2 j + e is (row 16 h + 8 e + t/4, packed column 4 j + t % 4): the
          // 16x128b register order
          tmem_st16x128_x4(s_tm + ((uint32_t)(16 * h) << 16), pk);
          tmem_st16x128_x4(s_tm + 16 + ((uint32_t)(16 * h) << 16), ds);
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive_warp(&sm.p_ready, lane);
        ++qc;
      }
      if (!ok) break;
      // item epilogue: column groups 0-1 write dV, 2-3 dK (64 columns each)
      if (!mbar_wait_warp(&sm.dkv_full, items_done & 1, wc, hdr)) break;
      tc_fence_after();
      const int c0 = (cg & 1) * 64;
      if (c0 < D) {
        const int64_t key = (int64_t)it.ktile * 128 + r;
        const bool is_dk = cg >= 2;
        const int64_t at = (key * p.Hkv + it.g) * D + c0;
        __nv_bfloat16* dst = (is_dk ? a.dk : a.dv) + at;
        float* part = a.parts + (it.part * 2 + is_dk) * (p.kv_len * p.Hkv * D) + at;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t v[32];
          tmem_ld32(tmem + lane_base + (is_dk ? 384u : 256u) + c0 + c * 32, v);
          tmem_wait_ld();
          if (key >= p.kv_len) continue;
          if (it.whole) {
            store_row32(dst + c * 32, v, is_dk ? p.scale : 1.f);
            continue;
          }
#pragma unroll
          for (int i = 0; i < 8; ++i)                      // (a workspace is 16-byte aligned)
            *reinterpret_cast<uint4*>(part + c * 32 + 4 * i) =
                make_uint4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
        }
      }
      tc_fence_before();
      mbar_arrive_warp(&sm.dkv_empty, lane);
      ++items_done;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kKvWarpMma1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
}

// ================================================================ dQ

constexpr int kQThreads = 320;
constexpr int kQWarpProducer = 8, kQWarpMma = 9;
constexpr int K_NS = 2;

struct __align__(1024) SmemQ {
  uint8_t q[2][kTile], dout[2][kTile];     // this item's and the next one's
  uint8_t k[K_NS][kTile];
  uint8_t v[kTile];
  uint64_t q_full[2], q_empty[2];
  uint64_t k_full[K_NS], k_empty[K_NS], v_full, v_empty;
  uint64_t s_full[2], p_full[2], dp_full, dp_free, o_full, o_free;
  uint64_t item_full[2], item_empty[2];
  uint64_t sum_full;
  QueryItem items[2];
  float sum[2][128];                       // [item parity][row]: sum of P_2 dP over columns 64-127 of every tile
  uint64_t drain;
  uint32_t tmem_base;
  WaitCtl wait;
};
static_assert(sizeof(SmemQ) <= kSmemLimit, "dQ tile set exceeds shared memory");

template <int D>
__global__ void __launch_bounds__(kQThreads, 1)
    diff_bwd_dq_tc_kernel(const __grid_constant__ CUtensorMap tm_q,
                          const __grid_constant__ CUtensorMap tm_do,
                          const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v,
                          const __grid_constant__ BwdArgs a) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const AttnProblem& p = a.p;
  WsHeader* hdr = p.hdr;
  // Launched behind the dK/dV kernel, which triggers only after its own wait:
  // everything this kernel reads is complete.  It starts on the SMs that kernel
  // frees and waits for it only before it exits, so that what follows in the
  // stream follows both.
  if (block_leaves(status_bad(hdr))) {
    grid_dep_wait();
    return;
  }
  SmemQ* smp = smem_view<SmemQ>(smem_raw, hdr);
  if (smp == nullptr) {
    grid_dep_wait();
    return;
  }
  SmemQ& sm = *smp;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.q_full[s], 1);
      mbar_init(&sm.q_empty[s], 1);
      mbar_init(&sm.s_full[s], 1);
      mbar_init(&sm.p_full[s], 8);
      mbar_init(&sm.item_full[s], 1);
      mbar_init(&sm.item_empty[s], 1 + 8);
    }
    for (int s = 0; s < K_NS; ++s) {
      mbar_init(&sm.k_full[s], 1);
      mbar_init(&sm.k_empty[s], 1);
    }
    mbar_init(&sm.v_full, 1);
    mbar_init(&sm.v_empty, 1);
    mbar_init(&sm.dp_full, 1);
    mbar_init(&sm.dp_free, 8);
    mbar_init(&sm.o_full, 1);
    mbar_init(&sm.o_free, 8);
    mbar_init(&sm.sum_full, 8);
    mbar_init(&sm.drain, 1);
    wait_ctl_init(&sm.wait, p.wait_budget);
    fence_mbar_init();
  }
  if (warp == kQWarpMma) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  if (warp == kQWarpProducer && lane == 0) {
    tma_prefetch_desc(&tm_q);
    tma_prefetch_desc(&tm_do);
    tma_prefetch_desc(&tm_k);
    tma_prefetch_desc(&tm_v);
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  const uint32_t tmem = sm.tmem_base;
  WaitCtl* const wc = &sm.wait;
  const int n_items = hdr->n_items * p.Hq;
  constexpr int kBlocks = D / 64;
  constexpr uint32_t kLoad = kBlocks * kBlk;

  if (warp == kQWarpProducer) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      uint32_t it_count = 0, k_count = 0, v_count = 0;
      bool ok = true;
      while (ok) {
        const int idx = atomicAdd(&hdr->counter, 1);
        QueryItem it = {};
        it.n_kv = -1;
        if (idx < n_items && !query_item(it, p, a.qorder, idx, a.shift)) continue;
        const uint32_t slot = it_count & 1, use = it_count >> 1;
        if (use >= 1 && !mbar_wait(&sm.item_empty[slot], (use - 1) & 1, wc, hdr)) break;
        sm.items[slot] = it;
        mbar_arrive(&sm.item_full[slot]);
        if (it.n_kv < 0) break;
        if (use >= 1 && !mbar_wait(&sm.q_empty[slot], (use - 1) & 1, wc, hdr)) break;
        mbar_arrive_expect_tx(&sm.q_full[slot], 2 * kLoad);
#pragma unroll
        for (int cb = 0; cb < kBlocks; ++cb) {
          tma_load_3d(sm.q[slot] + cb * kBlk, &tm_q, &sm.q_full[slot], cb * 64, it.h0, it.t0);
          tma_load_3d(sm.dout[slot] + cb * kBlk, &tm_do, &sm.q_full[slot], cb * 64, it.h0, it.t0);
        }
        ++it_count;
        for (int jj = 0; jj < it.n_kv; ++jj) {
          const int key0 = it.lo + jj * 128;
          const uint32_t st = k_count % K_NS, n = k_count / K_NS;
          if (n >= 1 && !mbar_wait(&sm.k_empty[st], (n - 1) & 1, wc, hdr)) { ok = false; break; }
          mbar_arrive_expect_tx(&sm.k_full[st], kLoad);
#pragma unroll
          for (int cb = 0; cb < kBlocks; ++cb)
            tma_load_2d(sm.k[st] + cb * kBlk, &tm_k, &sm.k_full[st], it.g * D + cb * 64, key0);
          ++k_count;
          if (v_count >= 1 && !mbar_wait(&sm.v_empty, (v_count - 1) & 1, wc, hdr)) { ok = false; break; }
          mbar_arrive_expect_tx(&sm.v_full, kLoad);
#pragma unroll
          for (int cb = 0; cb < kBlocks; ++cb)
            tma_load_2d(sm.v + cb * kBlk, &tm_v, &sm.v_full, it.g * D + cb * 64, key0);
          ++v_count;
        }
      }
      // leaving, normally or on an abort: every issued copy lands first
      for (uint32_t j = it_count > 2 ? it_count - 2 : 0; j < it_count; ++j)
        drain_wait(&sm.q_full[j & 1], (j >> 1) & 1);
      for (uint32_t j = k_count > K_NS ? k_count - K_NS : 0; j < k_count; ++j)
        drain_wait(&sm.k_full[j % K_NS], (j / K_NS) & 1);
      if (v_count >= 1) drain_wait(&sm.v_full, (v_count - 1) & 1);
    }
  } else if (warp == kQWarpMma) {
    // ------------------------------------------------------------ MMA issuer
    // Products run in issue order, so S_m of the next tile may follow dQ_m,
    // which reads dS_m from the same columns, without a wait.
    if (lane == 0) {
      uint32_t it_count = 0, jc = 0;
      while (true) {
        const uint32_t slot = it_count & 1, use = it_count >> 1;
        if (!wait_one(&sm.item_full[slot], use & 1, wc, hdr)) break;
        const QueryItem it = sm.items[slot];
        mbar_arrive(&sm.item_empty[slot]);
        if (it.n_kv < 0) break;
        if (!wait_one(&sm.q_full[slot], use & 1, wc, hdr)) break;
        const uint32_t q_s = smem_u32(sm.q[slot]), do_s = smem_u32(sm.dout[slot]);
        bool ok = true;
        // S_1 and dP of tile t are issued before dQ_2 of tile t - 1, S_2 after it
        auto issue_s1_dp = [&](uint32_t t) {
          if (!wait_one(&sm.k_full[t % K_NS], (t / K_NS) & 1, wc, hdr)) return false;
          tc_fence_after();
          mma_kk<D / 2>(0, tmem, q_s, smem_u32(sm.k[t % K_NS]));            // S_1 = Q_1 K_1^T
          mma_commit(&sm.s_full[0]);
          if (!wait_one(&sm.v_full, t & 1, wc, hdr)) return false;
          if (t >= 1 && !wait_one(&sm.dp_free, (t - 1) & 1, wc, hdr)) return false;
          tc_fence_after();
          mma_kk<D>(0, tmem + 256, do_s, smem_u32(sm.v));                   // dP = dOut V^T
          mma_commit(&sm.dp_full);
          mma_commit(&sm.v_empty);
          return true;
        };
        auto issue_s2 = [&](uint32_t t) {
          mma_kk<D / 2>(1, tmem + 128, q_s, smem_u32(sm.k[t % K_NS]));
          mma_commit(&sm.s_full[1]);
        };
        if (!issue_s1_dp(jc)) break;
        issue_s2(jc);
        for (int jj = 0; jj < it.n_kv; ++jj, ++jc) {
          const uint32_t k_s = smem_u32(sm.k[jc % K_NS]);
          const bool has_next = jj + 1 < it.n_kv;
          if (!wait_one(&sm.p_full[0], jc & 1, wc, hdr)) { ok = false; break; }
          // the first product overwrites dQ: read by the previous item's epilogue
          if (jj == 0 && it_count >= 1 && !wait_one(&sm.o_free, (it_count - 1) & 1, wc, hdr)) {
            ok = false;
            break;
          }
          tc_fence_after();
          mma_ts_mn<64, D / 2>(tmem + 384, tmem, k_s, 0, jj > 0);           // dQ_1 += dS_1 K_1
          if (has_next && !issue_s1_dp(jc + 1)) { ok = false; break; }
          if (!wait_one(&sm.p_full[1], jc & 1, wc, hdr)) { ok = false; break; }
          tc_fence_after();
          mma_ts_mn<64, D / 2>(tmem + 384 + D / 2, tmem + 128, k_s, D / 2, jj > 0);   // dQ_2 += dS_2 K_2
          mma_commit(&sm.k_empty[jc % K_NS]);
          if (has_next) issue_s2(jc + 1);
        }
        if (!ok) break;
        mma_commit(&sm.q_empty[slot]);
        mma_commit(&sm.o_full);
        ++it_count;
      }
      mma_drain(&sm.drain);               // every product done before TMEM is freed
    }
  } else {
    // ------------------------------------------------------------ softmax + dQ epilogue
    const int wg = warp >> 2, wq = warp & 3;              // key columns 64 wg .. 64 wg + 63
    const int r = wq * 32 + lane;                          // TMEM lane = query row
    const uint32_t lane_base = (uint32_t)(wq * 32) << 16;
    const float sl2 = p.scale * kLog2e;
    const uint64_t sl2x2 = f2_pack(sl2, sl2);
    uint32_t it_count = 0, jc = 0;
    // the next item's row is found, and its vectors read, under the current item
    QueryItem it;
    const int hr = r & ((1 << a.shift) - 1), tr = r >> a.shift;    // the row's head and token in the item
    int lo, hi;                                              // visible keys [lo, hi)
    float nl[2], nd[2], c;
    auto next_item = [&](uint32_t n) {
      if (!wait_warp(&sm.item_full[n & 1], (n >> 1) & 1, wc, hdr)) return false;
      it = sm.items[n & 1];
      mbar_arrive_warp(&sm.item_empty[n & 1], lane);
      lo = hi = 0;
      nl[0] = nl[1] = nd[0] = nd[1] = c = 0.f;
      if (it.n_kv < 0) return true;
      const int64_t row = (int64_t)it.t0 + tr;
      const Span32 doc = document_of_rows(p.cu, p.ndoc, (int64_t)it.t0 + ((wq * 32) >> a.shift), p.q_len,
                                          lane, a.shift);
      if (row < p.q_len) {
        lo = doc.first;
        hi = p.causal ? (int)row + 1 : (int)min((int64_t)doc.last, p.kv_len);
        const int64_t hg = it.h0 >> a.shift, np = a.Tp << a.shift, j = ((int64_t)it.t0 << a.shift) + r;
        const int64_t v1 = 2 * hg * np + j;
        nl[0] = __ldg(a.nlse2 + v1);
        nl[1] = __ldg(a.nlse2 + v1 + np);
        nd[0] = __ldg(a.ndelta + v1);
        nd[1] = __ldg(a.cndelta + hg * np + j);
        c = __ldg(a.coef + hg * np + j);
      }
      return true;
    };
    if (!next_item(0)) it.n_kv = -1;
    bool ok = true;
    while (it.n_kv >= 0) {
      float pdp = 0.f;                                       // sum of P_2 dP over the thread's columns
      for (int jj = 0; jj < it.n_kv; ++jj, ++jc) {
        const int key0 = it.lo + jj * 128 + wg * 64;
        const bool full_w = __all_sync(0xffffffffu, lo <= key0 && key0 + 64 <= hi);
        uint32_t dp[64];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
          const uint32_t s_tm = tmem + lane_base + 128 * m + wg * 64;
          if (!ok) continue;
          if (!wait_warp(&sm.s_full[m], jc & 1, wc, hdr)) { ok = false; continue; }
          tc_fence_after();
          uint32_t x[64];
          tmem_ld32(s_tm, *reinterpret_cast<uint32_t(*)[32]>(x));
          tmem_ld32(s_tm + 32, *reinterpret_cast<uint32_t(*)[32]>(x + 32));
          tmem_wait_ld();
          const uint64_t nl2 = f2_pack(nl[m], nl[m]);
#pragma unroll
          for (int e = 0; e < 32; ++e) {
            float u0, u1;
            f2_unpack(f2_fma(f2_pack(__uint_as_float(x[2 * e]), __uint_as_float(x[2 * e + 1])), sl2x2,
                             nl2), u0, u1);
            x[2 * e] = __float_as_uint(ex2(u0));
            x[2 * e + 1] = __float_as_uint(ex2(u1));
          }
          if (m == 0) {
            if (!wait_warp(&sm.dp_full, jc & 1, wc, hdr)) { ok = false; continue; }
            tc_fence_after();
            const uint32_t dp_tm = tmem + lane_base + 256 + wg * 64;
            tmem_ld32(dp_tm, *reinterpret_cast<uint32_t(*)[32]>(dp));
            tmem_ld32(dp_tm + 32, *reinterpret_cast<uint32_t(*)[32]>(dp + 32));
            tmem_wait_ld();
            tc_fence_before();
            mbar_arrive_warp(&sm.dp_free, lane);
          }
          // dS over the S columns this warp has read; the second map's factor c
          // is taken in with dP - delta: c dP - c delta
          const float f = m == 0 ? 1.f : c, g = nd[m];
          const uint64_t f2 = f2_pack(f, f), g2 = f2_pack(g, g);
          uint64_t sum[2] = {0, 0};
#pragma unroll
          for (int cc = 0; cc < 2; ++cc) {
            const uint32_t bits = column_bits(lo - key0 - 32 * cc, hi - key0 - 32 * cc);
            uint32_t w[16];
#pragma unroll
            for (int e = 0; e < 16; ++e) {
              const int i = 32 * cc + 2 * e;
              const uint64_t pe = f2_pack(__uint_as_float(x[i]), __uint_as_float(x[i + 1]));
              const uint64_t de = f2_pack(__uint_as_float(dp[i]), __uint_as_float(dp[i + 1]));
              float u0, u1;
              if (m == 1) {                // P_2 dP (a masked column's is dropped, whatever it is)
                if (full_w) {
                  sum[e & 1] = f2_fma(pe, de, sum[e & 1]);
                } else {
                  f2_unpack(f2_mul(pe, de), u0, u1);
                  sum[e & 1] = f2_add(sum[e & 1], f2_pack(bits & (1u << (2 * e)) ? u0 : 0.f,
                                                          bits & (2u << (2 * e)) ? u1 : 0.f));
                }
              }
              f2_unpack(f2_mul(pe, f2_fma(de, f2, g2)), u0, u1);
              w[e] = pack_bf16x2(u0, u1);
            }
            if (!full_w) {
#pragma unroll
              for (int i = 0; i < 4; ++i) {                // pairs of columns 8 j + 2 i
                uint32_t mask[4];
                pair_masks(bits >> (2 * i), mask);
#pragma unroll
                for (int j = 0; j < 4; ++j) w[4 * j + i] &= mask[j];
              }
            }
            tmem_st16(s_tm + cc * 16, w);
          }
          tmem_wait_st();
          tc_fence_before();
          mbar_arrive_warp(&sm.p_full[m], lane);
          if (m == 1) {
            float u0, u1;
            f2_unpack(f2_add(sum[0], sum[1]), u0, u1);
            pdp += u0 + u1;
          }
        }
        if (!ok) break;
      }
      if (!ok) break;
      // epilogue: map wg of the row's gradient, and lambda's
      const int64_t row = (int64_t)it.t0 + tr;
      const int h = it.h0 + hr;
      __nv_bfloat16* const dst = a.dq + (row * p.Hq + h) * D + wg * (D / 2);
      const int64_t sum_at = (2 * (int64_t)(it.h0 >> a.shift) + 1) * (a.Tp << a.shift) +
                             ((int64_t)it.t0 << a.shift) + r;
      if (wg == 1) sm.sum[it_count & 1][r] = pdp;
      // (every warp arrives, so that the next item's phase cannot end before a warp
      // that waits for this one)
      mbar_arrive_warp(&sm.sum_full, lane);
      if (!next_item(it_count + 1)) break;
      if (wg == 0) {                       // (read before o_free, which the slot's next writer follows)
        if (!mbar_wait_warp(&sm.sum_full, it_count & 1, wc, hdr)) break;
        const float s = -(pdp + sm.sum[it_count & 1][r]);
        if (row < p.q_len) {
          if (a.dlam != nullptr) st_out(a.dlam + (int64_t)h * p.q_len + row, s);
          else a.dlam_rows[sum_at] = s;
        }
      }
      if (!mbar_wait_warp(&sm.o_full, it_count & 1, wc, hdr)) break;
      tc_fence_after();
#pragma unroll
      for (int cc = 0; cc < D / 64; ++cc) {
        uint32_t v[32];
        tmem_ld32(tmem + lane_base + 384 + wg * (D / 2) + cc * 32, v);
        tmem_wait_ld();
        if (cc == D / 64 - 1) {
          tc_fence_before();
          mbar_arrive_warp(&sm.o_free, lane);
        }
        if (row < p.q_len) store_row32(dst + cc * 32, v, p.scale);
      }
      ++it_count;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kQWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  grid_dep_wait();
}

// dV, dK = sums of the parts' shares, in order.  One block for 128 keys of a KV head and one of
// the two.
constexpr int kJoinThreads = 256;
template <int D>
__global__ void __launch_bounds__(kJoinThreads) diff_bwd_join_kernel(const BwdArgs a) {
  const AttnProblem& p = a.p;
  if (status_bad(p.hdr)) return;
  const bool is_dk = blockIdx.y & 1;
  const int g = blockIdx.y >> 1;
  int q_lo, n_q;
  const int parts = parts_of(a, key_tile_pairs(p, blockIdx.x, a.shift, q_lo, n_q));
  if (parts == 1) return;                          // written whole
  const int64_t size = p.kv_len * p.Hkv * D;
  __nv_bfloat16* const out = is_dk ? a.dk : a.dv;
  const float f = is_dk ? p.scale : 1.f;
  for (int e = threadIdx.x; e < 128 * (D / 8); e += kJoinThreads) {
    const int64_t key = (int64_t)blockIdx.x * 128 + e / (D / 8);
    if (key >= p.kv_len) break;
    const int64_t at = (key * p.Hkv + g) * D + e % (D / 8) * 8;
    const float* src = a.parts + (int64_t)is_dk * size + at;
    float x[8] = {};
#pragma unroll 4
    for (int s = 0; s < parts; ++s, src += 2 * size) {
      const float4 u = __ldcg(reinterpret_cast<const float4*>(src));
      const float4 v = __ldcg(reinterpret_cast<const float4*>(src) + 1);
      x[0] += u.x; x[1] += u.y; x[2] += u.z; x[3] += u.w;
      x[4] += v.x; x[5] += v.y; x[6] += v.z; x[7] += v.w;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] *= f;
    *reinterpret_cast<uint4*>(out + at) = Vec<__nv_bfloat16>::pack(x);
  }
}

template <int D>
cudaError_t launch_d(const CUtensorMap& mq, const CUtensorMap& mdo, const CUtensorMap& mk,
                     const CUtensorMap& mv, const BwdArgs& a, cudaStream_t s) {
  cudaError_t e = launch_persistent<2 * D>(diff_bwd_dkdv_tc_kernel<D>, kKvThreads,
                                                 smem_bytes<SmemKV>(), s, mq, mdo, mk, mv, a);
  if (e != cudaSuccess) return e;
  e = launch_persistent<2 * D + 1>(diff_bwd_dq_tc_kernel<D>, kQThreads, smem_bytes<SmemQ>(), s, mq, mdo,
                                   mk, mv, a);
  if (e != cudaSuccess || a.n_parts == 1) return e;
  diff_bwd_join_kernel<D><<<dim3((unsigned)ceil_div(a.p.kv_len, 128), 2 * a.p.Hkv), kJoinThreads, 0, s>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_diff_bwd_tc(const DiffProblem& d, const BwdWsLayout& L, char* ws, cudaStream_t s) {
  const AttnProblem& p = d.p;
  CUtensorMap mq, mdo, mk, mv;
  const int64_t kc = (int64_t)p.Hkv * p.d;
  if (!diff_tile_map(&mk, p.k, p.kv_len, kc) || !diff_tile_map(&mv, p.v, p.kv_len, kc) ||
      !diff_heads_map(&mq, p.q, p.q_len, p.Hq, p.d, 1 << d.shift) ||
      !diff_heads_map(&mdo, d.dout, p.q_len, p.Hq, p.d, 1 << d.shift))
    return cudaErrorNotSupported;
  BwdArgs a;
  a.p = p;
  a.nlse2 = d.nlse2; a.ndelta = d.ndelta; a.coef = d.coef; a.cndelta = d.cndelta; a.Tp = d.Tp;
  a.dq = reinterpret_cast<__nv_bfloat16*>(d.dq);
  a.dk = reinterpret_cast<__nv_bfloat16*>(d.dk);
  a.dv = reinterpret_cast<__nv_bfloat16*>(d.dv);
  a.shift = d.shift;
  a.dlam_rows = d.ndelta;
  a.dlam = d.n_lambda > 1 ? reinterpret_cast<__nv_bfloat16*>(d.dlambda) : nullptr;
  a.parts = d.parts;
  a.n_parts = key_parts(p.kv_len, p.Hkv);
  a.qorder = reinterpret_cast<const int*>(ws + L.qorder);
  a.korder = reinterpret_cast<const int*>(ws + L.korder);
  return p.d == 128 ? launch_d<128>(mq, mdo, mk, mv, a, s) : launch_d<64>(mq, mdo, mk, mv, a, s);
}

}  // namespace nsp
