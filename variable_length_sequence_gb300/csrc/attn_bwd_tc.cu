// Varlen attention backward on the tcgen05 tensor cores, bf16 inputs,
// float32 accumulation, head dimension D = 128 or 64: persistent kernels,
// no atomics on the whole-stream path.
//
// Gradients of L = sum(dOut * out) for document-masked attention (BASP
// Sec. II-A, HSAP Sec. 2.1), recomputing the probabilities from the saved
// lse instead of storing them (the recomputation NSP Sec. 2.3 discusses):
//   P = exp(scale Q K^T - lse),  dP = dOut V^T,  dS = P (dP - delta),
//   dV = P^T dOut,  dK = scale dS^T Q,  dQ = scale dS K,
// with delta = rowsum(dOut * out) and -lse * log2(e) prepared by
// bwd_delta_kernel in padded [Hq, Tp] rows.
//
// Both kernels use 128 x 128 x 128 products only, and issue them from two
// threads (two tcgen05 streams): products of one thread run in issue order,
// so a product that must wait for the softmax would otherwise hold up the
// independent products queued behind it.
//
// dK/dV kernel (key-stationary).  Work item: one 128-key tile of one KV
// head; it walks every (query head of the group, 128-row query tile that
// can see the keys) pair.  TMEM: two 128-column score regions [0,256) that
// swap roles every step (step qc puts S^T in region qc & 1 and dP^T in the
// other), dV [256,384), dK [384,512).  Stream 1 issues S^T = K Q^T and
// dP^T = V dOut^T; the softmax warpgroups read S^T, write P^T (bf16) back
// over it, then read dP^T and write dS^T (bf16) to shared memory in a
// 128-byte-swizzled layout; stream 2 issues dV += P^T dOut (A from TMEM) and
// dK += dS^T Q (A from shared memory).  The next S^T goes into the region
// the softmax has just read dP^T from, and the next dP^T into the region
// whose P^T dV has consumed, so stream 1 works on step qc + 1 while the
// softmax and stream 2 are on step qc.  dK and dV are written once per item,
// in bf16.
//
// dQ kernel (query-stationary).  Work item: one 128-row query tile of one
// query head; it walks the 128-key tiles its rows can see.  TMEM: S
// double-buffered [0,128) and [128,256), dP [256,384), dQ [384,512).
// Stream 1 issues S = Q K^T (into the free S buffer, while the softmax is
// still on the other one); dP = dOut V^T is issued by stream 1 for even and
// by stream 2 for odd tiles of an item, so that both streams carry three
// products per two tiles; the softmax frees dP as soon as it has read it and
// writes dS = P (dP - delta) (bf16) back over S; stream 2 issues
// dQ += dS K (A from TMEM).  K tiles have three shared-memory stages (they
// are read until dQ of their tile is done), V tiles two.  dQ is scaled and
// written once per item, in bf16.
//
// dS cache (workspace past the layout, when every visible tile pair's dS
// fits): the dK/dV kernel also bulk-copies each dS^T tile it builds to the
// cache, and a third kernel computes dQ += dS K from the cached tiles (one
// product per tile pair instead of the dQ kernel's three); the dQ kernel
// then returns at once.
//
// Roles, dQ kernel: warps 0-3 and 4-7 are the softmax / epilogue
// warpgroups (one TMEM lane each; they split the 128 columns of each tile in
// halves), warp 8 is the TMA producer and work fetcher, warp 9 allocates
// TMEM and one of its threads issues stream 1, one thread of warp 10 issues
// stream 2.  dK/dV kernel: 16 softmax / epilogue warps (four column groups
// of four lane quadrants), warp 16 the producer, warp 17 TMEM and stream 1,
// warp 18 stream 2 (and the dS cache copies), warp 19 idle so that the
// control warpgroup can hand registers to the softmax warps (setmaxnreg).
// Masking is one unsigned compare per element against the row's (or key's)
// visible interval, skipped for fully visible chunks.  All waits are
// bounded.
#include <cudaTypedefs.h>

#include "tc_ptx.cuh"

namespace nsp {
namespace {

using namespace tc;

constexpr int kThreads = 352;                        // dQ kernel
constexpr int kKvThreads = 640;                      // dK/dV kernel: 16 softmax warps + 4
constexpr int kKvSoftmaxWarps = 16;
constexpr int kKvWarpProducer = 16, kKvWarpMma1 = 17, kKvWarpMma2 = 18;   // warp 19 idle
constexpr int kKvRegsControl = 64, kKvRegsSoftmax = 104;   // 128 x 64 + 512 x 104 = 640 x 96
constexpr int kWarpProducer = 8, kWarpMma1 = 9, kWarpMma2 = 10;
constexpr uint32_t kBlk = 128 * 64 * 2;               // 128 rows x 64 bf16 column block
constexpr uint32_t kTile = 2 * kBlk;                   // 128 x 128 bf16
constexpr float kLog2e = 1.4426950408889634f;
constexpr size_t kSmemLimit = 232448;

constexpr uint32_t kIdescKK = idesc_bf16_f32(128, 128, false, false);   // A, B K-major
// B MN-major, N = the head dimension D
template <int D>
__host__ __device__ constexpr uint32_t idesc_km() { return idesc_bf16_f32(128, D, true, false); }

// D = A B^T, A and B K-major 128-row tiles (128-byte swizzle), K = the
// head dimension HK (128, or 64: the first column block only).
template <int HK>
__device__ __forceinline__ void mma_kk(uint32_t d_tmem, uint32_t a_saddr, uint32_t b_saddr,
                                       bool accumulate) {
  const uint64_t ad = smem_desc_sw128(a_saddr, 16, 1024);
  const uint64_t bd = smem_desc_sw128(b_saddr, 16, 1024);
#pragma unroll
  for (int kk = 0; kk < HK / 16; ++kk) {
    const uint32_t off = ((kk >> 2) * kBlk + (kk & 3) * 32) >> 4;
    mma_ss(d_tmem, ad + off, bd + off, kIdescKK, (accumulate || kk > 0) ? 1u : 0u);
  }
}

// D (+)= A B, A from TMEM, B MN-major in shared memory (K along its rows,
// 16 rows = 2048 B per step; N = D columns, blocks of 64 16 KB apart).  A
// holds bf16 pairs written by the softmax warps in groups of QPG K-columns:
// group j sits at TMEM columns a_tmem + j QPG + [0, QPG / 2), so K-step kk
// (16 columns, 8 TMEM columns) starts at (kk / (QPG / 16)) QPG +
// (kk % (QPG / 16)) 8.
template <int QPG, int D>
__device__ __forceinline__ void mma_t_split(uint32_t d_tmem, uint32_t a_tmem, uint32_t b_saddr,
                                            bool accumulate) {
  constexpr int kSteps = QPG / 16;
  const uint64_t bd = smem_desc_sw128(b_saddr, kBlk, 1024);
#pragma unroll
  for (int kk = 0; kk < 8; ++kk) {
    const uint32_t a_col = (kk / kSteps) * QPG + (kk % kSteps) * 8;
    mma_ts(d_tmem, a_tmem + a_col, bd + ((kk * 2048) >> 4), idesc_km<D>(),
           (accumulate || kk > 0) ? 1u : 0u);
  }
}

__device__ __forceinline__ void store_row32_bf16(__nv_bfloat16* dst, const uint32_t (&v)[32],
                                                 float scale) {
  uint32_t w[16];
#pragma unroll
  for (int i = 0; i < 16; ++i)
    w[i] = pack_bf16x2(__uint_as_float(v[2 * i]) * scale, __uint_as_float(v[2 * i + 1]) * scale);
#pragma unroll
  for (int i = 0; i < 2; ++i)
    st_global_v8(dst + 16 * i, w[8 * i], w[8 * i + 1], w[8 * i + 2], w[8 * i + 3], w[8 * i + 4],
                 w[8 * i + 5], w[8 * i + 6], w[8 * i + 7]);
}

// dst[0..31] = scale * v (raw float32 bits), a float32 row chunk (16-byte
// aligned: rows are 512 bytes, chunks 128).
__device__ __forceinline__ void store_row32_f32(float* dst, const uint32_t (&v)[32], float scale) {
  float4* d4 = reinterpret_cast<float4*>(dst);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    d4[i] = make_float4(__uint_as_float(v[4 * i]) * scale, __uint_as_float(v[4 * i + 1]) * scale,
                        __uint_as_float(v[4 * i + 2]) * scale,
                        __uint_as_float(v[4 * i + 3]) * scale);
}

// Ring block: a TMEM accumulator's 32 columns of this thread's lane start as
// src[0..31] * mul (zero when src is null), so the block's products add onto
// the running float32 gradient and the epilogue writes it back whole.
__device__ __forceinline__ void preload_row32(uint32_t taddr, const float* src, float mul) {
  uint32_t v[32];
  const float4* s4 = reinterpret_cast<const float4*>(src);
#pragma unroll
  for (int i = 0; i < 8; ++i) {
    const float4 x = src != nullptr ? __ldcg(s4 + i) : make_float4(0.f, 0.f, 0.f, 0.f);
    v[4 * i] = __float_as_uint(x.x * mul);
    v[4 * i + 1] = __float_as_uint(x.y * mul);
    v[4 * i + 2] = __float_as_uint(x.z * mul);
    v[4 * i + 3] = __float_as_uint(x.w * mul);
  }
  tmem_st32(taddr, v);
}

// dst[0..31] += scale * v as float4 atomic reductions (rows shared by items).
__device__ __forceinline__ void red_row32_f32(float* dst, const uint32_t (&v)[32], float scale) {
  float4* d4 = reinterpret_cast<float4*>(dst);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    atomicAdd(d4 + i, make_float4(__uint_as_float(v[4 * i]) * scale,
                                  __uint_as_float(v[4 * i + 1]) * scale,
                                  __uint_as_float(v[4 * i + 2]) * scale,
                                  __uint_as_float(v[4 * i + 3]) * scale));
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

struct BwdArgs {
  AttnProblem p;
  const float* nlse2;     // [Hq, Tp] -lse * log2(e)
  const float* delta;     // [Hq, Tp]
  int64_t Tp;
  int hsplit;             // dK/dV items per (key tile, KV head): each takes G / hsplit
                          // query heads (> 1 only when accumulating with atomics)
  __nv_bfloat16* dq;      // [q_len, Hq, d]
  __nv_bfloat16* dk;      // [kv_len, Hkv, d]
  __nv_bfloat16* dv;
  float* dq_acc;          // ring block (p.accumulate): float32 accumulators, same shapes
  float* dk_acc;
  float* dv_acc;
  const int2* qtiles;     // per 128-row query tile: first/last 128-key tile
  const int* qorder;
  const int2* ktiles;     // per 128-key tile: first/last 128-row query tile
  const int* korder;
  // dS cache (whole-stream or batched call, header flag ds_on): the dK/dV
  // kernel copies every dS^T tile it builds to slot h * ds_pairs + qoff[i] +
  // (key tile - first key tile of scheduled query tile i), and the dQ kernel
  // of the cache reads them instead of recomputing S and dP
  uint8_t* ds_cache;
  const int64_t* qoff;
};

// Block of a batched call's scheduled tile t: the largest index whose first
// tile (key tiles: ktile0, query tiles: tile0) is <= t.
template <bool KEY>
__device__ __forceinline__ int block_of(const FwdBlocks& B, int t) {
  int lo = 0, hi = B.n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if ((KEY ? B.b[mid].ktile0 : B.b[mid].tile0) <= t) lo = mid; else hi = mid - 1;
  }
  return lo;
}

// ================================================================ dK / dV

struct KvItem {
  int ktile, g, h0, i_lo, n_q, steps;   // heads h0 .., steps = heads * n_q; -1 stops
  int blk, pad;                         // block of a batched call (MULTI)
};

struct __align__(1024) SmemKV {
  uint8_t k[kTile];
  uint8_t v[kTile];
  // Q / dOut pool: Q of step j in slot j % 4, dOut of step j in slot
  // (j + 2) % 4, both the (j / 2)-th fill of their slot.  Every slot
  // alternates Q and dOut roles, so Q of step j + 2 lands in the slot that
  // dOut of step j frees in the middle of step j (after dV), not in the one
  // Q of step j frees at its end (after dK).
  uint8_t qd[4][kTile];
  uint8_t ds[kTile];            // dS^T, [q-block][key][64 q], 128-byte swizzle
  float vec[4][128];            // -lse log2(e) with a Q tile, delta with a dOut tile
  uint64_t kv_full, kv_empty;
  uint64_t slot_full[4], slot_empty[4];
  uint64_t s_full, dp_full, dp_free, ds_ready, dk_done;
  uint64_t p_ready[2], dv_done[2];
  uint64_t dkv_full, dkv_empty;
  uint64_t item_full[2], item_empty[2];
  KvItem items[2];
  uint64_t drain1, drain2;      // each MMA stream's own barrier for its final drain
  uint64_t ds_stored;           // dS cache: the copy of the previous dS^T has left ds
  uint32_t tmem_base;
  WaitCtl wait;
};
static_assert(sizeof(SmemKV) <= kSmemLimit, "dK/dV tile set exceeds shared memory");

// MULTI: a batched call (nsp_attn_bwd_blocks): the tiles of every block of
// blks, rows addressed by global token ids, every contribution added into the
// whole-stream float32 accumulators with atomics (no preload).  D: the head
// dimension, 128 or 64 (tiles of 64 columns use the first column block of
// each tile buffer, dV and dK the first 64 of their TMEM columns, and the
// column groups of the epilogue that would hold columns 64-127 idle).
template <bool MULTI, int D>
__global__ void __launch_bounds__(kKvThreads, 1)
    attn_bwd_dkdv_tc_kernel(const __grid_constant__ CUtensorMap tm_q,
                            const __grid_constant__ CUtensorMap tm_do,
                            const __grid_constant__ CUtensorMap tm_k,
                            const __grid_constant__ CUtensorMap tm_v, const BwdArgs a,
                            const __grid_constant__ FwdBlocks blks) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const AttnProblem& p = a.p;
  WsHeader* hdr = p.hdr;
  grid_dep_wait();                          // delta and -lse log2(e) of bwd_delta_kernel
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
      // one commit from each stream (Q: S^T, dK; dOut: dP^T, dV) and one
      // arrival per softmax warp (its lse or delta read)
      mbar_init(&sm.slot_empty[s], 2 + kKvSoftmaxWarps);
    }
    for (int s = 0; s < 2; ++s) {
      mbar_init(&sm.p_ready[s], kKvSoftmaxWarps);
      mbar_init(&sm.dv_done[s], 1);
      mbar_init(&sm.item_full[s], 1);
      mbar_init(&sm.item_empty[s], 2 + kKvSoftmaxWarps);
    }
    mbar_init(&sm.s_full, 1);
    mbar_init(&sm.dp_full, 1);
    mbar_init(&sm.dp_free, kKvSoftmaxWarps);
    mbar_init(&sm.ds_ready, kKvSoftmaxWarps);
    mbar_init(&sm.dk_done, 1);
    mbar_init(&sm.dkv_full, 1);
    mbar_init(&sm.dkv_empty, kKvSoftmaxWarps);
    mbar_init(&sm.drain1, 1);
    mbar_init(&sm.drain2, 1);
    mbar_init(&sm.ds_stored, 1);
    wait_ctl_init(&sm.wait, p.wait_budget);
    fence_mbar_init();
  }
  if (warp == kKvWarpMma1) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  if (warp == kKvWarpProducer && lane == 0) {
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
  const int64_t n_keys = p.kv_len;           // keys of the range (row index of K, V, dK, dV)
  const int n_per_tile = p.Hkv * a.hsplit;   // items per key tile
  const int n_items = hdr->n_items2 * n_per_tile;
  const int heads_per_item = G / a.hsplit;
  constexpr int kBlocks = D / 64;                        // 64-column blocks of a row
  constexpr uint32_t kLoad = kBlocks * kBlk;             // one Q, dOut, K or V tile
  // the schedule found room for every visible tile pair's dS in the cache
  const bool ds_on = a.ds_cache != nullptr && *((volatile const int32_t*)&hdr->ds_on) != 0;
  const int64_t ds_pairs = ds_on ? *((volatile const int64_t*)&hdr->ds_pairs) : 0;

  if (warp >= 16) {
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(kKvRegsControl));
    if (warp == kKvWarpProducer) {
      // ------------------------------------------------------------ producer
      if (lane == 0) {
        uint32_t it_count = 0, kv_count = 0, q_count = 0, loads = 0;
        bool ok = true;
        while (ok) {
          const int idx = atomicAdd(&hdr->counter2, 1);
          KvItem it;
          it.ktile = 0; it.g = 0; it.h0 = 0; it.i_lo = 0; it.n_q = 0; it.steps = -1; it.blk = 0;
          if (idx < n_items) {
            const int kt = a.korder[idx / n_per_tile];
            const int2 tr = a.ktiles[kt];
            const int rem = idx - (idx / n_per_tile) * n_per_tile;
            it.ktile = kt;
            if constexpr (MULTI) {
              it.blk = block_of<true>(blks, kt);
              it.ktile = kt - blks.b[it.blk].ktile0;         // key tile within its block
            }
            it.g = rem / a.hsplit;
            it.h0 = it.g * G + (rem - it.g * a.hsplit) * heads_per_item;
            it.i_lo = tr.x;
            it.n_q = tr.y - tr.x + 1;
            it.steps = heads_per_item * it.n_q;
          }
          const uint32_t slot = it_count & 1;
          if (it_count >= 2 &&
              !mbar_wait(&sm.item_empty[slot], ((it_count >> 1) - 1) & 1, wc, hdr)) {
            ok = false;
            break;
          }
          sm.items[slot] = it;
          mbar_arrive(&sm.item_full[slot]);
          ++it_count;
          if (it.steps < 0) break;
          if (it.steps == 0) continue;            // no query of the range sees these keys
          if (kv_count >= 1 && !mbar_wait(&sm.kv_empty, (kv_count - 1) & 1, wc, hdr)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&sm.kv_full, 2 * kLoad);
          // a batched call's maps span the whole stream (rows = global ids)
          const int k_base = MULTI ? blks.b[it.blk].kv_start : 0;
          const int q_base = MULTI ? blks.b[it.blk].q_start : 0;
#pragma unroll
          for (int cb = 0; cb < kBlocks; ++cb) {
            tma_load_2d(sm.k + cb * kBlk, &tm_k, &sm.kv_full, it.g * D + cb * 64,
                        k_base + it.ktile * 128);
            tma_load_2d(sm.v + cb * kBlk, &tm_v, &sm.kv_full, it.g * D + cb * 64,
                        k_base + it.ktile * 128);
          }
          ++kv_count;
          for (int n = 0; n < it.steps; ++n) {
            const int hh = n / it.n_q;
            const int h = it.h0 + hh;
            const int i = it.i_lo + (n - hh * it.n_q);
            const uint32_t fill = q_count >> 1;             // fill index of both slots
            const uint32_t sq = q_count & 3, sd = (q_count + 2) & 3;
            if (q_count >= 2 &&
                !mbar_wait(&sm.slot_empty[sq], (fill - 1) & 1, wc, hdr)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&sm.slot_full[sq], kLoad + 128 * sizeof(float));
            // packed q / dOut: map [q_len, Hq d]; head groups: [P q_len, (Hq/P) d]
            int qx = h * D, qy = q_base + i * 128;
            if (p.q_groups > 1) {
              const int hpg = p.Hq / p.q_groups, grp = h / hpg;
              qx = (h - grp * hpg) * D;
              qy += (int)(grp * p.q_len);
            }
#pragma unroll
            for (int cb = 0; cb < kBlocks; ++cb)
              tma_load_2d(sm.qd[sq] + cb * kBlk, &tm_q, &sm.slot_full[sq], qx + cb * 64, qy);
            const int64_t row = (int64_t)h * a.Tp + q_base + (int64_t)i * 128;
            bulk_load(sm.vec[sq], a.nlse2 + row, 128 * sizeof(float), &sm.slot_full[sq]);
            ++loads;
            if (q_count >= 2 &&
                !mbar_wait(&sm.slot_empty[sd], (fill - 1) & 1, wc, hdr)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&sm.slot_full[sd], kLoad + 128 * sizeof(float));
#pragma unroll
            for (int cb = 0; cb < kBlocks; ++cb)
              tma_load_2d(sm.qd[sd] + cb * kBlk, &tm_do, &sm.slot_full[sd], qx + cb * 64, qy);
            bulk_load(sm.vec[sd], a.delta + row, 128 * sizeof(float), &sm.slot_full[sd]);
            ++loads;
            ++q_count;
          }
        }
        {
          // leaving, normally or on an abort: every copy issued so far lands on
          // its stage barrier before the CTA exits
          if (kv_count >= 1) drain_wait(&sm.kv_full, (kv_count - 1) & 1);
          // load l: step l / 2, Q (l even) or dOut (l odd)
          for (uint32_t l = (loads > 4 ? loads - 4 : 0); l < loads; ++l) {
            const uint32_t j = l >> 1;
            drain_wait(&sm.slot_full[(l & 1) ? ((j + 2) & 3) : (j & 3)], (j >> 1) & 1);
          }
        }
      }
    } else if (warp == kKvWarpMma1) {
      // ------------------------------------------------------------ stream 1: S^T, dP^T
      // Step qc puts S^T in region qc & 1 and dP^T in the other one; the two
      // regions swap roles every step.
      if (lane == 0) {
        const uint32_t k_s = smem_u32(sm.k), v_s = smem_u32(sm.v);
        uint32_t it_count = 0, items_done = 0, qc = 0;
        bool ok = true;
        while (ok) {
          const uint32_t slot = it_count & 1;
          if (!mbar_wait(&sm.item_full[slot], (it_count >> 1) & 1, wc, hdr)) break;
          const KvItem it = sm.items[slot];
          mbar_arrive(&sm.item_empty[slot]);
          ++it_count;
          if (it.steps < 0) break;
          if (it.steps == 0) continue;
          if (!mbar_wait(&sm.kv_full, items_done & 1, wc, hdr)) break;
          for (int n = 0; n < it.steps; ++n) {
            const uint32_t sq = qc & 3, sd = (qc + 2) & 3, fp = (qc >> 1) & 1, rb = qc & 1;
            if (!mbar_wait(&sm.slot_full[sq], fp, wc, hdr)) { ok = false; break; }
            // region rb held the previous dP^T: free once the softmax has read it
            if (qc >= 1 && !mbar_wait(&sm.dp_free, (qc - 1) & 1, wc, hdr)) { ok = false; break; }
            tc_fence_after();
            mma_kk<D>(tmem + 128 * rb, k_s, smem_u32(sm.qd[sq]), false);      // S^T = K Q^T
            mma_commit(&sm.s_full);
            mma_commit(&sm.slot_empty[sq]);
            if (!mbar_wait(&sm.slot_full[sd], fp, wc, hdr)) { ok = false; break; }
            // region rb ^ 1 held the previous P^T: free once dV has read it
            if (qc >= 1 && !mbar_wait(&sm.dv_done[rb ^ 1], ((qc - 1) >> 1) & 1, wc, hdr)) {
              ok = false;
              break;
            }
            tc_fence_after();
            mma_kk<D>(tmem + 128 * (rb ^ 1), v_s, smem_u32(sm.qd[sd]), false);   // dP^T = V dOut^T
            mma_commit(&sm.dp_full);
            mma_commit(&sm.slot_empty[sd]);
            ++qc;
          }
          if (!ok) break;
          mma_commit(&sm.kv_empty);
          ++items_done;
        }
        mma_drain(&sm.drain1);            // every product done before TMEM is freed
      }
    } else if (warp == kKvWarpMma2) {
      // ------------------------------------------------------------ stream 2: dV, dK
      if (lane == 0) {
        const uint32_t ds_s = smem_u32(sm.ds);
        const uint64_t ds_pol = l2_evict_first_policy();   // cached dS: not read in this kernel
        uint32_t it_count = 0, items_done = 0, qc = 0;
        bool ok = true, ds_pending = false;
        while (ok) {
          const uint32_t slot = it_count & 1;
          if (!mbar_wait(&sm.item_full[slot], (it_count >> 1) & 1, wc, hdr)) break;
          const KvItem it = sm.items[slot];
          mbar_arrive(&sm.item_empty[slot]);
          ++it_count;
          if (it.steps < 0) break;
          if (it.steps == 0) continue;
          for (int n = 0; n < it.steps; ++n) {
            const uint32_t sq = qc & 3, sd = (qc + 2) & 3, fp = (qc >> 1) & 1, rb = qc & 1;
            uint8_t* ds_dst = nullptr;               // this step's dS slot
            if (ds_on) {
              const int hh = n / it.n_q;
              // scheduled query tile (a batched call's tiles follow its blocks)
              const int i = it.i_lo + (n - hh * it.n_q) + (MULTI ? blks.b[it.blk].tile0 : 0);
              const int2 tr = __ldg(a.qtiles + i);
              const int kofs = it.ktile - tr.x;      // < the tile's listed count (schedules agree)
              if (kofs >= 0 && kofs <= tr.y - tr.x)
                ds_dst = a.ds_cache +
                         ((int64_t)(it.h0 + hh) * ds_pairs + __ldg(a.qoff + i) + kofs) *
                             (int64_t)kTile;
              else
                atomicCAS(&hdr->status, 0, (int32_t)NSP_ERR_INVALID);   // no copy out of bounds
            }
            if (!mbar_wait(&sm.p_ready[rb], fp, wc, hdr)) { ok = false; break; }
            if (ds_pending) {
              // the copy of the previous dS^T has read its shared memory
              bulk_wait_read_all();
              mbar_arrive(&sm.ds_stored);
              ds_pending = false;
            }
            if (n == 0 && items_done > 0 &&
                !mbar_wait(&sm.dkv_empty, (items_done - 1) & 1, wc, hdr)) {
              ok = false;
              break;
            }
            if (!mbar_wait(&sm.slot_full[sd], fp, wc, hdr)) { ok = false; break; }
            tc_fence_after();
            // a ring block with one item per (key tile, KV head) adds onto the
            // preloaded running dK / dV
            const bool acc = n > 0 || (!MULTI && p.accumulate && a.hsplit == 1);
            mma_t_split<32, D>(tmem + 256, tmem + 128 * rb, smem_u32(sm.qd[sd]), acc);   // dV += P^T dOut
            mma_commit(&sm.dv_done[rb]);
            mma_commit(&sm.slot_empty[sd]);
            if (!mbar_wait(&sm.ds_ready, qc & 1, wc, hdr)) { ok = false; break; }
            tc_fence_after();
            {
              // dK += dS^T Q: A = dS^T K-major (rows = keys), B = Q MN-major
              const uint64_t ad = smem_desc_sw128(ds_s, 16, 1024);
              const uint64_t bd = smem_desc_sw128(smem_u32(sm.qd[sq]), kBlk, 1024);
#pragma unroll
              for (int kk = 0; kk < 8; ++kk) {
                const uint32_t aoff = ((kk >> 2) * kBlk + (kk & 3) * 32) >> 4;
                mma_ss(tmem + 384, ad + aoff, bd + ((kk * 2048) >> 4), idesc_km<D>(),
                       (acc || kk > 0) ? 1u : 0u);
              }
            }
            mma_commit(&sm.dk_done);
            mma_commit(&sm.slot_empty[sq]);
            if (ds_on) {
              if (ds_dst != nullptr) {
                bulk_store(ds_dst, sm.ds, kTile, ds_pol);
                bulk_commit();
              }
              ds_pending = true;
            }
            ++qc;
          }
          if (!ok) break;
          mma_commit(&sm.dkv_full);
          ++items_done;
        }
        if (ds_on) bulk_wait_all();       // the cached dS is in memory before the CTA exits
        mma_drain(&sm.drain2);
      }
    }
  } else {
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(kKvRegsSoftmax));
    // ------------------------------------------------------------ softmax + dK/dV epilogue
    // Warp (cg, wq) covers TMEM lane quadrant wq (32 keys) and query columns
    // 32 cg .. 32 cg + 31.  Scores are read as 16-lane fragments (16x256b,
    // two loads per quadrant): thread t holds key rows wq 32 + t/4 + 8 i
    // (i = 0..3) at columns 8 j + 2 (t % 4) + {0, 1} (j = 0..3), so it needs
    // the lse and delta of 8 columns only, read as 4 float pairs each.
    // Register x[16 h + 4 j + 2 e + u] is row 16 h + 8 e + t/4, column
    // 8 j + 2 (t % 4) + u; fragment row index i = 2 h + e.
    const int cg = warp >> 2;
    const int wq = warp & 3;
    const int r = wq * 32 + lane;                          // epilogue: TMEM lane = key row
    // epilogue: column group cg & 1 holds head-dimension columns 64 (cg & 1) ..
    const bool epi_cols = (cg & 1) * 64 < D;
    const int tr = lane >> 2, tc2 = 2 * (lane & 3);
    const uint32_t lane_base = (uint32_t)(wq * 32) << 16;
    const float sl2 = p.scale * kLog2e;
    const uint64_t sl2x2 = f2_pack(sl2, sl2);
    // dS^T tile: query block cg / 2, 16-byte chunks 4 (cg & 1) + j, swizzled
    // by key & 7 (= tr for every fragment row)
    const uint32_t ds_base = smem_u32(sm.ds) + (cg >> 1) * kBlk + (wq * 32 + tr) * 128 + 2 * tc2;
    uint32_t it_count = 0, items_done = 0, qc = 0;
    bool ok = true;
    while (ok) {
      const uint32_t slot = it_count & 1;
      if (!mbar_wait_warp(&sm.item_full[slot], (it_count >> 1) & 1, wc, hdr)) break;
      const KvItem it = sm.items[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.item_empty[slot]);
      ++it_count;
      if (it.steps < 0) break;
      if (it.steps == 0) {
        // no query of the range sees these keys: the whole-stream backward
        // writes zero rows (a ring block adds nothing)
        if (!p.accumulate && epi_cols) {
          const int64_t key = (int64_t)it.ktile * 128 + r;
          __nv_bfloat16* dst = (cg >= 2 ? a.dk : a.dv) + (key * p.Hkv + it.g) * D + (cg & 1) * 64;
          uint32_t z[32];
#pragma unroll
          for (int i = 0; i < 32; ++i) z[i] = 0u;
          if (key < n_keys) {
            store_row32_bf16(dst, z, 0.f);
            store_row32_bf16(dst + 32, z, 0.f);
          }
        }
        continue;
      }
      // the item's ranges: its block's (batched call) or the call's
      const int64_t it_kv_start = MULTI ? (int64_t)blks.b[it.blk].kv_start : p.kv_start;
      const int64_t it_keys = MULTI ? (int64_t)blks.b[it.blk].kv_len : n_keys;
      const int64_t it_q_start = MULTI ? (int64_t)blks.b[it.blk].q_start : p.q_start;
      const int64_t it_q_len = MULTI ? (int64_t)blks.b[it.blk].q_len : p.q_len;
      int qlo[4], qhi[4];                                   // queries (range-relative) that see fragment row i
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t key = (int64_t)it.ktile * 128 + wq * 32 + tr + 8 * i;
        qlo[i] = 0;
        qhi[i] = 0;
        if (key < it_keys) {
          const int64_t kg = it_kv_start + key;
          const int b = doc_of(p.cu, p.ndoc, kg);
          const int64_t glo = p.causal ? kg : (int64_t)__ldg(p.cu + b);
          const int64_t ghi = __ldg(p.cu + b + 1);
          qlo[i] = (int)min(max(glo - it_q_start, (int64_t)0), it_q_len);
          qhi[i] = (int)min(max(ghi - it_q_start, (int64_t)0), it_q_len);
        }
      }
      if (!MULTI && p.accumulate && a.hsplit == 1 && epi_cols) {
        // ring block, one item per (key tile, KV head): dV and dK start as the
        // running accumulators (dK / scale), TMEM lane = key row
        const int64_t key = (int64_t)it.ktile * 128 + r;
        const bool is_dk = cg >= 2;
        const float* src = key < n_keys ? (is_dk ? a.dk_acc : a.dv_acc) +
                                              (key * p.Hkv + it.g) * D + (cg & 1) * 64
                                        : nullptr;
        const uint32_t col = (is_dk ? 384u : 256u) + (cg & 1) * 64;
        const float mul = is_dk ? 1.f / p.scale : 1.f;
        preload_row32(tmem + lane_base + col, src, mul);
        preload_row32(tmem + lane_base + col + 32, src ? src + 32 : nullptr, mul);
        tmem_wait_st();
      }
      for (int n = 0; n < it.steps; ++n) {
        const int hh = n / it.n_q;
        const int q0 = (it.i_lo + (n - hh * it.n_q)) * 128 + cg * 32;
        const uint32_t sq = qc & 3, sd = (qc + 2) & 3, fp = (qc >> 1) & 1, rb = qc & 1;
        const uint32_t s_tm = tmem + lane_base + 128 * rb + cg * 32;
        const uint32_t dp_tm = tmem + lane_base + 128 * (rb ^ 1) + cg * 32;
        if (!mbar_wait_warp(&sm.slot_full[sq], fp, wc, hdr)) { ok = false; break; }
        if (!mbar_wait_warp(&sm.s_full, qc & 1, wc, hdr)) { ok = false; break; }
        tc_fence_after();
        uint32_t x[32];
        tmem_ld16x256_x4(s_tm, x);
        tmem_ld16x256_x4(s_tm + (16u << 16), x + 16);
        uint64_t nl[4];                                     // -lse log2(e) column pairs
        {
          const float* src = sm.vec[sq] + cg * 32 + tc2;
#pragma unroll
          for (int j = 0; j < 4; ++j) nl[j] = *reinterpret_cast<const uint64_t*>(src + 8 * j);
        }
        int loc[4];
        uint32_t span[4];
        bool full = true;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          loc[i] = min(max(qlo[i] - q0, 0), 32);
          const int hic = min(max(qhi[i] - q0, 0), 32);
          span[i] = (uint32_t)(hic - loc[i]);
          full = full && loc[i] == 0 && hic == 32;
        }
        const bool full_w = __all_sync(0xffffffffu, full);
        tmem_wait_ld();
        // phase 1: P = exp2(S sl2 - lse2), masked; P^T (bf16 pairs) goes back
        // over the first 16 of the S^T columns this warp has read
        uint64_t pp[16];                                   // P, float pairs
        uint32_t pk[16];
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int j = (k >> 1) & 3;
          pp[k] = f2_fma(f2_pack(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])),
                         sl2x2, nl[j]);
        }
        if (full_w) {
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            float u0, u1;
            f2_unpack(pp[k], u0, u1);
            u0 = ex2(u0);
            u1 = ex2(u1);
            pp[k] = f2_pack(u0, u1);
            pk[k] = pack_bf16x2(u0, u1);
          }
        } else {
#pragma unroll
          for (int k = 0; k < 16; ++k) {
            const int i = 2 * (k >> 3) + (k & 1);          // fragment row
            const int col = 8 * ((k >> 1) & 3) + tc2;
            float u0, u1;
            f2_unpack(pp[k], u0, u1);
            u0 = ex2((uint32_t)(col - loc[i]) < span[i] ? u0 : -INFINITY);
            u1 = ex2((uint32_t)(col + 1 - loc[i]) < span[i] ? u1 : -INFINITY);
            pp[k] = f2_pack(u0, u1);
            pk[k] = pack_bf16x2(u0, u1);
          }
        }
        // pk[8 h + 2 j + e] is (row 16 h + 8 e + t/4, packed column 4 j + t % 4):
        // the 16x128b register order
        tmem_st16x128_x4(s_tm, pk);
        tmem_st16x128_x4(s_tm + (16u << 16), pk + 8);
        tmem_wait_st();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sm.p_ready[rb]);
          mbar_arrive(&sm.slot_empty[sq]);                  // lse read
        }
        // phase 2: dS = P (dP - delta); masked P is zero, so dS is too
        if (!mbar_wait_warp(&sm.slot_full[sd], fp, wc, hdr)) { ok = false; break; }
        if (!mbar_wait_warp(&sm.dp_full, qc & 1, wc, hdr)) { ok = false; break; }
        tc_fence_after();
        tmem_ld16x256_x4(dp_tm, x);
        tmem_ld16x256_x4(dp_tm + (16u << 16), x + 16);
        uint64_t dd[4];                                     // delta column pairs
        {
          const float* src = sm.vec[sd] + cg * 32 + tc2;
#pragma unroll
          for (int j = 0; j < 4; ++j) dd[j] = *reinterpret_cast<const uint64_t*>(src + 8 * j);
        }
        tmem_wait_ld();
        tc_fence_before();
        __syncwarp();
        if (lane == 0) mbar_arrive(&sm.dp_free);
        // the dS^T buffer is free once dK (and the cache copy) have read the previous one
        if (qc >= 1 && !mbar_wait_warp(&sm.dk_done, (qc - 1) & 1, wc, hdr)) { ok = false; break; }
        if (ds_on && qc >= 1 && !mbar_wait_warp(&sm.ds_stored, (qc - 1) & 1, wc, hdr)) {
          ok = false;
          break;
        }
#pragma unroll
        for (int k = 0; k < 16; ++k) {
          const int j = (k >> 1) & 3;
          const int rowoff = 16 * (k >> 3) + 8 * (k & 1);   // key row - (wq 32 + t/4)
          const uint64_t s2 =
              f2_mul(pp[k], f2_sub(f2_pack(__uint_as_float(x[2 * k]), __uint_as_float(x[2 * k + 1])),
                                   dd[j]));
          float a0, a1;
          f2_unpack(s2, a0, a1);
          const int chunk = (cg & 1) * 4 + j;               // 8 query columns per 16 bytes
          st_shared_u32(ds_base + rowoff * 128 + ((chunk ^ tr) << 4), pack_bf16x2(a0, a1));
        }
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
          mbar_arrive(&sm.ds_ready);
          mbar_arrive(&sm.slot_empty[sd]);                  // delta consumed
        }
        ++qc;
      }
      if (!ok) break;
      // item epilogue: warps of column groups 0-1 write dV, 2-3 write dK (64
      // columns each), TMEM lane = key row
      if (!mbar_wait_warp(&sm.dkv_full, items_done & 1, wc, hdr)) break;
      tc_fence_after();
      if (epi_cols) {
        const int64_t key = (int64_t)it.ktile * 128 + r;
        const bool is_dk = cg >= 2;
        const uint32_t col = (is_dk ? 384u : 256u) + (cg & 1) * 64;
        const float scale = is_dk ? p.scale : 1.f;
        // whole-stream accumulators of a batched call: global key rows
        const int64_t key_row = MULTI ? (int64_t)blks.b[it.blk].kv_start + key : key;
        const int64_t off = (key_row * p.Hkv + it.g) * D + (cg & 1) * 64;
        const int64_t keys_here = MULTI ? (int64_t)blks.b[it.blk].kv_len : n_keys;
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t v[32];
          tmem_ld32(tmem + lane_base + col + c * 32, v);
          tmem_wait_ld();
          if (key >= keys_here) continue;
          if (MULTI || (p.accumulate && a.hsplit > 1))     // other items add into the same rows
            red_row32_f32((is_dk ? a.dk_acc : a.dv_acc) + off + c * 32, v, scale);
          else if (p.accumulate)                // the running value was preloaded
            store_row32_f32((is_dk ? a.dk_acc : a.dv_acc) + off + c * 32, v, scale);
          else
            store_row32_bf16((is_dk ? a.dk : a.dv) + off + c * 32, v, scale);
        }
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.dkv_empty);
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

constexpr int K_NS = 3;   // K tiles are read until dQ of their tile is done: one more stage
constexpr int V_NS = 2;

struct QItem {
  int qtile, h, g, j_lo, n_kv;     // n_kv 128-key tiles; -1 stops
  int blk, pad[2];                 // block of a batched call (MULTI)
};

struct __align__(1024) SmemQ {
  uint8_t q[kTile];
  uint8_t dout[kTile];
  uint8_t k[K_NS][kTile];
  uint8_t v[V_NS][kTile];
  uint64_t q_full, q_empty;
  uint64_t k_full[K_NS], k_empty[K_NS], v_full[V_NS], v_empty[V_NS];
  uint64_t s_full[2], p_full[2], dq_done[2];
  uint64_t dp_full, dp_free, o_full, epi_done;
  uint64_t item_full[2], item_empty[2];
  QItem items[2];
  uint64_t drain1, drain2;      // each MMA stream's own barrier for its final drain
  uint32_t tmem_base;
  WaitCtl wait;
};
static_assert(sizeof(SmemQ) <= kSmemLimit, "dQ tile set exceeds shared memory");

// dP = dOut V^T for tile jc (any stream): dP region free once the softmax
// has read the previous dP.
template <int D>
__device__ __forceinline__ bool issue_dp(SmemQ& sm, uint32_t tmem, uint32_t jc,
                                         WaitCtl* wc, WsHeader* hdr) {
  const uint32_t vst = jc % V_NS, vuse = jc / V_NS;
  if (!mbar_wait(&sm.v_full[vst], vuse & 1, wc, hdr)) return false;
  if (jc >= 1 && !mbar_wait(&sm.dp_free, (jc - 1) & 1, wc, hdr)) return false;
  tc_fence_after();
  mma_kk<D>(tmem + 256, smem_u32(sm.dout), smem_u32(sm.v[vst]), false);
  mma_commit(&sm.dp_full);
  mma_commit(&sm.v_empty[vst]);
  return true;
}

template <bool MULTI, int D>
__global__ void __launch_bounds__(kThreads, 1)
    attn_bwd_dq_tc_kernel(const __grid_constant__ CUtensorMap tm_q,
                          const __grid_constant__ CUtensorMap tm_do,
                          const __grid_constant__ CUtensorMap tm_k,
                          const __grid_constant__ CUtensorMap tm_v, const BwdArgs a,
                          const __grid_constant__ FwdBlocks blks) {
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const AttnProblem& p = a.p;
  WsHeader* hdr = p.hdr;
  // Launched behind the dK/dV kernel, which triggers only after its own
  // wait: everything this kernel reads (schedules, delta, -lse log2(e)) is
  // complete.  It reads nothing the dK/dV kernel writes, so it starts on the
  // SMs that kernel frees and waits for it only before it exits (work after
  // this call in the stream then also follows the dK/dV kernel).
  // (with the dS cache in use, the cache's dQ kernel does this call's dQ)
  if (block_leaves(status_bad(hdr) ||
                   (a.ds_cache != nullptr && *((volatile const int32_t*)&hdr->ds_on) != 0))) {
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
    mbar_init(&sm.q_full, 1);
    mbar_init(&sm.q_empty, 2);               // both streams read Q or dOut
    for (int s = 0; s < K_NS; ++s) {
      mbar_init(&sm.k_full[s], 1);
      mbar_init(&sm.k_empty[s], 2);          // S (stream 1) and dQ (stream 2) read K
    }
    for (int s = 0; s < V_NS; ++s) {
      mbar_init(&sm.v_full[s], 1);
      mbar_init(&sm.v_empty[s], 1);          // dP, issued by one of the streams
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sm.s_full[b], 1);
      mbar_init(&sm.p_full[b], 256);
      mbar_init(&sm.dq_done[b], 1);
      mbar_init(&sm.item_full[b], 1);
      mbar_init(&sm.item_empty[b], 2 + 8);
    }
    mbar_init(&sm.dp_full, 1);
    mbar_init(&sm.dp_free, 256);
    mbar_init(&sm.o_full, 1);
    mbar_init(&sm.epi_done, 256);
    mbar_init(&sm.drain1, 1);
    mbar_init(&sm.drain2, 1);
    wait_ctl_init(&sm.wait, p.wait_budget);
    fence_mbar_init();
  }
  if (warp == kWarpMma1) {
    tmem_alloc(&sm.tmem_base, 512);
    tmem_relinquish();
  }
  if (warp == kWarpProducer && lane == 0) {
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
  const int64_t T = p.q_len;
  // a ring block's query tiles that see no key add nothing: not work items
  const int n_items = (p.accumulate ? hdr->n_nonempty : hdr->n_items) * p.Hq;
  constexpr int kBlocks = D / 64;                        // 64-column blocks of a row
  constexpr uint32_t kLoad = kBlocks * kBlk;             // one Q, dOut, K or V tile

  if (warp == kWarpProducer) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      uint32_t it_count = 0, q_count = 0, k_count = 0, v_count = 0;
      bool ok = true;
      while (ok) {
        const int idx = atomicAdd(&hdr->counter, 1);
        QItem it;
        it.qtile = 0; it.h = 0; it.g = 0; it.j_lo = 0; it.n_kv = -1; it.blk = 0;
        if (idx < n_items) {
          const int qt = a.qorder[idx / p.Hq];
          const int2 tr = a.qtiles[qt];
          it.qtile = qt;
          if constexpr (MULTI) {
            it.blk = block_of<false>(blks, qt);
            it.qtile = qt - blks.b[it.blk].tile0;           // query tile within its block
          }
          it.h = idx - (idx / p.Hq) * p.Hq;
          it.g = it.h / G;
          it.j_lo = tr.x;
          it.n_kv = tr.y - tr.x + 1;
        }
        const uint32_t slot = it_count & 1;
        if (it_count >= 2 &&
            !mbar_wait(&sm.item_empty[slot], ((it_count >> 1) - 1) & 1, wc, hdr)) {
          ok = false;
          break;
        }
        sm.items[slot] = it;
        mbar_arrive(&sm.item_full[slot]);
        ++it_count;
        if (it.n_kv <= 0) {
          if (it.n_kv < 0) break;
          continue;
        }
        if (q_count >= 1 && !mbar_wait(&sm.q_empty, (q_count - 1) & 1, wc, hdr)) {
          ok = false;
          break;
        }
        mbar_arrive_expect_tx(&sm.q_full, 2 * kLoad);
        {
          // packed q / dOut: map [q_len, Hq d]; head groups: [P q_len, (Hq/P) d]
          // a batched call's maps span the whole stream (rows = global ids)
          const int hpg = p.Hq / p.q_groups, grp = it.h / hpg;
          const int qx = (it.h - grp * hpg) * D,
                    qy = (MULTI ? blks.b[it.blk].q_start : 0) + (int)(grp * p.q_len) + it.qtile * 128;
#pragma unroll
          for (int cb = 0; cb < kBlocks; ++cb) {
            tma_load_2d(sm.q + cb * kBlk, &tm_q, &sm.q_full, qx + cb * 64, qy);
            tma_load_2d(sm.dout + cb * kBlk, &tm_do, &sm.q_full, qx + cb * 64, qy);
          }
        }
        ++q_count;
        const int k_base = MULTI ? blks.b[it.blk].kv_start : 0;
        for (int jj = 0; jj < it.n_kv; ++jj) {
          const int key0 = k_base + (it.j_lo + jj) * 128;
          {
            const uint32_t st = k_count % K_NS, use = k_count / K_NS;
            if (use >= 1 && !mbar_wait(&sm.k_empty[st], (use - 1) & 1, wc, hdr)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&sm.k_full[st], kLoad);
#pragma unroll
            for (int cb = 0; cb < kBlocks; ++cb)
              tma_load_2d(sm.k[st] + cb * kBlk, &tm_k, &sm.k_full[st], it.g * D + cb * 64, key0);
            ++k_count;
          }
          {
            const uint32_t st = v_count % V_NS, use = v_count / V_NS;
            if (use >= 1 && !mbar_wait(&sm.v_empty[st], (use - 1) & 1, wc, hdr)) {
              ok = false;
              break;
            }
            mbar_arrive_expect_tx(&sm.v_full[st], kLoad);
#pragma unroll
            for (int cb = 0; cb < kBlocks; ++cb)
              tma_load_2d(sm.v[st] + cb * kBlk, &tm_v, &sm.v_full[st], it.g * D + cb * 64, key0);
            ++v_count;
          }
        }
      }
      {
        // leaving, normally or on an abort: every issued copy lands first
        if (q_count >= 1) drain_wait(&sm.q_full, (q_count - 1) & 1);
        for (uint32_t j = (k_count > K_NS ? k_count - K_NS : 0); j < k_count; ++j)
          drain_wait(&sm.k_full[j % K_NS], (j / K_NS) & 1);
        for (uint32_t j = (v_count > V_NS ? v_count - V_NS : 0); j < v_count; ++j)
          drain_wait(&sm.v_full[j % V_NS], (j / V_NS) & 1);
      }
    }
  } else if (warp == kWarpMma1) {
    // ------------------------------------------------------------ stream 1: S, dP of even tiles
    if (lane == 0) {
      const uint32_t q_s = smem_u32(sm.q);
      uint32_t it_count = 0, q_count = 0, jc = 0;
      bool ok = true;
      while (ok) {
        const uint32_t slot = it_count & 1;
        if (!mbar_wait(&sm.item_full[slot], (it_count >> 1) & 1, wc, hdr)) break;
        const QItem it = sm.items[slot];
        mbar_arrive(&sm.item_empty[slot]);
        ++it_count;
        if (it.n_kv < 0) break;
        if (it.n_kv == 0) continue;
        if (!mbar_wait(&sm.q_full, q_count & 1, wc, hdr)) break;
        ++q_count;
        for (int jj = 0; jj < it.n_kv; ++jj) {
          const uint32_t st = jc % K_NS, use = jc / K_NS, b = jc & 1;
          if (!mbar_wait(&sm.k_full[st], use & 1, wc, hdr)) { ok = false; break; }
          // S buffer b is free once dQ has read the dS written over it two tiles ago
          if (jc >= 2 && !mbar_wait(&sm.dq_done[b], ((jc - 2) >> 1) & 1, wc, hdr)) {
            ok = false;
            break;
          }
          tc_fence_after();
          mma_kk<D>(tmem + 128 * b, q_s, smem_u32(sm.k[st]), false);     // S = Q K^T
          mma_commit(&sm.s_full[b]);
          mma_commit(&sm.k_empty[st]);
          if ((jj & 1) == 0 && !issue_dp<D>(sm, tmem, jc, wc, hdr)) { ok = false; break; }
          ++jc;
        }
        if (!ok) break;
        mma_commit(&sm.q_empty);
      }
      mma_drain(&sm.drain1);              // every product done before TMEM is freed
    }
  } else if (warp == kWarpMma2) {
    // ------------------------------------------------------------ stream 2: dP of odd tiles, dQ
    if (lane == 0) {
      uint32_t it_count = 0, items_done = 0, jc = 0;
      bool ok = true;
      while (ok) {
        const uint32_t slot = it_count & 1;
        if (!mbar_wait(&sm.item_full[slot], (it_count >> 1) & 1, wc, hdr)) break;
        const QItem it = sm.items[slot];
        mbar_arrive(&sm.item_empty[slot]);
        ++it_count;
        if (it.n_kv < 0) break;
        if (it.n_kv == 0) continue;
        for (int jj = 0; jj < it.n_kv; ++jj) {
          const uint32_t st = jc % K_NS, b = jc & 1;
          // dP of the next tile when its in-item index is odd: it is due
          // before this tile's dQ (the softmax frees dP mid-tile)
          if (((jj + 1) & 1) == 1 && jj + 1 < it.n_kv &&
              !issue_dp<D>(sm, tmem, jc + 1, wc, hdr)) {
            ok = false;
            break;
          }
          if (!mbar_wait(&sm.p_full[b], (jc >> 1) & 1, wc, hdr)) { ok = false; break; }
          if (jj == 0 && items_done > 0 &&
              !mbar_wait(&sm.epi_done, (items_done - 1) & 1, wc, hdr)) {
            ok = false;
            break;
          }
          tc_fence_after();
          // (a ring block adds onto the preloaded running dQ)
          mma_t_split<64, D>(tmem + 384, tmem + 128 * b, smem_u32(sm.k[st]),
                          jj > 0 || (!MULTI && p.accumulate));                 // dQ += dS K
          mma_commit(&sm.dq_done[b]);
          mma_commit(&sm.k_empty[st]);
          ++jc;
        }
        if (!ok) break;
        mma_commit(&sm.q_empty);
        mma_commit(&sm.o_full);
        ++items_done;
      }
      mma_drain(&sm.drain2);
    }
  } else if (warp < 8) {
    // ------------------------------------------------------------ softmax + dQ epilogue
    const int wg = warp >> 2;                             // key columns 64 wg .. 64 wg + 63
    const bool epi_cols = wg * 64 < D;                    // epilogue: head-dimension columns 64 wg ..
    const int wq = warp & 3;
    const int r = wq * 32 + lane;                          // TMEM lane = query row
    const uint32_t lane_base = (uint32_t)(wq * 32) << 16;
    const float sl2 = p.scale * kLog2e;
    uint32_t it_count = 0, items_done = 0, jc = 0;
    bool ok = true;
    while (ok) {
      const uint32_t slot = it_count & 1;
      if (!mbar_wait_warp(&sm.item_full[slot], (it_count >> 1) & 1, wc, hdr)) break;
      const QItem it = sm.items[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.item_empty[slot]);
      ++it_count;
      if (it.n_kv < 0) break;
      const int h = it.h;
      const int64_t row = (int64_t)it.qtile * 128 + r;      // relative to the (block's) query range
      // the item's ranges: its block's (batched call) or the call's
      const int64_t it_q_start = MULTI ? (int64_t)blks.b[it.blk].q_start : p.q_start;
      const bool valid = row < (MULTI ? (int64_t)blks.b[it.blk].q_len : T);
      int lo = 0, hi = 0;                                    // visible keys [lo, hi)
      float nlse2r = 0.f, deltar = 0.f;
      if (valid) {
        // visible keys, relative to the key range
        const int64_t kvs = MULTI ? (int64_t)blks.b[it.blk].kv_start : p.kv_start;
        const int64_t kve = kvs + (MULTI ? (int64_t)blks.b[it.blk].kv_len : p.kv_len);
        const int64_t tg = it_q_start + row;
        const int b = doc_of(p.cu, p.ndoc, tg);
        const int64_t glo = max((int64_t)__ldg(p.cu + b), kvs);
        const int64_t ghi = min(p.causal ? tg + 1 : (int64_t)__ldg(p.cu + b + 1), kve);
        lo = (int)(glo - kvs);
        hi = (int)max(ghi - kvs, glo - kvs);
        // delta and -lse log2(e): per call, or over the whole stream (batched)
        const int64_t vrow = MULTI ? tg : row;
        nlse2r = __ldg(a.nlse2 + (int64_t)h * a.Tp + vrow);
        deltar = __ldg(a.delta + (int64_t)h * a.Tp + vrow);
      }
      if (!MULTI && p.accumulate && it.n_kv > 0 && epi_cols) {
        // ring block: dQ's TMEM accumulator starts as the running dq / scale
        const float* src = valid ? a.dq_acc + qo_offset(p, row, h) + wg * 64 : nullptr;
        const uint32_t col = tmem + lane_base + 384 + wg * 64;
        preload_row32(col, src, 1.f / p.scale);
        preload_row32(col + 32, src ? src + 32 : nullptr, 1.f / p.scale);
        tmem_wait_st();
      }
      for (int jj = 0; jj < it.n_kv; ++jj) {
        const uint32_t b = jc & 1;
        const uint32_t s_tm = tmem + lane_base + 128 * b + wg * 64;
        const uint32_t dp_tm = tmem + lane_base + 256 + wg * 64;
        if (!mbar_wait_warp(&sm.s_full[b], (jc >> 1) & 1, wc, hdr)) { ok = false; break; }
        tc_fence_after();
        // phase 1: P = exp2(S sl2 - nlse2), masked to the row's visible keys
        uint32_t pf[64];
        tmem_ld32(s_tm, *reinterpret_cast<uint32_t(*)[32]>(pf));
        tmem_ld32(s_tm + 32, *reinterpret_cast<uint32_t(*)[32]>(pf + 32));
        tmem_wait_ld();
        const int key0 = (it.j_lo + jj) * 128 + wg * 64;
        const int aa = lo - key0;
        const uint32_t span = (uint32_t)(hi - lo);
        const bool full_w = __all_sync(0xffffffffu, lo <= key0 && key0 + 64 <= hi);
        if (full_w) {
#pragma unroll
          for (int e = 0; e < 64; ++e)
            pf[e] = __float_as_uint(ex2(fmaf(__uint_as_float(pf[e]), sl2, nlse2r)));
        } else {
#pragma unroll
          for (int e = 0; e < 64; ++e) {
            const bool vis = (uint32_t)(e - aa) < span;
            pf[e] = __float_as_uint(
                ex2(vis ? fmaf(__uint_as_float(pf[e]), sl2, nlse2r) : -INFINITY));
          }
        }
        // phase 2: dS = P (dP - delta) in bf16 over S (masked P is zero)
        if (!mbar_wait_warp(&sm.dp_full, jc & 1, wc, hdr)) { ok = false; break; }
        tc_fence_after();
        uint32_t dp[64];
        tmem_ld32(dp_tm, *reinterpret_cast<uint32_t(*)[32]>(dp));
        tmem_ld32(dp_tm + 32, *reinterpret_cast<uint32_t(*)[32]>(dp + 32));
        tmem_wait_ld();
        tc_fence_before();
        mbar_arrive(&sm.dp_free);
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          uint32_t dk[16];
#pragma unroll
          for (int e = 0; e < 16; ++e) {
            const int i0 = c * 32 + 2 * e;
            dk[e] = pack_bf16x2(__uint_as_float(pf[i0]) * (__uint_as_float(dp[i0]) - deltar),
                                __uint_as_float(pf[i0 + 1]) *
                                    (__uint_as_float(dp[i0 + 1]) - deltar));
          }
          tmem_st16(s_tm + c * 16, dk);       // dS over S (columns already read)
        }
        tmem_wait_st();
        tc_fence_before();
        mbar_arrive(&sm.p_full[b]);
        ++jc;
      }
      if (!ok) break;
      // epilogue: dQ = scale * accumulated dS K, written once in bf16 (my half of d)
      __nv_bfloat16* dst = a.dq + qo_offset(p, row, h) + wg * 64;
      if (it.n_kv > 0) {
        if (!mbar_wait_warp(&sm.o_full, items_done & 1, wc, hdr)) break;
        tc_fence_after();
#pragma unroll
        for (int c = 0; c < 2; ++c) {
          if (!epi_cols) continue;
          uint32_t v[32];
          tmem_ld32(tmem + lane_base + 384 + wg * 64 + c * 32, v);
          tmem_wait_ld();
          if (!valid) continue;
          if (MULTI)                  // other blocks add into the same whole-stream rows
            red_row32_f32(a.dq_acc + ((it_q_start + row) * p.Hq + h) * D + wg * 64 + c * 32, v,
                          p.scale);
          else if (p.accumulate)      // the running value was preloaded
            store_row32_f32(a.dq_acc + qo_offset(p, row, h) + wg * 64 + c * 32, v, p.scale);
          else
            store_row32_bf16(dst + c * 32, v, p.scale);
        }
        tc_fence_before();
        mbar_arrive(&sm.epi_done);
        ++items_done;
      } else if (valid && !p.accumulate && epi_cols) {
        uint32_t z[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) z[i] = 0u;
#pragma unroll
        for (int c = 0; c < 2; ++c) store_row32_bf16(dst + c * 32, z, 0.f);
      }
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kWarpMma1) {
    tc_fence_after();
    tmem_dealloc(tmem, 512);
  }
  grid_dep_wait();
}

// ================================================================ dQ from the dS cache
//
// dQ = scale dS K with dS read back from the cache the dK/dV kernel filled:
// one 128 x 128 x 128 product per visible (query tile, key tile) pair
// instead of three.  Work item: one 128-row query tile of one query head
// (the dQ kernel's items and order); its cached tiles are consecutive
// slots.  Warps 0-3 write dQ (TMEM lane = query row), warp 4 loads (a bulk
// copy of the cached tile, a TMA load of K), one thread of warp 5 issues the
// products into one of two TMEM accumulators (items alternate, so the
// epilogue of one item overlaps the products of the next).  The cached tile
// is dS^T as the dK/dV kernel laid it out ([query block][key][64 queries],
// 128-byte swizzle): for dQ it is the A operand in MN-major form, with the
// same descriptor as K, the MN-major B operand.

constexpr int kCqThreads = 192;
constexpr int kCqWarpProducer = 4, kCqWarpMma = 5;
constexpr int CQ_NS = 3;

struct __align__(1024) SmemCQ {
  uint8_t ds[CQ_NS][kTile];
  uint8_t k[CQ_NS][kTile];
  uint64_t full[CQ_NS], empty[CQ_NS];
  uint64_t acc_full[2], acc_empty[2];
  uint64_t item_full[2], item_empty[2];
  QItem items[2];
  uint64_t drain;
  uint32_t tmem_base;
  WaitCtl wait;
};
static_assert(sizeof(SmemCQ) <= kSmemLimit, "cached-dS tile set exceeds shared memory");

// MULTI: a batched call; its tiles' dQ contributions are added into the
// whole-stream float32 accumulator (global rows) with atomics.
template <bool MULTI, int D>
__global__ void __launch_bounds__(kCqThreads, 1)
    attn_bwd_dq_cached_kernel(const __grid_constant__ CUtensorMap tm_k, const BwdArgs a,
                              const __grid_constant__ FwdBlocks blks) {
  constexpr uint32_t kIdescMM = idesc_bf16_f32(128, D, true, true);   // A, B MN-major, N = D
  constexpr int kBlocks = D / 64;                        // 64-column blocks of a K row
  extern __shared__ __align__(1024) uint8_t smem_raw[];
  const AttnProblem& p = a.p;
  WsHeader* hdr = p.hdr;
  grid_dep_wait();                          // the dK/dV kernel (and its cache copies) are done
  if (block_leaves(status_bad(hdr) || *((volatile const int32_t*)&hdr->ds_on) == 0)) return;
  SmemCQ* smp = smem_view<SmemCQ>(smem_raw, hdr);
  if (smp == nullptr) return;
  SmemCQ& sm = *smp;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;

  if (threadIdx.x == 0) {
    for (int s = 0; s < CQ_NS; ++s) {
      mbar_init(&sm.full[s], 1);
      mbar_init(&sm.empty[s], 1);
    }
    for (int b = 0; b < 2; ++b) {
      mbar_init(&sm.acc_full[b], 1);
      mbar_init(&sm.acc_empty[b], 4);          // one arrival per epilogue warp
      mbar_init(&sm.item_full[b], 1);
      mbar_init(&sm.item_empty[b], 1 + 4);     // MMA thread and the epilogue warps
    }
    mbar_init(&sm.drain, 1);
    wait_ctl_init(&sm.wait, p.wait_budget);
    fence_mbar_init();
  }
  if (warp == kCqWarpMma) {
    tmem_alloc(&sm.tmem_base, 256);
    tmem_relinquish();
  }
  if (warp == kCqWarpProducer && lane == 0) tma_prefetch_desc(&tm_k);
  tc_fence_before();
  __syncthreads();
  tc_fence_after();

  const uint32_t tmem = sm.tmem_base;
  WaitCtl* const wc = &sm.wait;
  const int G = p.Hq / p.Hkv;
  // (a batched call's query tiles that see no key add nothing: not work items)
  const int n_items = (MULTI ? hdr->n_nonempty : hdr->n_items) * p.Hq;
  const int64_t ds_pairs = *((volatile const int64_t*)&hdr->ds_pairs);

  if (warp == kCqWarpProducer) {
    // ------------------------------------------------------------ producer
    if (lane == 0) {
      const uint64_t ds_pol = l2_evict_first_policy();   // each cached tile is read once
      uint32_t it_count = 0, loads = 0;
      bool ok = true;
      while (ok) {
        const int idx = atomicAdd(&hdr->counter, 1);
        QItem it;
        it.qtile = 0; it.h = 0; it.g = 0; it.j_lo = 0; it.n_kv = -1; it.blk = 0;
        int qt = 0;                               // scheduled query tile
        if (idx < n_items) {
          qt = a.qorder[idx / p.Hq];
          const int2 tr = a.qtiles[qt];
          it.qtile = qt;
          if constexpr (MULTI) {
            it.blk = block_of<false>(blks, qt);
            it.qtile = qt - blks.b[it.blk].tile0;           // query tile within its block
          }
          it.h = idx - (idx / p.Hq) * p.Hq;
          it.g = it.h / G;
          it.j_lo = tr.x;
          it.n_kv = tr.y - tr.x + 1;
        }
        const uint32_t slot = it_count & 1;
        if (it_count >= 2 &&
            !mbar_wait(&sm.item_empty[slot], ((it_count >> 1) - 1) & 1, wc, hdr)) {
          ok = false;
          break;
        }
        sm.items[slot] = it;
        mbar_arrive(&sm.item_full[slot]);
        ++it_count;
        if (it.n_kv <= 0) {
          if (it.n_kv < 0) break;
          continue;
        }
        // the item's cached tiles: consecutive slots from qoff[qt]; a batched
        // call's maps span the whole stream (key rows = global ids)
        const uint8_t* src =
            a.ds_cache + ((int64_t)it.h * ds_pairs + a.qoff[qt]) * (int64_t)kTile;
        const int k_base = MULTI ? blks.b[it.blk].kv_start : 0;
        for (int jj = 0; jj < it.n_kv; ++jj) {
          const uint32_t st = loads % CQ_NS, use = loads / CQ_NS;
          if (use >= 1 && !mbar_wait(&sm.empty[st], (use - 1) & 1, wc, hdr)) {
            ok = false;
            break;
          }
          mbar_arrive_expect_tx(&sm.full[st], kTile + kBlocks * kBlk);
          bulk_load(sm.ds[st], src + (int64_t)jj * kTile, kTile, &sm.full[st], ds_pol);
#pragma unroll
          for (int cb = 0; cb < kBlocks; ++cb)
            tma_load_2d(sm.k[st] + cb * kBlk, &tm_k, &sm.full[st], it.g * D + cb * 64,
                        k_base + (it.j_lo + jj) * 128);
          ++loads;
        }
      }
      // leaving, normally or on an abort: every issued copy lands first
      for (uint32_t j = (loads > CQ_NS ? loads - CQ_NS : 0); j < loads; ++j)
        drain_wait(&sm.full[j % CQ_NS], (j / CQ_NS) & 1);
    }
  } else if (warp == kCqWarpMma) {
    // ------------------------------------------------------------ dQ += dS K
    if (lane == 0) {
      uint32_t it_count = 0, items_done = 0, used = 0;
      bool ok = true;
      while (ok) {
        const uint32_t slot = it_count & 1;
        if (!mbar_wait(&sm.item_full[slot], (it_count >> 1) & 1, wc, hdr)) break;
        const QItem it = sm.items[slot];
        mbar_arrive(&sm.item_empty[slot]);
        ++it_count;
        if (it.n_kv < 0) break;
        if (it.n_kv == 0) continue;
        const uint32_t b = items_done & 1;
        // accumulator b is free once the epilogue has read it two items ago
        if (items_done >= 2 &&
            !mbar_wait(&sm.acc_empty[b], ((items_done >> 1) - 1) & 1, wc, hdr))
          break;
        for (int jj = 0; jj < it.n_kv; ++jj) {
          const uint32_t st = used % CQ_NS, use = used / CQ_NS;
          if (!mbar_wait(&sm.full[st], use & 1, wc, hdr)) { ok = false; break; }
          tc_fence_after();
          const uint64_t ad = smem_desc_sw128(smem_u32(sm.ds[st]), kBlk, 1024);
          const uint64_t bd = smem_desc_sw128(smem_u32(sm.k[st]), kBlk, 1024);
#pragma unroll
          for (int kk = 0; kk < 8; ++kk)        // 16 keys per product, 2048 bytes apart
            mma_ss(tmem + 128 * b, ad + ((kk * 2048) >> 4), bd + ((kk * 2048) >> 4), kIdescMM,
                   (jj > 0 || kk > 0) ? 1u : 0u);
          mma_commit(&sm.empty[st]);
          ++used;
        }
        if (!ok) break;
        mma_commit(&sm.acc_full[b]);
        ++items_done;
      }
      mma_drain(&sm.drain);               // every product done before TMEM is freed
    }
  } else if (warp < 4) {
    // ------------------------------------------------------------ dQ epilogue
    const int r = warp * 32 + lane;                        // TMEM lane = query row
    const uint32_t lane_base = (uint32_t)(warp * 32) << 16;
    const int64_t T = p.q_len;
    uint32_t it_count = 0, items_done = 0;
    while (true) {
      const uint32_t slot = it_count & 1;
      if (!mbar_wait_warp(&sm.item_full[slot], (it_count >> 1) & 1, wc, hdr)) break;
      const QItem it = sm.items[slot];
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.item_empty[slot]);
      ++it_count;
      if (it.n_kv < 0) break;
      const int64_t row = (int64_t)it.qtile * 128 + r;   // within the (block's) query range
      const bool valid = row < (MULTI ? (int64_t)blks.b[it.blk].q_len : T);
      __nv_bfloat16* dst = a.dq + qo_offset(p, row, it.h);
      if (it.n_kv == 0) {
        if (MULTI) continue;               // (not listed: see n_items)
        // no visible key (not met in a whole stream): zero rows
        uint32_t z[32];
#pragma unroll
        for (int i = 0; i < 32; ++i) z[i] = 0u;
        if (valid)
#pragma unroll
          for (int c = 0; c < D / 32; ++c) store_row32_bf16(dst + c * 32, z, 0.f);
        continue;
      }
      const uint32_t b = items_done & 1;
      if (!mbar_wait_warp(&sm.acc_full[b], (items_done >> 1) & 1, wc, hdr)) break;
      tc_fence_after();
#pragma unroll
      for (int c = 0; c < D / 32; ++c) {
        uint32_t v[32];
        tmem_ld32(tmem + lane_base + 128 * b + c * 32, v);
        tmem_wait_ld();
        if (!valid) continue;
        if (MULTI)                        // other blocks add into the same whole-stream rows
          red_row32_f32(a.dq_acc + (((int64_t)blks.b[it.blk].q_start + row) * p.Hq + it.h) * D +
                            c * 32,
                        v, p.scale);
        else
          store_row32_bf16(dst + c * 32, v, p.scale);
      }
      tc_fence_before();
      __syncwarp();
      if (lane == 0) mbar_arrive(&sm.acc_empty[b]);
      ++items_done;
    }
  }

  tc_fence_before();
  __syncthreads();
  if (warp == kCqWarpMma) {
    tc_fence_after();
    tmem_dealloc(tmem, 256);
  }
}

// ================================================================ host

PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
  static PFN_cuTensorMapEncodeTiled_v12000 fn = nullptr;
  static bool tried = false;
  if (!tried) {
    tried = true;
    void* ptr = nullptr;
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &ptr, 12000, cudaEnableDefault,
                                         &q) == cudaSuccess &&
        q == cudaDriverEntryPointSuccess)
      fn = reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(ptr);
  }
  return fn;
}

// [rows, cols] bf16 row-major; box = 64 columns x 128 rows, 128-byte swizzle.
bool make_map(CUtensorMap* m, const void* base, int64_t rows, int64_t cols) {
  auto fn = encode_fn();
  if (!fn) return false;
  cuuint64_t dims[2] = {(cuuint64_t)cols, (cuuint64_t)rows};
  cuuint64_t strides[1] = {(cuuint64_t)(cols * 2)};
  cuuint32_t box[2] = {64, 128};
  cuuint32_t estr[2] = {1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 2, const_cast<void*>(base), dims, strides, box,
            estr, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B,
            CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The three kernels of one head dimension D (dK/dV, dQ, dQ from the cache).
template <int D>
cudaError_t launch_kernels_d(const BwdArgs& a, const FwdBlocks* blocks, bool cache,
                             const CUtensorMap& mq, const CUtensorMap& mdo, const CUtensorMap& mk,
                             const CUtensorMap& mv, cudaStream_t s) {
  const int grid = persistent_grid();
  constexpr size_t kv_bytes = smem_bytes<SmemKV>();
  constexpr size_t q_bytes = smem_bytes<SmemQ>();
  const FwdBlocks B = blocks ? *blocks : single_block(a.p);
  auto kv_kern = blocks ? attn_bwd_dkdv_tc_kernel<true, D> : attn_bwd_dkdv_tc_kernel<false, D>;
  auto q_kern = blocks ? attn_bwd_dq_tc_kernel<true, D> : attn_bwd_dq_tc_kernel<false, D>;
  cudaError_t e =
      cudaFuncSetAttribute(kv_kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kv_bytes);
  if (e != cudaSuccess) return e;
  e = cudaFuncSetAttribute(q_kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)q_bytes);
  if (e != cudaSuccess) return e;
  e = launch_dependent(kv_kern, dim3(grid), dim3(kKvThreads), kv_bytes, s, mq, mdo, mk, mv, a, B);
  count_launches(1);
  count_path(true);
  if (e != cudaSuccess) return e;
  e = launch_dependent(q_kern, dim3(grid), dim3(kThreads), q_bytes, s, mq, mdo, mk, mv, a, B);
  count_launches(1);
  count_path(true);
  if (e != cudaSuccess) return e;
  if (cache) {
    // exactly one of the two dQ kernels does the work (header flag ds_on)
    constexpr size_t cq_bytes = smem_bytes<SmemCQ>();
    auto cq_kern = blocks ? attn_bwd_dq_cached_kernel<true, D> : attn_bwd_dq_cached_kernel<false, D>;
    e = cudaFuncSetAttribute(cq_kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)cq_bytes);
    if (e != cudaSuccess) return e;
    e = launch_dependent(cq_kern, dim3(grid), dim3(kCqThreads), cq_bytes, s, mk, a, B);
    count_launches(1);
    count_path(true);
    if (e != cudaSuccess) return e;
  }
  return cudaGetLastError();
}

}  // namespace

bool bwd_tc_eligible(int32_t io_dtype, int32_t d, int32_t Hq, int32_t Hkv) {
  return io_dtype == NSP_BF16 && (d == 128 || d == 64) && Hkv > 0 && Hq % Hkv == 0;
}

cudaError_t launch_attn_bwd_tc(const AttnProblem& p, const void* out, const void* dout,
                               const float* lse, void* dq, void* dk, void* dv,
                               const BwdWsLayout& L, char* ws, cudaStream_t s,
                               const FwdBlocks* blocks) {
  const int64_t T = p.q_len;
  CUtensorMap mq, mdo, mk, mv;
  const int64_t qc = (int64_t)p.Hq * p.d, kc = (int64_t)p.Hkv * p.d;
  const int64_t qrows = T * p.q_groups, qcols = qc / p.q_groups;   // grouped: [P T, (Hq/P) d]
  if (!make_map(&mq, p.q, qrows, qcols) || !make_map(&mdo, dout, qrows, qcols) ||
      !make_map(&mk, p.k, p.kv_len, kc) || !make_map(&mv, p.v, p.kv_len, kc))
    return cudaErrorNotSupported;
  float* delta = reinterpret_cast<float*>(ws + L.delta);
  float* nlse2 = reinterpret_cast<float*>(ws + L.nlse2);
  cudaError_t e = launch_bwd_delta(out, dout, lse, delta, nlse2, T, L.Tp, p.Hq, p.d, p.io_dtype,
                                   p.q_groups, p.hdr, s);
  if (e != cudaSuccess) return e;
  BwdArgs a;
  a.p = p;
  a.p.wait_budget = wait_budget_cycles();
  a.nlse2 = nlse2;
  a.delta = delta;
  a.Tp = L.Tp;
  a.dq = reinterpret_cast<__nv_bfloat16*>(dq);
  a.dk = reinterpret_cast<__nv_bfloat16*>(dk);
  a.dv = reinterpret_cast<__nv_bfloat16*>(dv);
  a.dq_acc = reinterpret_cast<float*>(dq);
  a.dk_acc = reinterpret_cast<float*>(dk);
  a.dv_acc = reinterpret_cast<float*>(dv);
  a.qtiles = reinterpret_cast<const int2*>(ws + L.qtiles);
  a.qorder = reinterpret_cast<const int*>(ws + L.qorder);
  a.ktiles = reinterpret_cast<const int2*>(ws + L.ktiles);
  a.korder = reinterpret_cast<const int*>(ws + L.korder);
  // dS cache: whole-stream and batched calls given workspace past the layout
  // (the schedule decides whether every visible pair's dS fits)
  const bool cache = (blocks != nullptr || !p.accumulate) && L.ds_cache_bytes > 0;
  a.ds_cache = cache ? reinterpret_cast<uint8_t*>(ws + L.ds_cache) : nullptr;
  a.qoff = reinterpret_cast<const int64_t*>(ws + L.qoff);
  const int grid = persistent_grid();
  // A ring block has few key tiles: split each (key tile, KV head) item over
  // query-head subsets until there are two items per SM (the subsets add
  // into the float32 accumulators with atomics).  The whole-stream backward
  // writes each dK/dV row once (hsplit = 1).
  const int G = p.Hq / p.Hkv;
  a.hsplit = 1;
  if (p.accumulate || blocks != nullptr)
    while (a.hsplit < G && G % (2 * a.hsplit) == 0 &&
           L.n_ktiles * p.Hkv * a.hsplit < 2 * (int64_t)grid)
      a.hsplit *= 2;
  return p.d == 128 ? launch_kernels_d<128>(a, blocks, cache, mq, mdo, mk, mv, s)
                    : launch_kernels_d<64>(a, blocks, cache, mq, mdo, mk, mv, s);
}

}  // namespace nsp
