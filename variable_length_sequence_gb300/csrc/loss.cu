// Losses of a packed stream over the log-probabilities of its scored rows (those
// with a target): the clipped policy loss and the preference loss over pairs of
// documents, each with its gradient.
//
// A few bytes a row: bound by launches and the latency of dependent loads.  One block
// counts the scored rows (32 rows a word, a running count a word, so that any document's
// count is two lookups) and writes the documents' weights: 6 us of 8192 rows.  A pair of
// documents is one block: both sums, the loss in float64 by one thread, the gradient over
// the rows: 10 us of 4099 rows.
#include <algorithm>

#include "policy.cuh"
#include "sums.cuh"

namespace nsp {
namespace {

constexpr int kPrepThreads = 1024;
constexpr int kThreads = 256;
constexpr int kPolicyBlocks = 304;

// Scored rows before row x.
__device__ __forceinline__ int scored_before(const LossArgs& a, int64_t x) {
  x = min(x, a.rows);
  const int64_t w = x >> 5;
  int n = w > 0 ? a.before[w - 1] : 0;               // (before[w]: up to the end of word w)
  if ((x & 31) != 0) n += __popc(a.bits[w] & ((1u << (x & 31)) - 1));
  return n;
}

// Walks the rows of a stream in a block's order: which are scored (below `end`, with a
// target), how many up to the end of each 32 (bits, before), and the list of both kinds
// (RowArgs::list); what is null is not wanted.  Returns the number of scored rows.
struct RowScan {
  int warp_sum[32];
  int base;
};
__device__ __forceinline__ int scan_rows(const int32_t* __restrict__ targets, int64_t rows, int64_t end,
                                         uint32_t* bits, int32_t* before, int2* list, float* logp,
                                         float* lse, RowScan& sh) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int64_t words = (rows + 31) >> 5;
  const int per = (int)min((int64_t)32, (words + 31) >> 5);    // words of a warp and turn
  if (tid == 0) sh.base = 0;
  for (int64_t w0 = 0; w0 < words; w0 += 32 * per) {
    const int64_t first = w0 + warp * per;
    uint32_t mine = 0;                                         // lane i keeps word i
#pragma unroll 8
    for (int i = 0; i < per; ++i) {
      const int64_t t = (first + i) * 32 + lane;
      const uint32_t b = __ballot_sync(0xffffffffu, t < end && __ldg(targets + t) >= 0);
      if (lane == i) mine = b;
    }
    int n = __popc(mine);
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int v = __shfl_up_sync(0xffffffffu, n, o);
      if (lane >= o) n += v;
    }
    if (lane == 31) sh.warp_sum[warp] = n;
    __syncthreads();
    const int others = sh.warp_sum[lane];
    n += sh.base + __reduce_add_sync(0xffffffffu, lane < warp ? others : 0);
    if (lane < per && first + lane < words && bits != nullptr) {
      bits[first + lane] = mine;
      before[first + lane] = n;
    }
    if (list != nullptr) {
#pragma unroll 4
      for (int i = 0; i < per; ++i) {
        const uint32_t b = __shfl_sync(0xffffffffu, mine, i);
        const int start = __shfl_sync(0xffffffffu, n, i) - __popc(b);
        const int64_t t = (first + i) * 32 + lane;
        const int k = start + __popc(b & ((1u << lane) - 1));  // scored rows before t
        if (t >= rows) continue;
        if (b >> lane & 1) {
          list[k] = make_int2((int)t, __ldg(targets + t));
        } else {
          list[rows - 1 - (t - k)] = make_int2((int)t, -1);
          if (logp) logp[t] = 0.f;
          if (lse) lse[t] = 0.f;
        }
      }
    }
    const int turn = __reduce_add_sync(0xffffffffu, others);
    __syncthreads();
    if (tid == 0) sh.base += turn;
    __syncthreads();
  }
  __syncthreads();
  return sh.base;
}

__global__ void __launch_bounds__(kPrepThreads) row_list_kernel(const __grid_constant__ RowArgs a) {
  __shared__ RowScan sh;
  grid_dep_trigger();
  const int n = scan_rows(a.targets, a.rows, a.rows, nullptr, nullptr, a.list, a.logp, a.lse, sh);
  if (threadIdx.x == 0) a.hdr->n_items = n;
}

__global__ void __launch_bounds__(kPrepThreads) loss_prep_kernel(const LossArgs a) {
  __shared__ RowScan sh;
  __shared__ int s_bad, s_docs;
  const int tid = threadIdx.x;
  grid_dep_trigger();
  if (tid == 0) s_bad = a.cu[0] != 0, s_docs = 0;
  __syncthreads();
  for (int i = tid; i < a.ndoc; i += kPrepThreads)
    if (a.cu[i] > a.cu[i + 1]) s_bad = 1;
  __syncthreads();
  if (tid == 0) a.hdr->status = s_bad ? NSP_ERR_INVALID : NSP_OK;
  if (s_bad) return;
  const int scored = scan_rows(a.targets, a.rows, min((int64_t)a.cu[a.ndoc], a.rows), a.bits, a.before,
                               a.list, nullptr, nullptr, sh);
  if (tid == 0) a.hdr->n_items = scored;
  __syncthreads();
  int docs = 0;
  for (int i = tid; i < a.ndoc; i += kPrepThreads) {
    const int n = scored_before(a, a.cu[i + 1]) - scored_before(a, a.cu[i]);
    a.weight[i] = (float)n;
    docs += n > 0;
  }
  atomicAdd(&s_docs, docs);
  __syncthreads();
  const float tokens = a.total > 0.f ? a.total : (float)scored;
  const float many = a.total > 0.f ? a.total : (float)s_docs;
  for (int i = tid; i < a.ndoc; i += kPrepThreads) {
    const float n = a.weight[i];
    a.weight[i] = n == 0.f ? 0.f : a.mean == NSP_MEAN_TOKENS ? 1.f / tokens : 1.f / (many * n);
  }
}

// Weight and advantage of every scored row, for a kernel that has no time for a search a
// row; zeros of the others.
__global__ void __launch_bounds__(kThreads) loss_rows_kernel(const __grid_constant__ RowArgs a) {
  grid_dep_wait();
  if (status_bad(a.p.hdr)) return;
  const int64_t t = (int64_t)blockIdx.x * kThreads + threadIdx.x;
  if (t >= a.rows) return;
  if (t >= (int64_t)__ldg(a.p.cu + a.p.ndoc) || __ldg(a.targets + t) < 0) {
    if (a.logp) a.logp[t] = 0.f;
    for (int i = 0; i < 3; ++i) a.p.terms[i * a.rows + t] = 0.f;
    return;
  }
  const int doc = doc_of(a.p.cu, a.p.ndoc, t);
  a.p.row_scalars[t] = make_float2(__ldcg(a.p.doc_weight + doc),
                                   __ldg(a.p.advantages + (a.p.per_token ? t : (int64_t)doc)));
}

// stats from sums of surrogate, kl and clipped.
__device__ __forceinline__ void write_stats(float* stats, float kl_coef, double pg, double kl, double cut) {
  stats[0] = (float)(pg + (double)kl_coef * kl);
  stats[1] = (float)pg;
  stats[2] = (float)kl;
  stats[3] = (float)cut;
}

__global__ void __launch_bounds__(kThreads) policy_kernel(const __grid_constant__ PolicyArgs a) {
  __shared__ Sum2 s_sum[3][kThreads / 32];
  grid_dep_trigger();
  grid_dep_wait();
  if (status_bad(a.p.hdr)) return;
  const int64_t end = min((int64_t)__ldg(a.p.cu + a.p.ndoc), a.rows);
  Sum2 pg = {0.f, 0.f}, kl = pg, cut = pg;
  for (int64_t t = (int64_t)blockIdx.x * kThreads + threadIdx.x; t < a.rows;
       t += (int64_t)gridDim.x * kThreads) {
    float g = 0.f;
    if (t < end && __ldg(a.targets + t) >= 0) {
      const PolicyScalars v = policy_scalars(a.p, t, doc_of(a.p.cu, a.p.ndoc, t));
      const PolicyRow r = policy_row(a.p, v, __ldg(a.logp + t));
      pg.add(r.surrogate);
      kl.add(r.kl);
      cut.add(r.clipped);
      g = r.grad;
    }
    a.dlogp[t] = g;
  }
  constexpr int W = kThreads / 32;
  pg = block_sum<W>(pg, s_sum[0]);
  kl = block_sum<W>(kl, s_sum[1]);
  cut = block_sum<W>(cut, s_sum[2]);
  if (threadIdx.x == 0) {
    float* const o = a.p.terms + blockIdx.x;
    o[0] = (float)pg.value();
    o[gridDim.x] = (float)kl.value();
    o[2 * gridDim.x] = (float)cut.value();
  }
}

// stats from n terms of each of the three.
__global__ void __launch_bounds__(kPrepThreads) policy_stats_kernel(const float* __restrict__ terms,
                                                                    int64_t n, float kl_coef,
                                                                    const WsHeader* hdr, float* stats) {
  __shared__ Sum2 s_sum[3][kPrepThreads / 32];
  grid_dep_wait();
  if (status_bad(hdr)) return;
  Sum2 sum[3] = {};
#pragma unroll 4
  for (int64_t t = threadIdx.x; t < n; t += kPrepThreads)
    for (int i = 0; i < 3; ++i) sum[i].add(__ldcg(terms + i * n + t));
  for (int i = 0; i < 3; ++i) sum[i] = block_sum<kPrepThreads / 32>(sum[i], s_sum[i]);
  if (threadIdx.x == 0) write_stats(stats, kl_coef, sum[0].value(), sum[1].value(), sum[2].value());
}

// One pair of documents a block: both sums, the pair's loss, and its gradient over the
// documents' rows; the blocks together clear the rows behind the last document.
constexpr int kPairThreads = 512, kPairWarps = kPairThreads / 32;
__global__ void __launch_bounds__(kPairThreads) preference_kernel(const __grid_constant__ PreferenceArgs a) {
  __shared__ Sum2 s_sum[2][kPairWarps];
  __shared__ int s_count[2][kPairWarps];
  __shared__ float s_grad[2];
  const int pairs = a.ndoc / 2, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  grid_dep_trigger();
  for (int i = blockIdx.x; i < pairs; i += gridDim.x) {
    const int64_t at[3] = {__ldg(a.cu + 2 * i), __ldg(a.cu + 2 * i + 1), __ldg(a.cu + 2 * i + 2)};
    const bool bad = at[0] > at[1] || at[1] > at[2] || at[0] < 0 || (i == 0 && at[0] != 0);
    if (threadIdx.x == 0) a.terms[2 * (int64_t)pairs + i] = bad ? 1.f : 0.f;
    if (bad) continue;
    __syncthreads();                   // (the last pair's sums and gradients have been read)
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int64_t hi = min(at[k + 1], a.rows);
      Sum2 x = {0.f, 0.f};
      int n = 0;
      // (loaded whether scored or not, so that the loads do not wait for one another)
#pragma unroll 4
      for (int64_t t = at[k] + threadIdx.x; t < hi; t += kPairThreads) {
        const int y = __ldg(a.targets + t);
        const float l = __ldg(a.logp + t), r = a.ref_logp ? __ldg(a.ref_logp + t) : 0.f;
        x.add(y >= 0 ? l : 0.f);
        x.add(y >= 0 ? -r : 0.f);
        n += y >= 0;
      }
      n = __reduce_add_sync(0xffffffffu, n);
      x = warp_sum(x);
      if (lane == 0) {
        s_count[k][warp] = n;
        s_sum[k][warp] = x;
      }
    }
    __syncthreads();
    if (warp == 0) {
      double score[2];
      int count[2];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        Sum2 x = {0.f, 0.f};
        if (lane < kPairWarps) x = s_sum[k][lane];
        score[k] = warp_sum(x).value();
        count[k] = max(1, __reduce_add_sync(0xffffffffu, lane < kPairWarps ? s_count[k][lane] : 0));
        if (a.average) score[k] /= count[k];
      }
      // (one thread: float64 units are few)
      if (lane == 0) {
        const double beta = a.beta, h = beta * (score[0] - score[1]) - a.margin;
        double loss, dh;
        if (a.kind == NSP_PREFERENCE_SIGMOID) {
          const double e = exp(-fabs(h)), low = log1p(e);          // log(1 + exp(-|h|))
          const double down = low + fmax(-h, 0.0), up = low + fmax(h, 0.0);   // -log sigmoid(+-h)
          loss = (1.0 - a.smoothing) * down + a.smoothing * up;
          dh = a.smoothing - (h > 0 ? e : 1.0) / (1.0 + e);        // smoothing - sigmoid(-h)
        } else if (a.kind == NSP_PREFERENCE_HINGE) {
          loss = h < 1.0 ? 1.0 - h : (h >= 1.0 ? 0.0 : h);         // (NaN stays)
          dh = h < 1.0 ? -1.0 : (h >= 1.0 ? 0.0 : h);
        } else {
          const double off = h / beta - 0.5 / beta;
          loss = off * off;
          dh = 2.0 * off / beta;
        }
        a.terms[i] = (float)loss;
        a.terms[pairs + i] = score[0] > score[1] ? 1.f : 0.f;
        a.rewards[2 * (int64_t)i] = (float)(beta * score[0]);
        a.rewards[2 * (int64_t)i + 1] = (float)(beta * score[1]);
        for (int k = 0; k < 2; ++k)
          s_grad[k] = (float)((k ? -dh : dh) * beta / pairs / (a.average ? count[k] : 1));
      }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const int64_t hi = min(at[k + 1], a.rows);
      const float g = s_grad[k];
#pragma unroll 4
      for (int64_t t = at[k] + threadIdx.x; t < hi; t += kPairThreads)
        a.dlogp[t] = __ldg(a.targets + t) >= 0 ? g : 0.f;
    }
  }
  for (int64_t t = max((int64_t)0, (int64_t)__ldg(a.cu + a.ndoc)) + (int64_t)blockIdx.x * kPairThreads + threadIdx.x;
       t < a.rows; t += (int64_t)gridDim.x * kPairThreads)
    a.dlogp[t] = 0.f;
}

__global__ void __launch_bounds__(kPrepThreads) preference_stats_kernel(const float* __restrict__ terms,
                                                                        int pairs, WsHeader* hdr,
                                                                        float* stats) {
  __shared__ Sum2 s_sum[3][kPrepThreads / 32];
  grid_dep_wait();
  Sum2 sum[3] = {};
#pragma unroll 2
  for (int t = threadIdx.x; t < pairs; t += kPrepThreads)
    for (int i = 0; i < 3; ++i) sum[i].add(__ldcg(terms + (int64_t)i * pairs + t));
  for (int i = 0; i < 3; ++i) sum[i] = block_sum<kPrepThreads / 32>(sum[i], s_sum[i]);
  if (threadIdx.x != 0) return;
  hdr->status = sum[2].hi != 0.f ? NSP_ERR_INVALID : NSP_OK;
  stats[0] = (float)(sum[0].value() / pairs);
  stats[1] = (float)(sum[1].value() / pairs);
}

}  // namespace

LossWsLayout loss_ws_layout(int64_t rows, int32_t ndoc, bool logits) {
  LossWsLayout L;
  const size_t words = (size_t)ceil_div(rows, 32);
  L.before = sizeof(WsHeader);
  L.bits = align_up(L.before + 4 * words, 256);
  L.weight = align_up(L.bits + 4 * words, 256);
  L.terms = align_up(L.weight + 4 * (size_t)ndoc, 256);
  L.scalars = align_up(L.terms + 12 * (logits ? (size_t)rows : (size_t)kPolicyBlocks), 256);
  L.list = align_up(L.scalars + (logits ? 8 * (size_t)rows : 0), 256);
  L.total = align_up(L.list + (logits ? 8 * (size_t)rows : 0), 256);
  return L;
}

cudaError_t launch_loss_prep(const LossArgs& a, cudaStream_t s) {
  loss_prep_kernel<<<1, kPrepThreads, 0, s>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_row_list(const RowArgs& a, cudaStream_t s) {
  row_list_kernel<<<1, kPrepThreads, 0, s>>>(a);
  count_launches(1);
  return cudaGetLastError();
}

cudaError_t launch_loss_rows(const RowArgs& a, cudaStream_t s) {
  count_launches(1);
  return launch_dependent(loss_rows_kernel, dim3((unsigned)ceil_div(a.rows, kThreads)), dim3(kThreads), 0, s, a);
}

static int policy_blocks(int64_t rows) {
  return (int)std::max<int64_t>(1, std::min<int64_t>(kPolicyBlocks, ceil_div(rows, kThreads)));
}

cudaError_t launch_policy(const PolicyArgs& a, cudaStream_t s) {
  const int blocks = policy_blocks(a.rows);
  count_launches(2);
  const cudaError_t e = launch_dependent(policy_kernel, dim3(blocks), dim3(kThreads), 0, s, a);
  if (e != cudaSuccess) return e;
  return launch_dependent(policy_stats_kernel, dim3(1), dim3(kPrepThreads), 0, s,
                          (const float*)a.p.terms, (int64_t)blocks, a.p.kl_coef, a.p.hdr, a.stats);
}

cudaError_t launch_policy_stats(const RowArgs& a, float* stats, cudaStream_t s) {
  count_launches(1);
  return launch_dependent(policy_stats_kernel, dim3(1), dim3(kPrepThreads), 0, s,
                          (const float*)a.p.terms, a.rows, a.p.kl_coef, a.p.hdr, stats);
}

cudaError_t launch_preference(const PreferenceArgs& a, cudaStream_t s) {
  const int pairs = a.ndoc / 2;
  const int blocks = (int)std::min<int64_t>(pairs, (int64_t)num_sms() * 4);
  preference_kernel<<<blocks, kPairThreads, 0, s>>>(a);
  count_launches(1);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  e = launch_dependent(preference_stats_kernel, dim3(1), dim3(kPrepThreads), 0, s,
                       (const float*)a.terms, pairs, a.hdr, a.stats);
  count_launches(1);
  return e;
}

}  // namespace nsp
