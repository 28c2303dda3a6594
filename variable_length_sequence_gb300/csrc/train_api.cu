// C ABI entry points of the operators of a packed post-training step: host
// validation, workspace carving and dispatch.  Nothing here allocates memory
// or synchronises.
#include <algorithm>
#include <cmath>

#include "checks.cuh"
#include "train.cuh"

using namespace nsp;

namespace {

Span strided(const void* p, int64_t rows, int64_t step, int64_t row) {
  return {reinterpret_cast<uintptr_t>(p), p ? rows : 0, step, row};
}

// The checks that both directions share, and their arguments.
int32_t qk_check(const nsp_qk_tensor_t* tensors, int32_t n, const int32_t* cu, int32_t ndoc,
                 const int32_t* positions, int64_t start, int64_t len, int32_t d, int32_t rot,
                 const double* freqs, int32_t interleaved, float mscale, float eps, int32_t io_dtype,
                 bool back, const void* workspace, size_t workspace_bytes, QkArgs& a) {
  if (!tensors || n < 1 || n > kRopeMaxTensors || !dtype_ok(io_dtype)) return NSP_ERR_INVALID;
  if (d < 2 || rot < 2 || rot % 2 != 0 || rot > d) return NSP_ERR_INVALID;
  if (d > kQkMaxDim) return NSP_ERR_UNSUPPORTED;
  if (interleaved != 0 && interleaved != 1) return NSP_ERR_INVALID;
  if (!std::isfinite(mscale) || !(eps > 0.f) || !std::isfinite(eps)) return NSP_ERR_INVALID;
  if (start < 0 || len < 0) return NSP_ERR_INVALID;
  if (len > kMaxTokens || start > kMaxTokens - len) return NSP_ERR_UNSUPPORTED;
  if (!freqs || (!positions && (!cu || ndoc < 1))) return NSP_ERR_INVALID;
  if (!aligned(freqs, 8) || !aligned(positions, 4) || !aligned(cu, 4)) return NSP_ERR_ALIGN;
  const int64_t es = elem_bytes(io_dtype);
  Span in[kRopeMaxTensors][3], out[2 * kRopeMaxTensors];   // x, dy, weight; y or dx, dweight
  a = {};
  for (int32_t i = 0; i < n; ++i) {
    const nsp_qk_tensor_t& t = tensors[i];
    if (t.heads < 1 || t.groups < 1 || t.heads % t.groups != 0) return NSP_ERR_INVALID;
    if (t.heads > kMaxHeads) return NSP_ERR_UNSUPPORTED;
    if (len > 0 && (!t.x || (back ? !t.dy || !t.dx : !t.y))) return NSP_ERR_INVALID;
    if (back && t.dweight && !t.weight) return NSP_ERR_INVALID;
    const void* ptrs[] = {t.x, t.weight, back ? t.dy : t.y, back ? t.dx : nullptr,
                          back ? t.dweight : nullptr};
    for (const void* p : ptrs)
      if (!aligned(p, es)) return NSP_ERR_ALIGN;
    const int64_t width = (int64_t)t.heads * d;
    const int64_t xs = t.x_stride == 0 ? width : t.x_stride;
    const int64_t ys = t.y_stride == 0 ? width : t.y_stride;
    const int64_t ds = !back || t.dx_stride == 0 ? width : t.dx_stride;
    for (const int64_t stride : {xs, ys, ds}) {
      if (stride < width) return NSP_ERR_INVALID;
      if (stride > ((int64_t)1 << 31)) return NSP_ERR_UNSUPPORTED;
    }
    if (t.groups > 1 && ys != width) return NSP_ERR_INVALID;   // the head-group-major side is packed
    a.t[i] = {t.x, t.weight, back ? t.dy : nullptr, back ? nullptr : t.y, back ? t.dx : nullptr,
              back ? t.dweight : nullptr, xs, ys, ds, t.heads, t.groups};
    in[i][0] = strided(t.x, len, xs * es, width * es);
    in[i][1] = back ? strided(t.dy, len, ys * es, width * es) : Span{0, 0, 1, 1};
    in[i][2] = packed(t.weight, 1, d * es);
    out[2 * i] = back ? strided(t.dx, len, ds * es, width * es) : strided(t.y, len, ys * es, width * es);
    out[2 * i + 1] = packed(a.t[i].dweight, 1, d * es);
  }
  if (back) {
    // (before the overlaps: they are checked over the workspace's own size)
    const size_t need = nsp_qk_norm_rope_bwd_workspace_size(tensors, n, len, d);
    if (!workspace || workspace_bytes < need) return NSP_ERR_WORKSPACE;
    if (!aligned(workspace, 16)) return NSP_ERR_ALIGN;
  }
  const Span ws = packed(
      workspace, 1, back ? (int64_t)nsp_qk_norm_rope_bwd_workspace_size(tensors, n, len, d) : 0);
  const Span read[] = {packed(positions, 1, len * 4), packed(freqs, 1, rot / 2 * 8),
                       packed(positions ? nullptr : cu, 1, ((int64_t)ndoc + 1) * 4)};
  for (int32_t j = 0; j < 2 * n; ++j) {
    const Span& o = out[j];
    for (int32_t i = 0; i < n; ++i)
      for (int32_t m = 0; m < 3; ++m) {
        // y may take its x's place, dx its x's or its dy's: a row is read whole before it is
        // written (not regrouped)
        const bool in_place = j == 2 * i && m < 2 && same_rows(o, in[i][m]) &&
                              (tensors[i].groups == 1 || (back && m == 0));
        if (!in_place && overlap(o, in[i][m])) return NSP_ERR_INVALID;
      }
    for (const Span& r : read)
      if (overlap(o, r)) return NSP_ERR_INVALID;
    for (int32_t i = 0; i < j; ++i)
      if (overlap(o, out[i])) return NSP_ERR_INVALID;
    if (overlap(o, ws)) return NSP_ERR_INVALID;
  }
  for (int32_t i = 0; i < n; ++i)
    for (const Span& r : in[i])
      if (overlap(ws, r)) return NSP_ERR_INVALID;
  for (const Span& r : read)
    if (overlap(ws, r)) return NSP_ERR_INVALID;
  a.n = n;
  a.cu = cu; a.ndoc = ndoc; a.positions = positions;
  a.start = start; a.len = len; a.d = d; a.rot = rot;
  a.interleaved = interleaved;
  a.freqs = freqs; a.mscale = mscale; a.eps = eps;
  a.partial = reinterpret_cast<float*>(const_cast<void*>(workspace));
  return NSP_OK;
}

// Rows of logits and of their gradient.
int32_t rows_check(const void* logits, int64_t row_stride, const int32_t* targets, int64_t rows,
                   int32_t vocab, double scale, int32_t io_dtype, RowArgs& a) {
  // (what a float holds of it without loss of precision)
  if (!dtype_ok(io_dtype) || rows < 0 || vocab < 1 || !(scale >= 1e-30) || !(scale <= 1e30)) return NSP_ERR_INVALID;
  if (rows > kMaxTokens || vocab > kMaxVocab) return NSP_ERR_UNSUPPORTED;
  if (row_stride == 0) row_stride = vocab;
  if (row_stride < vocab) return NSP_ERR_INVALID;
  if (row_stride > ((int64_t)1 << 31)) return NSP_ERR_UNSUPPORTED;
  if (rows > 0 && (!logits || !targets)) return NSP_ERR_INVALID;
  if (!aligned(logits, elem_bytes(io_dtype)) || !aligned(targets, 4)) return NSP_ERR_ALIGN;
  a = {};
  a.logits = logits; a.row_stride = row_stride; a.targets = targets;
  a.rows = rows; a.vocab = vocab; a.scale = (float)scale;
  const double c = scale * 1.44269504088896340736;
  // (a remainder above zero: it meets logits of minus infinity)
  a.c = (float)c;
  while ((double)a.c >= c) a.c = std::nextafterf(a.c, 0.f);
  a.c_lo = (float)(c - (double)a.c);
  return NSP_OK;
}

int32_t gradient_check(void* dlogits, int64_t out_stride, int32_t io_dtype, RowArgs& a) {
  if (out_stride == 0) out_stride = a.vocab;
  if (out_stride < a.vocab || (a.rows > 0 && !dlogits)) return NSP_ERR_INVALID;
  if (out_stride > ((int64_t)1 << 31)) return NSP_ERR_UNSUPPORTED;
  if (!aligned(dlogits, elem_bytes(io_dtype))) return NSP_ERR_ALIGN;
  a.dlogits = dlogits;
  a.out_stride = out_stride;
  return NSP_OK;
}

Span logits_span(const RowArgs& a, int64_t es) {
  return strided(a.logits, a.rows, a.row_stride * es, a.vocab * es);
}
Span gradient_span(const RowArgs& a, int64_t es) {
  return strided(a.dlogits, a.rows, a.out_stride * es, a.vocab * es);
}

// Whether any of the outputs shares a byte with an input or another output.
bool clash(const Span* outs, int n_out, const Span* ins, int n_in) {
  for (int i = 0; i < n_out; ++i) {
    for (int j = 0; j < n_in; ++j)
      if (overlap(outs[i], ins[j])) return true;
    for (int j = 0; j < i; ++j)
      if (overlap(outs[i], outs[j])) return true;
  }
  return false;
}

// What a policy loss reads, and its workspace.
int32_t policy_check(const nsp_policy_t* policy, const int32_t* cu, int32_t ndoc, int64_t rows,
                     const float* stats, void* workspace, size_t workspace_bytes, bool logits,
                     PolicyRows& p, LossArgs& l) {
  if (!policy || ndoc < 1 || rows < 0 || !cu || !stats) return NSP_ERR_INVALID;
  if (rows > kMaxTokens) return NSP_ERR_UNSUPPORTED;
  if (!(policy->clip_low >= 0.f) || !(policy->clip_low <= 1.f) || !(policy->clip_high >= 0.f) ||
      !std::isfinite(policy->clip_high) || !std::isfinite(policy->kl_coef) ||
      !(policy->total >= 0.f) || !std::isfinite(policy->total))
    return NSP_ERR_INVALID;
  if ((policy->mean != NSP_MEAN_TOKENS && policy->mean != NSP_MEAN_DOCUMENTS) ||
      (policy->per_token != 0 && policy->per_token != 1))
    return NSP_ERR_INVALID;
  if (rows > 0 && (!policy->advantages || !policy->old_logp)) return NSP_ERR_INVALID;
  if (policy->kl_coef != 0.f && rows > 0 && !policy->ref_logp) return NSP_ERR_INVALID;
  const void* ptrs[] = {policy->old_logp, policy->ref_logp, policy->advantages, cu, stats};
  for (const void* x : ptrs)
    if (!aligned(x, 4)) return NSP_ERR_ALIGN;
  const LossWsLayout L = loss_ws_layout(rows, ndoc, logits);
  if (!workspace || workspace_bytes < L.total) return NSP_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return NSP_ERR_ALIGN;
  char* const ws = reinterpret_cast<char*>(workspace);
  p.old_logp = policy->old_logp; p.ref_logp = policy->ref_logp; p.advantages = policy->advantages;
  p.per_token = policy->per_token;
  p.clip_low = policy->clip_low; p.clip_high = policy->clip_high; p.kl_coef = policy->kl_coef;
  p.cu = cu; p.ndoc = ndoc;
  p.hdr = reinterpret_cast<WsHeader*>(ws);
  p.doc_weight = reinterpret_cast<float*>(ws + L.weight);
  p.terms = reinterpret_cast<float*>(ws + L.terms);
  p.row_scalars = reinterpret_cast<float2*>(ws + L.scalars);
  l.list = logits ? reinterpret_cast<int2*>(ws + L.list) : nullptr;
  l.cu = cu; l.ndoc = ndoc; l.rows = rows;
  l.mean = policy->mean; l.total = policy->total;
  l.hdr = reinterpret_cast<WsHeader*>(ws);
  l.bits = reinterpret_cast<uint32_t*>(ws + L.bits);
  l.before = reinterpret_cast<int32_t*>(ws + L.before);
  l.weight = reinterpret_cast<float*>(ws + L.weight);
  return NSP_OK;
}

int32_t status_of(cudaError_t e) { return e == cudaSuccess ? NSP_OK : NSP_ERR_CUDA; }

}  // namespace

extern "C" {

int32_t nsp_qk_norm_rope_fwd(const nsp_qk_tensor_t* tensors, int32_t n, const int32_t* cu_seqlens,
                             int32_t ndoc, const int32_t* positions, int64_t start, int64_t len,
                             int32_t d, int32_t rot, const double* freqs, int32_t interleaved,
                             float mscale, float eps, int32_t io_dtype, nsp_stream_t stream) {
  QkArgs a;
  const int32_t st = qk_check(tensors, n, cu_seqlens, ndoc, positions, start, len, d, rot, freqs,
                              interleaved, mscale, eps, io_dtype, false, nullptr, 0, a);
  if (st != NSP_OK || len == 0) return st;
  return status_of(launch_qk_norm_rope(a, io_dtype, reinterpret_cast<cudaStream_t>(stream)));
}

size_t nsp_qk_norm_rope_bwd_workspace_size(const nsp_qk_tensor_t* tensors, int32_t n, int64_t len,
                                           int32_t d) {
  if (!tensors || n < 1 || n > kRopeMaxTensors || len < 0 || len > kMaxTokens || d < 1 ||
      d > kQkMaxDim)
    return 0;
  size_t blocks = 0;
  for (int32_t i = 0; i < n; ++i)
    if (tensors[i].heads < 1 || tensors[i].heads > kMaxHeads) return 0;
  for (int32_t i = 0; i < n; ++i) blocks += (size_t)qk_bwd_blocks(tensors, n, i, len);
  return blocks * (size_t)d * sizeof(float);
}

int32_t nsp_qk_norm_rope_bwd(const nsp_qk_tensor_t* tensors, int32_t n, const int32_t* cu_seqlens,
                             int32_t ndoc, const int32_t* positions, int64_t start, int64_t len,
                             int32_t d, int32_t rot, const double* freqs, int32_t interleaved,
                             float mscale, float eps, int32_t io_dtype, void* workspace,
                             size_t workspace_bytes, nsp_stream_t stream) {
  QkArgs a;
  const int32_t st = qk_check(tensors, n, cu_seqlens, ndoc, positions, start, len, d, rot, freqs,
                              interleaved, mscale, eps, io_dtype, true, workspace, workspace_bytes, a);
  if (st != NSP_OK) return st;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (len == 0) {
    // no rows: the weights' gradients are zero
    for (int32_t i = 0; i < n; ++i)
      if (a.t[i].dweight && cudaMemsetAsync(a.t[i].dweight, 0, (size_t)(d * elem_bytes(io_dtype)), s) !=
                                cudaSuccess)
        return NSP_ERR_CUDA;
    return NSP_OK;
  }
  return status_of(launch_qk_norm_rope_bwd(a, io_dtype, s));
}

// ---------------------------------------------------------------- token log-probabilities

size_t nsp_token_logp_workspace_size(int64_t rows) {
  return rows < 0 || rows > kMaxTokens ? 0 : sizeof(WsHeader) + sizeof(int2) * (size_t)rows;
}

int32_t nsp_token_logp_fwd(const void* logits, int64_t row_stride, const int32_t* targets, int64_t rows,
                           int32_t vocab, double scale, int32_t io_dtype, float* logp, float* lse,
                           void* workspace, size_t workspace_bytes, nsp_stream_t stream) {
  RowArgs a;
  const int32_t st = rows_check(logits, row_stride, targets, rows, vocab, scale, io_dtype, a);
  if (st != NSP_OK) return st;
  if (rows > 0 && !logp) return NSP_ERR_INVALID;
  if (!aligned(logp, 4) || !aligned(lse, 4)) return NSP_ERR_ALIGN;
  const size_t need = nsp_token_logp_workspace_size(rows);
  if (!workspace || workspace_bytes < need) return NSP_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return NSP_ERR_ALIGN;
  const Span outs[] = {packed(logp, 1, rows * 4), packed(lse, 1, rows * 4), packed(workspace, 1, (int64_t)need)};
  const Span ins[] = {logits_span(a, elem_bytes(io_dtype)), packed(targets, 1, rows * 4)};
  if (clash(outs, 3, ins, 2)) return NSP_ERR_INVALID;
  if (rows == 0) return NSP_OK;
  a.logp = logp;
  a.lse = lse;
  a.hdr = reinterpret_cast<WsHeader*>(workspace);
  a.list = reinterpret_cast<int2*>(reinterpret_cast<char*>(workspace) + sizeof(WsHeader));
  return status_of(launch_rows(a, kRowForward, io_dtype, reinterpret_cast<cudaStream_t>(stream)));
}

int32_t nsp_token_logp_bwd(const void* logits, int64_t row_stride, const int32_t* targets,
                           const float* lse, const float* dlogp, int64_t rows, int32_t vocab,
                           double scale, int32_t io_dtype, void* dlogits, int64_t out_stride,
                           nsp_stream_t stream) {
  RowArgs a;
  int32_t st = rows_check(logits, row_stride, targets, rows, vocab, scale, io_dtype, a);
  if (st == NSP_OK) st = gradient_check(dlogits, out_stride, io_dtype, a);
  if (st != NSP_OK) return st;
  if (rows > 0 && (!lse || !dlogp)) return NSP_ERR_INVALID;
  if (!aligned(lse, 4) || !aligned(dlogp, 4)) return NSP_ERR_ALIGN;
  if (rows == 0) return NSP_OK;
  const int64_t es = elem_bytes(io_dtype);
  const Span in = logits_span(a, es), out = gradient_span(a, es);
  const Span ins[] = {packed(targets, 1, rows * 4), packed(lse, 1, rows * 4), packed(dlogp, 1, rows * 4)};
  if (clash(&out, 1, ins, 3) || (!same_rows(in, out) && overlap(in, out))) return NSP_ERR_INVALID;
  a.in_lse = lse;
  a.dlogp = dlogp;
  return status_of(launch_rows(a, kRowBackward, io_dtype, reinterpret_cast<cudaStream_t>(stream)));
}

// ---------------------------------------------------------------- losses

size_t nsp_policy_loss_workspace_size(int64_t rows, int32_t ndoc, int32_t logits) {
  if (rows < 0 || rows > kMaxTokens || ndoc < 1 || (logits != 0 && logits != 1)) return 0;
  return loss_ws_layout(rows, ndoc, logits != 0).total;
}

int32_t nsp_policy_loss(const float* logp, const int32_t* targets, const int32_t* cu_seqlens,
                        int32_t ndoc, int64_t rows, const nsp_policy_t* policy, float* stats,
                        float* dlogp, void* workspace, size_t workspace_bytes, nsp_stream_t stream) {
  PolicyArgs a = {};
  LossArgs l = {};
  const int32_t st = policy_check(policy, cu_seqlens, ndoc, rows, stats, workspace, workspace_bytes,
                                  false, a.p, l);
  if (st != NSP_OK) return st;
  if (rows > 0 && (!logp || !targets || !dlogp)) return NSP_ERR_INVALID;
  if (!aligned(logp, 4) || !aligned(targets, 4) || !aligned(dlogp, 4)) return NSP_ERR_ALIGN;
  const int64_t n = rows * 4;
  const Span outs[] = {packed(stats, 1, 16), packed(dlogp, 1, n),
                       packed(workspace, 1, (int64_t)loss_ws_layout(rows, ndoc, false).total)};
  const Span ins[] = {packed(logp, 1, n), packed(targets, 1, n), packed(a.p.old_logp, 1, n),
                      packed(a.p.ref_logp, 1, n), packed(cu_seqlens, 1, ((int64_t)ndoc + 1) * 4),
                      packed(a.p.advantages, 1, a.p.per_token ? n : (int64_t)ndoc * 4)};
  if (clash(outs, 3, ins, 6)) return NSP_ERR_INVALID;
  a.logp = logp; a.targets = targets; a.rows = rows;
  a.stats = stats; a.dlogp = dlogp;
  l.targets = targets;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = launch_loss_prep(l, s);
  return status_of(e != cudaSuccess ? e : launch_policy(a, s));
}

int32_t nsp_policy_loss_logits(const void* logits, int64_t row_stride, const int32_t* targets,
                               const int32_t* cu_seqlens, int32_t ndoc, int64_t rows, int32_t vocab,
                               double scale, int32_t io_dtype, const nsp_policy_t* policy, float* stats,
                               float* logp, void* dlogits, int64_t out_stride, void* workspace,
                               size_t workspace_bytes, nsp_stream_t stream) {
  RowArgs a;
  LossArgs l = {};
  int32_t st = rows_check(logits, row_stride, targets, rows, vocab, scale, io_dtype, a);
  if (st == NSP_OK) st = gradient_check(dlogits, out_stride, io_dtype, a);
  if (st == NSP_OK)
    st = policy_check(policy, cu_seqlens, ndoc, rows, stats, workspace, workspace_bytes, true, a.p, l);
  if (st != NSP_OK) return st;
  if (!aligned(logp, 4)) return NSP_ERR_ALIGN;
  const int64_t es = elem_bytes(io_dtype), n = rows * 4;
  const Span in = logits_span(a, es), out = gradient_span(a, es);
  const Span outs[] = {packed(stats, 1, 16), packed(logp, 1, n), out,
                       packed(workspace, 1, (int64_t)loss_ws_layout(rows, ndoc, true).total)};
  const Span ins[] = {packed(targets, 1, n), packed(a.p.old_logp, 1, n), packed(a.p.ref_logp, 1, n),
                      packed(cu_seqlens, 1, ((int64_t)ndoc + 1) * 4),
                      packed(a.p.advantages, 1, a.p.per_token ? n : (int64_t)ndoc * 4)};
  if (clash(outs, 4, ins, 5)) return NSP_ERR_INVALID;
  for (const Span& o : outs)
    if (overlap(o, in) && !(&o == &outs[2] && same_rows(in, out))) return NSP_ERR_INVALID;
  a.logp = logp;
  a.hdr = l.hdr;
  a.list = l.list;
  l.targets = targets;
  if (!rows_listed(a, kRowPolicy, io_dtype)) l.list = nullptr;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  cudaError_t e = launch_loss_prep(l, s);
  if (e == cudaSuccess && rows > 0) e = launch_rows(a, kRowPolicy, io_dtype, s);
  return status_of(e != cudaSuccess ? e : launch_policy_stats(a, stats, s));
}

size_t nsp_preference_loss_workspace_size(int32_t ndoc) {
  return ndoc < 2 || ndoc % 2 != 0 ? 0 : sizeof(WsHeader) + 3 * sizeof(float) * (size_t)(ndoc / 2);
}

int32_t nsp_preference_loss(const float* logp, const float* ref_logp, const int32_t* targets,
                            const int32_t* cu_seqlens, int32_t ndoc, int64_t rows, int32_t kind,
                            float beta, float smoothing, float margin, int32_t average, float* stats,
                            float* rewards, float* dlogp, void* workspace, size_t workspace_bytes,
                            nsp_stream_t stream) {
  if (ndoc < 2 || ndoc % 2 != 0 || rows < 0 || !cu_seqlens || !stats || !rewards) return NSP_ERR_INVALID;
  if (rows > kMaxTokens) return NSP_ERR_UNSUPPORTED;
  if (kind < NSP_PREFERENCE_SIGMOID || kind > NSP_PREFERENCE_SQUARE || (average != 0 && average != 1))
    return NSP_ERR_INVALID;
  if (!(beta > 0.f) || !std::isfinite(beta) || !(smoothing >= 0.f) || !(smoothing <= 1.f) ||
      !std::isfinite(margin))
    return NSP_ERR_INVALID;
  if (rows > 0 && (!logp || !targets || !dlogp)) return NSP_ERR_INVALID;
  const void* ptrs[] = {logp, ref_logp, targets, cu_seqlens, stats, rewards, dlogp};
  for (const void* x : ptrs)
    if (!aligned(x, 4)) return NSP_ERR_ALIGN;
  const size_t need = nsp_preference_loss_workspace_size(ndoc);
  if (!workspace || workspace_bytes < need) return NSP_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return NSP_ERR_ALIGN;
  const int64_t n = rows * 4, docs = (int64_t)ndoc * 4;
  const Span outs[] = {packed(stats, 1, 8), packed(rewards, 1, docs), packed(dlogp, 1, n),
                       packed(workspace, 1, (int64_t)need)};
  const Span ins[] = {packed(logp, 1, n), packed(ref_logp, 1, n), packed(targets, 1, n),
                      packed(cu_seqlens, 1, docs + 4)};
  if (clash(outs, 4, ins, 4)) return NSP_ERR_INVALID;
  PreferenceArgs a = {};
  a.logp = logp; a.ref_logp = ref_logp; a.targets = targets; a.cu = cu_seqlens;
  a.ndoc = ndoc; a.rows = rows;
  a.kind = kind; a.beta = beta; a.smoothing = smoothing; a.margin = margin; a.average = average;
  a.hdr = reinterpret_cast<WsHeader*>(workspace);
  a.terms = reinterpret_cast<float*>(reinterpret_cast<char*>(workspace) + sizeof(WsHeader));
  a.stats = stats; a.rewards = rewards; a.dlogp = dlogp;
  return status_of(launch_preference(a, reinterpret_cast<cudaStream_t>(stream)));
}

// ---------------------------------------------------------------- many gradients

static int32_t grads_check(const GradArgs& a, size_t workspace_bytes) {
  if (a.n < 1 || !a.in || !a.counts || !a.in_dtypes || !a.norm) return NSP_ERR_INVALID;
  if (a.n > kMaxGrads) return NSP_ERR_UNSUPPORTED;
  if ((a.kind != NSP_NORM_2 && a.kind != NSP_NORM_INF) || !std::isfinite(a.unscale))
    return NSP_ERR_INVALID;
  if (!aligned(a.norm, 4)) return NSP_ERR_ALIGN;
  for (int32_t i = 0; i < a.n; ++i) {
    if (!dtype_ok(a.in_dtypes[i]) || a.counts[i] < 0) return NSP_ERR_INVALID;
    if (a.counts[i] > ((int64_t)1 << 40)) return NSP_ERR_UNSUPPORTED;
    if (a.counts[i] > 0 && !a.in[i]) return NSP_ERR_INVALID;
    if (!aligned(a.in[i], elem_bytes(a.in_dtypes[i]))) return NSP_ERR_ALIGN;
    if (!a.out) continue;
    if (!dtype_ok(a.out_dtypes[i]) || (a.counts[i] > 0 && !a.out[i])) return NSP_ERR_INVALID;
    if (!aligned(a.out[i], elem_bytes(a.out_dtypes[i]))) return NSP_ERR_ALIGN;
  }
  if (!a.workspace || workspace_bytes < grad_ws_size(a.counts, a.n)) return NSP_ERR_WORKSPACE;
  if (!aligned(a.workspace, 16)) return NSP_ERR_ALIGN;
  return NSP_OK;
}

// Whether an output shares a byte with another array of the call: all arrays in order of
// their addresses, none of which may begin before the end of an earlier output, nor an
// output before the end of any earlier array.  An output in its own input's place is one.
static bool grads_clash(const GradArgs& a) {
  struct Extent {
    uintptr_t base;
    int64_t bytes;                          // negative: written
  };
  const int64_t ws = (int64_t)grad_ws_size(a.counts, a.n);
  const Span outs[] = {packed(a.workspace, 1, ws), packed(a.norm, 1, 4)};
  if (overlap(outs[0], outs[1])) return true;
  Extent at[2 * kMaxGrads];
  int32_t n = 0;
  for (int32_t i = 0; i < a.n; ++i) {
    if (a.counts[i] == 0) continue;
    const bool in_place = a.out && a.out[i] == a.in[i];
    if (in_place && a.out_dtypes[i] != a.in_dtypes[i]) return true;
    const Span in = packed(a.in[i], 1, a.counts[i] * elem_bytes(a.in_dtypes[i]));
    if (overlap(in, outs[0]) || overlap(in, outs[1])) return true;
    at[n++] = {in.base, in_place ? -in.row : in.row};
    if (!a.out || in_place) continue;
    const Span out = packed(a.out[i], 1, a.counts[i] * elem_bytes(a.out_dtypes[i]));
    if (overlap(out, outs[0]) || overlap(out, outs[1])) return true;
    at[n++] = {out.base, -out.row};
  }
  if (!a.out) return false;                 // nothing else is written
  std::sort(at, at + n, [](const Extent& x, const Extent& y) { return x.base < y.base; });
  uintptr_t end = 0, written_end = 0;
  for (int32_t i = 0; i < n; ++i) {
    const bool written = at[i].bytes < 0;
    if (at[i].base < (written ? end : written_end)) return true;
    const uintptr_t e = at[i].base + (uintptr_t)(written ? -at[i].bytes : at[i].bytes);
    end = std::max(end, e);
    if (written) written_end = std::max(written_end, e);
  }
  return false;
}

size_t nsp_grad_norm_workspace_size(const int64_t* counts, int32_t n) {
  if (!counts || n < 1 || n > kMaxGrads) return 0;
  for (int32_t i = 0; i < n; ++i)
    if (counts[i] < 0 || counts[i] > ((int64_t)1 << 40)) return 0;
  return grad_ws_size(counts, n);
}

int32_t nsp_grad_norm(const void* const* grads, const int64_t* counts, const int32_t* dtypes, int32_t n,
                      int32_t kind, float unscale, float* norm, void* workspace, size_t workspace_bytes,
                      nsp_stream_t stream) {
  GradArgs a = {};
  a.n = n; a.in = grads; a.counts = counts; a.in_dtypes = dtypes;
  a.kind = kind; a.unscale = unscale; a.norm = norm;
  a.workspace = reinterpret_cast<char*>(workspace);
  const int32_t st = grads_check(a, workspace_bytes);
  if (st != NSP_OK) return st;
  if (grads_clash(a)) return NSP_ERR_INVALID;
  return status_of(launch_grads(a, reinterpret_cast<cudaStream_t>(stream)));
}

int32_t nsp_grad_clip(const void* const* grads, void* const* out, const int64_t* counts,
                      const int32_t* dtypes, const int32_t* out_dtypes, int32_t n, int32_t kind,
                      float unscale, float max_norm, float eps, float* norm, void* workspace,
                      size_t workspace_bytes, nsp_stream_t stream) {
  if (!out || !out_dtypes) return NSP_ERR_INVALID;
  if (!(max_norm >= 0.f) || !std::isfinite(max_norm) || !(eps > 0.f) || !std::isfinite(eps))
    return NSP_ERR_INVALID;
  GradArgs a = {};
  a.n = n; a.in = grads; a.out = out; a.counts = counts; a.in_dtypes = dtypes; a.out_dtypes = out_dtypes;
  a.kind = kind; a.unscale = unscale; a.max_norm = max_norm; a.eps = eps; a.norm = norm;
  a.workspace = reinterpret_cast<char*>(workspace);
  const int32_t st = grads_check(a, workspace_bytes);
  if (st != NSP_OK) return st;
  if (grads_clash(a)) return NSP_ERR_INVALID;
  return status_of(launch_grads(a, reinterpret_cast<cudaStream_t>(stream)));
}

}  // extern "C"
