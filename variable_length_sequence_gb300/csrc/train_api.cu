// C ABI entry points of the operators of a packed post-training step: host
// validation, workspace carving and dispatch.  Nothing here allocates memory
// or synchronises.
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
  for (int32_t i = 0; i < n; ++i) {
    if (tensors[i].heads < 1 || tensors[i].heads > kMaxHeads) return 0;
    blocks += (size_t)qk_bwd_blocks(len * tensors[i].heads);
  }
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

}  // extern "C"
