// C ABI entry points of the operators around differential attention: host
// validation, workspace carving and dispatch.  Nothing here allocates memory
// or synchronises.
#include <cmath>

#include "layer.cuh"

using namespace nsp;

namespace {

constexpr int64_t kMaxTokens = (int64_t)1 << 30;
constexpr int32_t kMaxHeads = 1 << 15;           // keeps grids, coordinates and counts in range

bool aligned(const void* p, uintptr_t n) { return (reinterpret_cast<uintptr_t>(p) & (n - 1)) == 0; }
bool dtype_ok(int32_t t) { return t == NSP_F32 || t == NSP_BF16; }
int64_t elem_bytes(int32_t t) { return t == NSP_BF16 ? 2 : 4; }

// rows of `row` bytes, `step` bytes apart
struct Span {
  uintptr_t base;
  int64_t rows, step, row;
  uintptr_t end() const { return base + (uintptr_t)((rows - 1) * step + row); }
};

// Whether two spans share a byte.  Spans of the same step (views of one
// tensor's columns) are compared column by column; others by their extents.
bool overlap(const Span& a, const Span& b) {
  if (a.rows < 1 || b.rows < 1 || a.end() <= b.base || b.end() <= a.base) return false;
  if (a.step != b.step || a.row > a.step || b.row > b.step) return true;
  const int64_t off = ((int64_t)(b.base - a.base) % a.step + a.step) % a.step;
  return off < a.row || off + b.row > a.step;
}

bool same_rows(const Span& a, const Span& b) {
  return a.base == b.base && a.rows == b.rows && a.step == b.step;
}

// `rows` rows of `row` bytes, one behind the other; none where p is NULL
Span packed(const void* p, int64_t rows, int64_t row) {
  return {reinterpret_cast<uintptr_t>(p), p ? rows : 0, row, row};
}

}  // namespace

extern "C" {

int32_t nsp_rope_freqs(int32_t rot, double base, int32_t scaling, double factor, double low,
                       double high, double orig_len, double* freqs_host) {
  if (rot < 2 || rot % 2 != 0 || rot > kRopeMaxDim || !freqs_host) return NSP_ERR_INVALID;
  if (!(base > 0) || !std::isfinite(base)) return NSP_ERR_INVALID;
  if (scaling < NSP_ROPE_PLAIN || scaling > NSP_ROPE_PARTS) return NSP_ERR_INVALID;
  if (scaling != NSP_ROPE_PLAIN && (!(factor >= 1) || !std::isfinite(factor))) return NSP_ERR_INVALID;
  if (scaling == NSP_ROPE_PARTS &&
      (!(orig_len > 0) || !std::isfinite(orig_len) || !(low >= 0) || !(high > low) ||
       !std::isfinite(high)))
    return NSP_ERR_INVALID;
  if (scaling == NSP_ROPE_BASE && rot == 2) return NSP_ERR_INVALID;   // its exponent divides by rot - 2
  const double b = scaling == NSP_ROPE_BASE ? base * std::pow(factor, (double)rot / (rot - 2)) : base;
  for (int32_t i = 0; i < rot / 2; ++i) {
    double f = std::pow(b, -2.0 * i / rot);
    if (scaling == NSP_ROPE_LINEAR) f /= factor;
    if (scaling == NSP_ROPE_PARTS) {
      const double turns = orig_len * f / 6.283185307179586476925;
      const double keep = std::fmin(1.0, std::fmax(0.0, (turns - low) / (high - low)));
      f = keep * f + (1.0 - keep) * f / factor;
    }
    freqs_host[i] = f;
  }
  return NSP_OK;
}

int32_t nsp_rope(const nsp_rope_tensor_t* tensors, int32_t n, const int32_t* cu_seqlens,
                 int32_t ndoc, const int32_t* positions, int64_t start, int64_t len, int32_t d,
                 int32_t rot, const double* freqs, int32_t interleaved, float mscale,
                 int32_t inverse, int32_t io_dtype, nsp_stream_t stream) {
  if (!tensors || n < 1 || n > kRopeMaxTensors || !dtype_ok(io_dtype)) return NSP_ERR_INVALID;
  if (d < 2 || rot < 2 || rot % 2 != 0 || rot > d) return NSP_ERR_INVALID;
  if (d > kRopeMaxDim) return NSP_ERR_UNSUPPORTED;
  if ((interleaved != 0 && interleaved != 1) || (inverse != 0 && inverse != 1))
    return NSP_ERR_INVALID;
  if (!std::isfinite(mscale) || start < 0 || len < 0) return NSP_ERR_INVALID;
  if (len > kMaxTokens || start > kMaxTokens - len) return NSP_ERR_UNSUPPORTED;
  if (!freqs || (!positions && (!cu_seqlens || ndoc < 1))) return NSP_ERR_INVALID;
  if (!aligned(freqs, 8) || !aligned(positions, 4) || !aligned(cu_seqlens, 4)) return NSP_ERR_ALIGN;
  const int64_t es = elem_bytes(io_dtype);
  RopeArgs a;
  Span in[kRopeMaxTensors], out[kRopeMaxTensors];
  for (int32_t i = 0; i < n; ++i) {
    const nsp_rope_tensor_t& t = tensors[i];
    if (t.heads < 1 || t.groups < 1 || t.heads % t.groups != 0) return NSP_ERR_INVALID;
    if (t.heads > kMaxHeads) return NSP_ERR_UNSUPPORTED;
    if (len > 0 && (!t.in || !t.out)) return NSP_ERR_INVALID;
    if (!aligned(t.in, es) || !aligned(t.out, es)) return NSP_ERR_ALIGN;
    const int64_t width = (int64_t)t.heads * d;
    const int64_t is = t.in_stride == 0 ? width : t.in_stride;
    const int64_t os = t.out_stride == 0 ? width : t.out_stride;
    if (is < width || os < width) return NSP_ERR_INVALID;
    if (is > ((int64_t)1 << 31) || os > ((int64_t)1 << 31)) return NSP_ERR_UNSUPPORTED;
    // the head-group-major side is packed
    if (t.groups > 1 && (inverse ? is : os) != width) return NSP_ERR_INVALID;
    a.t[i].in = t.in; a.t[i].out = t.out;
    a.t[i].in_stride = is; a.t[i].out_stride = os;
    a.t[i].heads = t.heads;
    a.t[i].in_groups = inverse ? t.groups : 1;
    a.t[i].out_groups = inverse ? 1 : t.groups;
    a.t[i].hpg = t.heads / t.groups;
    const int64_t jump = t.groups > 1 ? (len - 1) * a.t[i].hpg * d : 0;
    a.t[i].in_jump = inverse ? jump : 0;
    a.t[i].out_jump = inverse ? 0 : jump;
    in[i] = {reinterpret_cast<uintptr_t>(t.in), len, is * es, width * es};
    out[i] = {reinterpret_cast<uintptr_t>(t.out), len, os * es, width * es};
  }
  for (int32_t i = 0; i < n; ++i)
    for (int32_t j = 0; j < n; ++j) {
      // a tensor may be rotated in place: the same rows, not regrouped
      const bool in_place = i == j && in[i].base == out[i].base && in[i].step == out[i].step &&
                            tensors[i].groups == 1;
      if (!in_place && overlap(in[i], out[j])) return NSP_ERR_INVALID;
      if (i < j && overlap(out[i], out[j])) return NSP_ERR_INVALID;
    }
  const Span read[] = {packed(positions, 1, len * 4), packed(freqs, 1, rot / 2 * 8),
                       packed(positions ? nullptr : cu_seqlens, 1, ((int64_t)ndoc + 1) * 4)};
  for (int32_t j = 0; j < n; ++j)
    for (const Span& r : read)
      if (overlap(r, out[j])) return NSP_ERR_INVALID;
  if (len == 0) return NSP_OK;
  a.n = n;
  a.cu = cu_seqlens; a.ndoc = ndoc; a.positions = positions;
  a.start = start; a.len = len; a.d = d; a.rot = rot;
  a.interleaved = interleaved; a.inverse = inverse;
  a.freqs = freqs; a.mscale = mscale;
  return launch_rope(a, io_dtype, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? NSP_OK
             : NSP_ERR_CUDA;
}

static int32_t lambda_check(const void* const* v, const void* io, int32_t n, int32_t dl,
                            int32_t heads, int32_t io_dtype) {
  if (!dtype_ok(io_dtype) || dl < 1 || heads < 1 || (n != 1 && n != heads)) return NSP_ERR_INVALID;
  if (heads > kMaxHeads || dl > (1 << 20)) return NSP_ERR_UNSUPPORTED;
  const uintptr_t es = (uintptr_t)elem_bytes(io_dtype);
  for (int i = 0; i < 4; ++i) {
    if (!v[i]) return NSP_ERR_INVALID;
    if (!aligned(v[i], es)) return NSP_ERR_ALIGN;
  }
  if (!io) return NSP_ERR_INVALID;
  return aligned(io, es) ? NSP_OK : NSP_ERR_ALIGN;
}

int32_t nsp_diff_lambda_fwd(const void* q1, const void* k1, const void* q2, const void* k2, int32_t n,
                            int32_t dl, int32_t heads, float init, int32_t io_dtype, void* lambda,
                            nsp_stream_t stream) {
  const void* v[4] = {q1, k1, q2, k2};
  const int32_t st = lambda_check(v, lambda, n, dl, heads, io_dtype);
  if (st != NSP_OK) return st;
  if (!std::isfinite(init)) return NSP_ERR_INVALID;
  const int64_t es = elem_bytes(io_dtype);
  for (int i = 0; i < 4; ++i)
    if (overlap(packed(lambda, 1, heads * es), packed(v[i], n, dl * es))) return NSP_ERR_INVALID;
  return launch_diff_lambda(v, n, dl, heads, init, io_dtype, lambda,
                            reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? NSP_OK
             : NSP_ERR_CUDA;
}

int32_t nsp_diff_lambda_bwd(const void* dlambda, const void* q1, const void* k1, const void* q2,
                            const void* k2, int32_t n, int32_t dl, int32_t heads, int32_t io_dtype,
                            void* dq1, void* dk1, void* dq2, void* dk2, nsp_stream_t stream) {
  const void* v[4] = {q1, k1, q2, k2};
  int32_t st = lambda_check(v, dlambda, n, dl, heads, io_dtype);
  if (st != NSP_OK) return st;
  void* g[4] = {dq1, dk1, dq2, dk2};
  st = lambda_check(g, dlambda, n, dl, heads, io_dtype);
  if (st != NSP_OK) return st;
  const int64_t es = elem_bytes(io_dtype);
  for (int i = 0; i < 4; ++i) {
    const Span o = packed(g[i], n, dl * es);
    if (overlap(o, packed(dlambda, 1, heads * es))) return NSP_ERR_INVALID;
    for (int j = 0; j < 4; ++j)
      if (overlap(o, packed(v[j], n, dl * es)) || (j < i && overlap(o, packed(g[j], n, dl * es))))
        return NSP_ERR_INVALID;
  }
  return launch_diff_lambda_bwd(dlambda, v, n, dl, heads, io_dtype, g,
                                reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? NSP_OK
             : NSP_ERR_CUDA;
}

static int32_t norm_check(const NormArgs& a, int32_t io_dtype) {
  if (!dtype_ok(io_dtype) || a.tokens < 0 || a.heads < 1 || a.d < 1) return NSP_ERR_INVALID;
  if (!(a.eps > 0.f) || !std::isfinite(a.eps) || !std::isfinite(a.scale)) return NSP_ERR_INVALID;
  if (a.tokens > kMaxTokens || a.heads > kMaxHeads) return NSP_ERR_UNSUPPORTED;
  // rows are read in 16-byte pieces
  if (a.d * elem_bytes(io_dtype) % 16 != 0 || a.d > kNormMaxDim) return NSP_ERR_UNSUPPORTED;
  if (a.x_stride < (int64_t)a.heads * a.d) return NSP_ERR_INVALID;
  if (a.x_stride * elem_bytes(io_dtype) % 16 != 0) return NSP_ERR_ALIGN;
  if (a.tokens > 0 && !a.x) return NSP_ERR_INVALID;
  const void* ptrs[] = {a.x, a.gate, a.weight, a.dy, a.y, a.dx, a.dgate, a.dweight, a.partial};
  for (const void* p : ptrs)
    if (!aligned(p, 16)) return NSP_ERR_ALIGN;
  // an output shares no byte with another array, but y may take gate's or a packed
  // x's place, dx dy's and dgate gate's: a row is read whole before it is written
  const int64_t es = elem_bytes(io_dtype), width = a.heads * a.d * es;
  const Span x = {reinterpret_cast<uintptr_t>(a.x), a.tokens, a.x_stride * es, width};
  const Span gate = packed(a.gate, a.tokens, width), dy = packed(a.dy, a.tokens, width);
  const Span w = packed(a.weight, 1, a.d * es);
  const Span outs[] = {packed(a.y, a.tokens, width), packed(a.dx, a.tokens, width),
                       packed(a.dgate, a.tokens, width), packed(a.dweight, 1, a.d * es),
                       packed(a.partial, 1, (int64_t)norm_bwd_blocks(a.tokens * a.heads) * a.d *
                                                (int64_t)sizeof(float))};
  constexpr int kY = 0, kDx = 1, kDgate = 2;
  for (int i = 0; i < 5; ++i) {
    const Span& o = outs[i];
    if (overlap(o, w) || (overlap(o, x) && !(i == kY && same_rows(o, x))) ||
        (overlap(o, gate) && !((i == kY || i == kDgate) && same_rows(o, gate))) ||
        (overlap(o, dy) && !(i == kDx && same_rows(o, dy))))
      return NSP_ERR_INVALID;
    for (int j = 0; j < i; ++j)
      if (overlap(o, outs[j])) return NSP_ERR_INVALID;
  }
  return NSP_OK;
}

int32_t nsp_head_norm_fwd(const void* x, int64_t x_stride, const void* weight, const void* gate,
                          int64_t tokens, int32_t heads, int32_t d, float eps, float scale,
                          int32_t io_dtype, void* y, nsp_stream_t stream) {
  NormArgs a = {};
  a.x = x; a.weight = weight; a.gate = gate; a.y = y;
  a.x_stride = x_stride == 0 ? (int64_t)heads * d : x_stride;
  a.tokens = tokens; a.heads = heads; a.d = d; a.eps = eps; a.scale = scale;
  const int32_t st = norm_check(a, io_dtype);
  if (st != NSP_OK) return st;
  if (tokens == 0) return NSP_OK;
  if (!y) return NSP_ERR_INVALID;
  return launch_head_norm(a, io_dtype, reinterpret_cast<cudaStream_t>(stream)) == cudaSuccess
             ? NSP_OK
             : NSP_ERR_CUDA;
}

size_t nsp_head_norm_bwd_workspace_size(int64_t tokens, int32_t heads, int32_t d) {
  if (tokens < 0 || tokens > kMaxTokens || heads < 1 || heads > kMaxHeads || d < 1 ||
      d > kNormMaxDim)
    return 0;
  return (size_t)norm_bwd_blocks(tokens * heads) * (size_t)d * sizeof(float);
}

int32_t nsp_head_norm_bwd(const void* x, int64_t x_stride, const void* weight, const void* gate,
                          const void* dy, int64_t tokens, int32_t heads, int32_t d, float eps,
                          float scale, int32_t io_dtype, void* dx, void* dgate, void* dweight,
                          void* workspace, size_t workspace_bytes, nsp_stream_t stream) {
  NormArgs a = {};
  a.x = x; a.weight = weight; a.gate = gate; a.dy = dy;
  a.dx = dx; a.dgate = dgate; a.dweight = dweight;
  a.x_stride = x_stride == 0 ? (int64_t)heads * d : x_stride;
  a.tokens = tokens; a.heads = heads; a.d = d; a.eps = eps; a.scale = scale;
  a.partial = dweight ? reinterpret_cast<float*>(workspace) : nullptr;
  const int32_t st = norm_check(a, io_dtype);
  if (st != NSP_OK) return st;
  if ((dgate != nullptr && gate == nullptr) || (dweight != nullptr && weight == nullptr))
    return NSP_ERR_INVALID;
  if (tokens > 0 && (!dy || !dx || (gate && !dgate))) return NSP_ERR_INVALID;
  if (dweight && (!workspace ||
                  workspace_bytes < nsp_head_norm_bwd_workspace_size(tokens, heads, d)))
    return NSP_ERR_WORKSPACE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (tokens == 0) {
    // no rows: the weight's gradient is zero
    if (dweight && cudaMemsetAsync(dweight, 0, (size_t)(d * elem_bytes(io_dtype)), s) != cudaSuccess)
      return NSP_ERR_CUDA;
    return NSP_OK;
  }
  return launch_head_norm_bwd(a, io_dtype, s) == cudaSuccess ? NSP_OK : NSP_ERR_CUDA;
}

// ---------------------------------------------------------------- differential attention

static int32_t diff_check(const int32_t* cu, int32_t ndoc, int64_t T, int32_t Hq, int32_t Hkv,
                          int32_t d, float scale, int32_t causal, int64_t n_lambda,
                          int32_t io_dtype) {
  if (ndoc < 1 || Hq < 1 || Hkv < 1 || Hq % Hkv != 0) return NSP_ERR_INVALID;
  if ((causal != 0 && causal != 1) || !dtype_ok(io_dtype)) return NSP_ERR_INVALID;
  if (T < 0 || !cu || !scale_ok(scale) || (n_lambda != 1 && n_lambda != T)) return NSP_ERR_INVALID;
  if (d != 64 && d != 128) return NSP_ERR_UNSUPPORTED;
  if (T > kMaxTokens || Hq > kMaxHeads) return NSP_ERR_UNSUPPORTED;
  return NSP_OK;
}

static DiffProblem diff_problem(const void* q, const void* k, const void* v, const void* lambda,
                                int64_t n_lambda, const int32_t* cu, int32_t ndoc, int64_t T,
                                int32_t Hq, int32_t Hkv, int32_t d, float scale, int32_t causal,
                                int32_t io_dtype, char* ws) {
  DiffProblem a = {};
  AttnProblem& p = a.p;
  p.q = q; p.k = k; p.v = v; p.cu = cu; p.ndoc = ndoc;
  p.q_start = 0; p.q_len = T; p.kv_start = 0; p.kv_len = T;
  p.Hq = Hq; p.Hkv = Hkv; p.d = d; p.scale = scale; p.causal = causal;
  p.io_dtype = io_dtype; p.out_dtype = io_dtype;
  p.hdr = reinterpret_cast<WsHeader*>(ws);
  p.accumulate = 0;
  p.q_groups = 1;
  p.wait_budget = wait_budget_cycles();
  a.lambda = lambda;
  a.n_lambda = n_lambda;
  a.shift = io_dtype == NSP_BF16 ? item_shift(Hq / Hkv, T) : 0;
  return a;
}

size_t nsp_diff_attn_fwd_workspace_size(int64_t T) {
  if (T < 0 || T > kMaxTokens) return 0;
  return fwd_ws_layout(T, T).total;
}

int32_t nsp_diff_attn_fwd(const void* q, const void* k, const void* v, const void* lambda,
                          int64_t n_lambda, const int32_t* cu_seqlens, int32_t ndoc, int64_t T,
                          int32_t Hq, int32_t Hkv, int32_t d, float scale, int32_t causal,
                          int32_t io_dtype, void* out, void* out2, float* lse, void* workspace,
                          size_t workspace_bytes, nsp_stream_t stream) {
  int32_t st = diff_check(cu_seqlens, ndoc, T, Hq, Hkv, d, scale, causal, n_lambda, io_dtype);
  if (st != NSP_OK) return st;
  if (T > 0 && (!q || !k || !v || !lambda || !out)) return NSP_ERR_INVALID;
  const void* ptrs[] = {q, k, v, lambda, cu_seqlens, out, out2, lse, workspace};
  for (const void* x : ptrs)
    if (!aligned(x, 16)) return NSP_ERR_ALIGN;
  if (io_dtype == NSP_BF16 && (!aligned(out, 32) || !aligned(out2, 32))) return NSP_ERR_ALIGN;
  const FwdWsLayout L = fwd_ws_layout(T, T);
  if (!workspace || workspace_bytes < L.total) return NSP_ERR_WORKSPACE;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  char* ws = reinterpret_cast<char*>(workspace);
  DiffProblem a = diff_problem(q, k, v, lambda, n_lambda, cu_seqlens, ndoc, T, Hq, Hkv, d, scale,
                               causal, io_dtype, ws);
  a.p.out = out; a.p.lse = lse;
  a.out2 = out2;
  if (launch_fwd_schedule(a.p, L, ws, s) != cudaSuccess) return NSP_ERR_CUDA;
  if (T == 0) return NSP_OK;
  const cudaError_t e =
      io_dtype == NSP_BF16 ? launch_diff_fwd_tc(a, L, ws, s) : launch_diff_fwd_simt(a, s);
  return e == cudaSuccess ? NSP_OK : NSP_ERR_CUDA;
}

// Backward workspace: the attention backward's layout for 2 Hq rows of -delta
// and -lse log2 e, then -lambda and lambda delta_2 [Hq, Tp], then shares of dk and dv: for
// float32 with grouped heads each query head's, for bf16 each part's of a split key tile.
struct DiffBwdLayout {
  BwdWsLayout attn;
  size_t coef, heads, total;
};
static DiffBwdLayout diff_bwd_layout(int64_t T, int32_t Hq, int32_t Hkv, int32_t d,
                                     int32_t io_dtype) {
  DiffBwdLayout L;
  L.attn = bwd_ws_layout(T, T, 2 * Hq, d, false);
  L.coef = L.attn.total;
  L.heads = align_up(L.coef + 2 * sizeof(float) * (size_t)Hq * (size_t)L.attn.Tp, 256);
  const bool shares = io_dtype == NSP_F32 && Hq > Hkv;
  L.total = L.heads + (shares ? 2 * sizeof(float) * (size_t)T * (size_t)Hq * (size_t)d : 0);
  const int parts = io_dtype == NSP_BF16 ? key_parts(T, Hkv) : 1;
  if (parts > 1) L.total += 2 * sizeof(float) * (size_t)parts * (size_t)T * (size_t)Hkv * (size_t)d;
  return L;
}

size_t nsp_diff_attn_bwd_workspace_size(int64_t T, int32_t Hq, int32_t Hkv, int32_t d,
                                        int32_t io_dtype) {
  if (T < 0 || T > kMaxTokens || Hq < 1 || Hq > kMaxHeads || Hkv < 1 || d < 1 || d > 128 ||
      !dtype_ok(io_dtype))
    return 0;
  return diff_bwd_layout(T, Hq, Hkv, d, io_dtype).total;
}

int32_t nsp_diff_attn_bwd(const void* q, const void* k, const void* v, const void* lambda,
                          int64_t n_lambda, const void* out, const void* out2, const void* dout,
                          const float* lse, const int32_t* cu_seqlens, int32_t ndoc, int64_t T,
                          int32_t Hq, int32_t Hkv, int32_t d, float scale, int32_t causal,
                          int32_t io_dtype, void* dq, void* dk, void* dv, void* dlambda,
                          void* workspace, size_t workspace_bytes, nsp_stream_t stream) {
  int32_t st = diff_check(cu_seqlens, ndoc, T, Hq, Hkv, d, scale, causal, n_lambda, io_dtype);
  if (st != NSP_OK) return st;
  const void* ptrs[] = {q, k, v, lambda, out, out2, dout, lse, cu_seqlens, dq, dk, dv, dlambda};
  for (const void* x : ptrs) {
    if (T > 0 && !x) return NSP_ERR_INVALID;
    if (!aligned(x, 16)) return NSP_ERR_ALIGN;
  }
  if (io_dtype == NSP_BF16 && (!aligned(dq, 32) || !aligned(dk, 32) || !aligned(dv, 32)))
    return NSP_ERR_ALIGN;
  const DiffBwdLayout W = diff_bwd_layout(T, Hq, Hkv, d, io_dtype);
  const BwdWsLayout& L = W.attn;
  if (!workspace || workspace_bytes < W.total) return NSP_ERR_WORKSPACE;
  if (!aligned(workspace, 16)) return NSP_ERR_ALIGN;
  cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  char* ws = reinterpret_cast<char*>(workspace);
  DiffProblem a = diff_problem(q, k, v, lambda, n_lambda, cu_seqlens, ndoc, T, Hq, Hkv, d, scale,
                               causal, io_dtype, ws);
  a.p.lse = const_cast<float*>(lse);
  a.fout = out; a.out2 = const_cast<void*>(out2); a.dout = dout;
  a.dq = dq; a.dk = dk; a.dv = dv; a.dlambda = dlambda;
  a.ndelta = reinterpret_cast<float*>(ws + L.delta);
  a.nlse2 = reinterpret_cast<float*>(ws + L.nlse2);
  a.coef = reinterpret_cast<float*>(ws + W.coef);
  a.cndelta = a.coef + (size_t)Hq * (size_t)L.Tp;
  a.parts = reinterpret_cast<float*>(ws + W.heads);
  a.dk_heads = a.parts;
  a.dv_heads = a.dk_heads + (size_t)T * (size_t)Hq * (size_t)d;
  a.Tp = L.Tp;
  if (launch_bwd_schedules(a.p, L, ws, s) != cudaSuccess) return NSP_ERR_CUDA;
  if (T == 0) {
    // no token: a head's dlambda is an empty sum
    if (n_lambda == 1 && dlambda != nullptr &&
        cudaMemsetAsync(dlambda, 0, (size_t)(Hq * elem_bytes(io_dtype)), s) != cudaSuccess)
      return NSP_ERR_CUDA;
    return NSP_OK;
  }
  if (launch_diff_prep(a, s) != cudaSuccess) return NSP_ERR_CUDA;
  const cudaError_t e =
      io_dtype == NSP_BF16 ? launch_diff_bwd_tc(a, L, ws, s) : launch_diff_bwd_simt(a, s);
  if (e != cudaSuccess || launch_diff_dlambda(a, s) != cudaSuccess) return NSP_ERR_CUDA;
  return NSP_OK;
}

}  // extern "C"
