// Declarations of the operators of a packed post-training step: the norm of
// query and key heads with the rotation in the same pass, log-probabilities of
// given tokens, the policy and preference losses, and the norm and clipping of
// many gradients.
#pragma once

#include "rotary.cuh"

namespace nsp {

// ---- head norm with rotation (qk_norm.cu)
constexpr int kQkMaxDim = 512;

struct QkTensor {
  const void *x, *weight, *dy;
  void *y, *dx, *dweight;
  int64_t x_stride, y_stride, dx_stride;   // elements between tokens; y_stride: of y or dy
  int32_t heads, groups;                   // groups > 1: y / dy head-group-major
};

struct QkArgs {
  QkTensor t[kRopeMaxTensors];
  int32_t n;
  const int32_t* cu;
  int32_t ndoc;
  const int32_t* positions;
  int64_t start, len;
  int32_t d, rot, interleaved;
  const double* freqs;
  float mscale, eps;
  float* partial;                          // backward: [blocks of a tensor][d] sums, tensor by tensor
};
// The blocks that the backward gives tensor i of n, whatever the device.
int qk_bwd_blocks(const QkTensor* t, int n, int i, int64_t len);
int qk_bwd_blocks(const nsp_qk_tensor_t* t, int n, int i, int64_t len);
cudaError_t launch_qk_norm_rope(const QkArgs& a, int32_t io_dtype, cudaStream_t s);
cudaError_t launch_qk_norm_rope_bwd(const QkArgs& a, int32_t io_dtype, cudaStream_t s);

// ---- log-probabilities of given tokens (token_logp.cu)
constexpr int32_t kMaxVocab = 1 << 20;

// A policy loss on top of the rows: what each row's weight and loss are made of.
struct PolicyRows {
  const float *old_logp, *ref_logp, *advantages;
  int32_t per_token;                       // advantages of each row, or of each document
  float clip_low, clip_high, kl_coef;
  const int32_t* cu;
  int32_t ndoc;
  const WsHeader* hdr;
  const float* doc_weight;                 // [ndoc] weight of a row of the document
  float* terms;                            // [3][rows]: weighted surrogate, kl, clipped
  float2* row_scalars;                     // [rows] weight and advantage (launch_loss_rows)
};

struct RowArgs {
  const void* logits;
  int64_t row_stride;                      // elements
  const int32_t* targets;
  int64_t rows;
  int32_t vocab;
  float scale, c, c_lo;                    // s; s log2(e) in two floats
  float *logp, *lse;                       // forward and policy: written (may be null)
  const float *in_lse, *dlogp;             // backward
  WsHeader* hdr;                           // forward and policy: workspace, n_items scored rows
  int2* list;                              // [rows] row and target of the scored rows, in order;
                                           // from the end backwards the rows not scored
  void* dlogits;
  int64_t out_stride;
  PolicyRows p;
};
enum RowMode { kRowForward, kRowBackward, kRowPolicy };
// Whether launch_rows walks a list of the scored rows.
bool rows_listed(const RowArgs& a, RowMode mode, int32_t io_dtype);
cudaError_t launch_rows(const RowArgs& a, RowMode mode, int32_t io_dtype, cudaStream_t s);

// ---- losses (loss.cu)
// Workspace of a loss: header; per 32 rows the number of scored ones before them and
// which of them are; each document's weight; terms or partial sums; with logits, each
// row's weight and advantage, and the list of rows.
struct LossWsLayout {
  size_t before, bits, weight, terms, scalars, list, total;
};
LossWsLayout loss_ws_layout(int64_t rows, int32_t ndoc, bool logits);

struct LossArgs {
  const int32_t* targets;
  const int32_t* cu;
  int32_t ndoc;
  int64_t rows;
  int32_t mean;
  float total;
  WsHeader* hdr;
  uint32_t* bits;
  int32_t* before;
  float* weight;
  int2* list;                              // null: not wanted
};
// Checks cu_seqlens (status word), counts each document's scored rows and writes
// the documents' weights.
cudaError_t launch_loss_prep(const LossArgs& a, cudaStream_t s);
// each scored row's weight and advantage, and the other rows' zeros, behind launch_loss_prep
cudaError_t launch_loss_rows(const RowArgs& a, cudaStream_t s);
// the list of a forward's scored rows, and the other rows' zeros
cudaError_t launch_row_list(const RowArgs& a, cudaStream_t s);

struct PolicyArgs {
  const float* logp;
  const int32_t* targets;
  int64_t rows;
  PolicyRows p;                            // (p.terms: partial sums of the blocks)
  float *stats, *dlogp;
};
cudaError_t launch_policy(const PolicyArgs& a, cudaStream_t s);
// stats from the rows' terms of a kRowPolicy pass
cudaError_t launch_policy_stats(const RowArgs& a, float* stats, cudaStream_t s);

struct PreferenceArgs {
  const float *logp, *ref_logp;
  const int32_t *targets, *cu;
  int32_t ndoc;
  int64_t rows;
  int32_t kind;
  float beta, smoothing, margin;
  int32_t average;
  WsHeader* hdr;
  float* terms;                            // [3][pairs]: loss, ahead, bad cu_seqlens
  float *stats, *rewards, *dlogp;
};
cudaError_t launch_preference(const PreferenceArgs& a, cudaStream_t s);

// ---- norm and clipping of many gradients (grad_norm.cu)
constexpr int32_t kMaxGrads = 16384;
struct GradArgs {
  int32_t n;
  const void* const* in;                   // HOST arrays
  void* const* out;                        // null: the norm alone
  const int64_t* counts;
  const int32_t *in_dtypes, *out_dtypes;
  int32_t kind;
  float unscale, max_norm, eps;
  float* norm;
  char* workspace;
};
size_t grad_ws_size(const int64_t* counts, int32_t n);
cudaError_t launch_grads(const GradArgs& a, cudaStream_t s);

}  // namespace nsp
