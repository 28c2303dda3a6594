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
// Most blocks that the backward gives a tensor, whatever the device.
int qk_bwd_blocks(int64_t rows);
cudaError_t launch_qk_norm_rope(const QkArgs& a, int32_t io_dtype, cudaStream_t s);
cudaError_t launch_qk_norm_rope_bwd(const QkArgs& a, int32_t io_dtype, cudaStream_t s);

}  // namespace nsp
