// moe_norm.cuh -- parameters of the root-mean-square norm and of its backward
// pass, and their launchers.
#pragma once

#include "moe_common.cuh"

namespace moe {

struct NormParams {
  const uint16_t *x;           // [N, H]
  const uint16_t *residual;    // [N, H], or null
  const uint16_t *gain;        // [H]
  uint16_t *sum;               // [N, H], or null
  uint16_t *y;                 // [N, H], or null
  uint8_t *y_q;                // [N, H] E4M3, or null
  float *y_scale;              // [N, ceil(H/128)], or [ceil(H/128), N] with scale_t
  float eps;
  int N, H;
  int scale_t;
};

struct NormBackwardParams {
  const uint16_t *d_y;         // [N, H]
  const uint16_t *d_sum;       // [N, H], or null
  const uint16_t *sum;         // [N, H]: the rows that were normalised
  const uint16_t *gain;        // [H]
  uint16_t *d_x;               // [N, H]
  float *part;                 // [parts][H]: each block's share of the gain's gradient
  float eps;
  int N, H;
};

// Blocks of the backward pass, and thereby partial sums of the gain's gradient.
constexpr int kNormMaxBlocks = 320;

cudaError_t launch_norm(const NormParams &p, cudaStream_t stream);
cudaError_t launch_norm_backward(const NormBackwardParams &p, float *d_gain, cudaStream_t stream);

}  // namespace moe
