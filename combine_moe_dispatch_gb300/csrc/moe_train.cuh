// moe_train.cuh -- parameters of the combine's backward pass and of gradient
// clipping, and their launchers.
#pragma once

#include "moe_common.cuh"

namespace moe {

struct CombineBackwardParams {
  const uint16_t *d_y;         // [N, H]
  const uint16_t *expert_y;    // [E, cap, H]
  const int32_t *topk_idx;
  const int32_t *slot_of;
  const float *topk_weights;
  uint16_t *d_expert_y;        // [E, cap, H]
  float *d_weights;            // [N, K]
  float *d_logits;             // [N, E], or null
  WsHeader *hdr;
  int N, H, E, K, cap;
};

// Workspace of the gradient norm: this header, then one partial sum per block.
struct ClipHeader {
  double total;                // sum of squares so far
  float coef;
  uint32_t done;               // blocks that have left their sum (reset by the last)
  uint32_t reserved[60];
};
static_assert(sizeof(ClipHeader) == 256, "clip header is 256 bytes");
constexpr int kClipMaxBlocks = 1024;

cudaError_t launch_combine_backward(const CombineBackwardParams &p, cudaStream_t stream);
size_t clip_workspace_bytes();
cudaError_t launch_clip(const moe_grad_tensor *tensors, int num, float max_norm, float *norm,
                        void *workspace, cudaStream_t stream);

}  // namespace moe
