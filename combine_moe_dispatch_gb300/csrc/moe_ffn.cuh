// moe_ffn.cuh -- parameters of the experts' feed-forward and its launchers.
#pragma once

#include "moe_common.cuh"

namespace moe {

// All arrays bf16 and dense.  Forward: x, w_gate_up, w_down -> h (or null),
// act, y.  Backward: dy, x, h, w_gate_up, w_down -> act, dh, and dx,
// dw_gate_up, dw_down (each null when not wanted).
struct FfnParams {
  const int32_t *counts;         // [E] rows per expert, or null (cap each)
  WsHeader *hdr;
  float *part;                   // scratch, see FfnScratch
  void *row_maps;
  int E, cap, H, I;
  const uint16_t *x;             // [E, cap, H]
  const uint16_t *w_gate_up;     // [E, 2I, H]
  const uint16_t *w_down;        // [E, H, I]
  uint16_t *h;                   // [E, cap, 2I] gate | up
  uint16_t *act;                 // [E, cap, I]
  uint16_t *y;                   // [E, cap, H]
  const uint16_t *dy;            // [E, cap, H]
  uint16_t *dh;                  // [E, cap, 2I]
  uint16_t *dx;                  // [E, cap, H]
  uint16_t *dw_gate_up;          // [E, 2I, H]
  uint16_t *dw_down;             // [E, H, I]
};

// Scratch past the plan's part of the workspace, of any content between calls:
// the partial sums of split contractions, then the backward pass's tensor maps.
struct FfnScratch {
  size_t maps_off, total;
};
FfnScratch ffn_scratch(int64_t E, int64_t cap, int64_t H, int64_t I);

cudaError_t launch_ffn(const FfnParams &p, cudaStream_t stream);
cudaError_t launch_ffn_backward(const FfnParams &p, cudaStream_t stream);

}  // namespace moe
