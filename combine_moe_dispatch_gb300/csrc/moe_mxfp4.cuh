// moe_mxfp4.cuh -- MXFP4: the layout of its arrays, its conversions, and the
// parameters of the kernels that quantise.
#pragma once

#include "moe_common.cuh"

namespace moe {

// Scale bytes stand in tiles of 128 rows x 4 blocks of 32, 512 bytes each, the
// order in which a copy into tensor memory takes them: lane r of the copy's 32
// gets the 16 bytes of rows r, r + 32, r + 64 and r + 96, 4 blocks each.
constexpr int kScaleTileRows = 128;
constexpr int kScaleTileBytes = 512;

struct ScaleLayout {
  int row_tiles, block_tiles;
};
inline ScaleLayout scale_layout(int64_t rows, int64_t cols) {
  return ScaleLayout{(int)((rows + kScaleTileRows - 1) / kScaleTileRows), (int)((cols + 127) / 128)};
}
inline size_t scale_bytes(int64_t experts, int64_t rows, int64_t cols) {
  const ScaleLayout l = scale_layout(rows, cols);
  return (size_t)experts * l.row_tiles * l.block_tiles * kScaleTileBytes;
}

// MXFP4 rows in memory.
struct Mxfp4Rows {
  uint8_t *q;                  // [E, rows, cols/2]
  uint8_t *scale;              // [E, row tiles, block tiles, 512]
  int rows, cols;
  int row_tiles, block_tiles;
  int gate;                    // rows of the gate and of up, 64 of each in a tile; 0: rows in order
};

struct QuantParams {
  const uint16_t *src;         // [E, rows, cols] bf16
  const int32_t *counts;       // [E] rows per expert, or null (all)
  const WsHeader *hdr;         // of the plan behind the counts, or null
  Mxfp4Rows out;
  int E;
};

struct DequantParams {
  Mxfp4Rows in;                // q and scale are read only
  const int32_t *counts;
  const WsHeader *hdr;
  uint16_t *out;               // [E, rows, cols] bf16
  int E;
};

struct DispatchMxfp4Params {
  const uint16_t *x;           // [N, H] bf16
  const int32_t *topk_idx;
  const int32_t *slot_of;
  WsHeader *hdr;
  Mxfp4Rows out;               // rows = cap, cols = H
  int N, E, K;
};

// The experts' feed-forward on MXFP4 operands.
struct FfnMxfp4Params {
  const int32_t *counts;       // [E] rows per expert, or null (cap each)
  WsHeader *hdr;
  float *part;                 // scratch: partial sums of split contractions
  int E, cap, H, I;
  const uint8_t *x, *x_scale;                  // rows [E, cap, H]
  const uint8_t *w_gate_up, *w_gate_up_scale;  // rows [E, 2I, H], the scales 64 and 64
  const uint8_t *w_down, *w_down_scale;        // rows [E, H, I]
  uint8_t *act, *act_scale;                    // rows [E, cap, I]
  uint16_t *y;                                 // [E, cap, H] bf16
};
size_t ffn_mxfp4_scratch(int64_t E, int64_t cap, int64_t H, int64_t I);

cudaError_t launch_ffn_mxfp4(const FfnMxfp4Params &p, cudaStream_t stream);
cudaError_t launch_quant_mxfp4(const QuantParams &p, cudaStream_t stream);
cudaError_t launch_dequant_mxfp4(const DequantParams &p, cudaStream_t stream);
cudaError_t launch_dispatch_mxfp4(const DispatchMxfp4Params &p, cudaStream_t stream);

#ifdef __CUDACC__
// Where the 4 scale bytes of (row, blocks 4 j to 4 j + 3) stand, from the
// expert's first tile.
__device__ __forceinline__ int64_t scale_word(const Mxfp4Rows &m, int row, int j) {
  if (m.gate) {
    const int up = row >= m.gate, f = row - (up ? m.gate : 0);
    row = (f >> 6) * 128 + up * 64 + (f & 63);
  }
  return ((int64_t)(row >> 7) * m.block_tiles + j) * kScaleTileBytes + (row & 31) * 16 + ((row >> 5) & 3) * 4;
}
__device__ __forceinline__ int64_t expert_tiles(const Mxfp4Rows &m, int e) {
  return (int64_t)e * m.row_tiles * m.block_tiles * kScaleTileBytes;
}

// The biased exponent of X = 2^(floor(log2 amax) - 2), from amax's own exponent
// field; never below 2^-127.  A block with an infinity or a NaN gets 255, NaN.
__device__ __forceinline__ uint32_t mx_scale(uint32_t exponent) {
  return exponent == 255u ? 255u : (exponent > 2u ? exponent - 2u : 0u);
}
// 1 / X, exact; for a block that is NaN 0, so that its elements are 0.
__device__ __forceinline__ float mx_inverse(uint32_t scale) {
  return scale == 255u ? 0.0f : __uint_as_float((254u - scale) << 23);
}
// 8 values -> 8 E2M1, 4 bits each, the first lowest: to nearest, ties to even, at
// most 6 in magnitude.
__device__ __forceinline__ uint32_t e2m1x8(const float (&f)[8]) {
  uint32_t r;
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 a, %2, %1;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 b, %4, %3;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 c, %6, %5;\n\t"
      "cvt.rn.satfinite.e2m1x2.f32 d, %8, %7;\n\t"
      "mov.b32 %0, {a, b, c, d};\n\t}"
      : "=r"(r)
      : "f"(f[0]), "f"(f[1]), "f"(f[2]), "f"(f[3]), "f"(f[4]), "f"(f[5]), "f"(f[6]), "f"(f[7]));
  return r;
}
#endif

}  // namespace moe
