// moe_norm.cu -- root-mean-square norm of the hidden states, with the
// residual's addition and an output in 8 bits, and its backward pass.
//
// What it computes, for each row of H elements:
//   s = bf16(x + residual)                    (s = x without a residual)
//   y = s rstd gain,  rstd = 1 / sqrt(mean(s^2) + eps)
// y rounded to bf16 and, from the same unrounded values, to E4M3 with one scale
// per 128 elements (amax/448, the rule of the fp8 dispatch; NaN if one of them is); and
//   u = s rstd,  g = dy gain
//   d_x = rstd (g - u mean(g u)) + d_sum,     d_gain = sum over rows of dy u
// from dy, the gradient d_sum that arrives at s by the residual stream, and s.
// The norm is that of the rounded s, which is what the backward pass reads:
// what is differentiated is what was computed.  Sums are binary32.
//
// How: one pass over the data.  WPR warps share a row, each lane has C chunks of
// 16 bytes of it in registers between the sum of squares and the result, so that
// every byte is read and written once.  A block of 8 warps (of 16 for rows of 8193
// to 16384 elements) takes 8 / WPR rows at a time from a grid that fills the SMs.
// Backward, a lane's columns are the same for all of its rows: their share of
// d_gain is summed in registers, joined over the block's warps in shared memory,
// stored once per block, and a second launch adds the blocks' shares, all in an
// order that depends on the sizes and the device alone.  Rows of more than 16384
// elements do not fit the registers: a block then reads its row twice (the second
// time from the caches; 2048 x 20480: forward 70 us, backward 134).
//
// What bounds it, measured on GB300 (copy 6.78 TB/s): memory.  8192 x 7168 with a
// residual and both outputs 88 us, 6.0 TB/s; backward with d_sum 84 us, of which
// the rows are 76 (6.2 TB/s) and adding 304 shares of 7168 columns 6.  Blocks
// per SM: 4 of 64 registers forward (3 of 80: 87.8 us, 5 of 48: 96.5), 2 of 128
// backward (1: 108 us, 3: 168, which spill).  One token: 2.0 us on the GPU, 4.2 through
// the binding.
#include <cuda_bf16.h>

#include "moe_norm.cuh"

namespace moe {

namespace {

constexpr int kNormThreads = 256;      // a block, but 512 for rows of 8193 to 16384 elements
constexpr int kNormWarps = kNormThreads / 32;
constexpr unsigned kFull = 0xFFFFFFFFu;

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ void unpack8(const uint4 &v, float (&f)[8]) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(w[i]);
    f[2 * i + 1] = bf16_hi(w[i]);
  }
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
  return make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]), pack_bf16(f[4], f[5]),
                    pack_bf16(f[6], f[7]));
}
__device__ __forceinline__ uint4 add8(const uint4 &a, const uint4 &b) {
  float x[8], r[8];
  unpack8(a, x);
  unpack8(b, r);
#pragma unroll
  for (int i = 0; i < 8; ++i) x[i] += r[i];
  return pack8(x);
}
__device__ __forceinline__ uint4 load16(const uint16_t *p, int64_t chunk) {
  return __ldcs(reinterpret_cast<const uint4 *>(p) + chunk);
}

// The gain's chunk, from the L1: kept in registers it costs resident blocks
// (8192 x 7168: forward 101 us, so 87; backward 109, so 84).
__device__ __forceinline__ uint4 load_gain(const uint16_t *gain, int c, int cpr) {
  return c < cpr ? __ldg(reinterpret_cast<const uint4 *>(gain) + c) : make_uint4(0, 0, 0, 0);
}

__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
  return v;
}
// The sum over a row's WPR warps, in the order of the warps.  `s` is used again
// two calls later: the barrier of the call between keeps the reads before it.
template <int WPR>
__device__ __forceinline__ float row_sum(float v, float *s, int warp) {
  v = warp_sum(v);
  if (WPR == 1) return v;
  if ((threadIdx.x & 31) == 0) s[warp] = v;
  __syncthreads();
  float t = 0.0f;
#pragma unroll
  for (int i = 0; i < WPR; ++i) t += s[warp / WPR * WPR + i];
  return t;
}

// Squares of elements below 2^-63 lose bits in binary32, and vanish below 2^-75.  With
// eps of 2^-90 or more that is below mean(s^2) + eps's rounding; a smaller eps (0 among
// them) leaves such a row to its own elements.  Then every row is first multiplied by
// a power of two, `lift`, that brings its largest magnitude to 1 to 2 (to 2^-7 at
// least, from bf16's subnormals), or stops where eps lift^2 is about 1.  That is
// exact, and with eps lift^2 for eps u and y are the same; the backward pass
// multiplies by lift once more.  Rows of 1 and more stay as they are (lift 1), so
// that all calls end at the same sum of squares.  eps is the launch's: every thread
// takes this branch, or none.  8192 x 7168, both outputs: 98.5 us, 88 with an ordinary
// eps; backward with d_sum 92 and 84.
constexpr float kSmallEps = 0x1p-90f;
__device__ __forceinline__ float row_lift(uint32_t most, float eps) {
  const int row = max((int)(most >> 7), 1) - 127;        // exponent of the largest magnitude
  const int half = eps > 0.0f ? ((int)(__float_as_uint(eps) >> 23) - 127) >> 1 : -126;
  return __uint_as_float((uint32_t)(127 - min(max(row, half), 0)) << 23);
}
__device__ __forceinline__ uint32_t most8(uint32_t m, const uint4 &v) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) m = max(m, max(w[i] & 0x7FFFu, w[i] >> 16 & 0x7FFFu));
  return m;
}
// The largest of a row's WPR warps.
template <int WPR>
__device__ __forceinline__ uint32_t row_most(uint32_t m, uint32_t *s, int warp) {
  m = __reduce_max_sync(kFull, m);
  if (WPR == 1) return m;
  __syncthreads();                           // the row before has been read
  if ((threadIdx.x & 31) == 0) s[warp] = m;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < WPR; ++i) m = max(m, s[warp / WPR * WPR + i]);
  return m;
}
// The row's chunks multiplied by its lift, which is returned; eps becomes eps lift^2.
template <int C, int WPR>
__device__ __forceinline__ float lift_row(uint4 (&v)[C], float &eps, uint32_t *s, int warp) {
  uint32_t m = 0;
#pragma unroll
  for (int u = 0; u < C; ++u) m = most8(m, v[u]);
  const float lift = row_lift(row_most<WPR>(m, s, warp), eps);
  eps = eps * lift * lift;
#pragma unroll
  for (int u = 0; u < C; ++u) {
    float f[8];
    unpack8(v[u], f);
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] *= lift;
    v[u] = pack8(f);
  }
  return lift;
}

// Largest |f| of a half-warp's 128 values, NaN if one of them is: one NaN in a row
// makes all of its y NaN, which the 8 bits have to say as the bf16 output does.  (The
// shared half_warp_amax passes over NaN.)  All 32 lanes call it.
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float half_warp_amax_nan(const float (&f)[8]) {
  float amax = fabsf(f[0]);
#pragma unroll
  for (int i = 1; i < 8; ++i) amax = max_nan(amax, fabsf(f[i]));
#pragma unroll
  for (int off = 8; off >= 1; off >>= 1) amax = max_nan(amax, __shfl_xor_sync(kFull, amax, off));
  return amax;
}

// A half-warp's 128 values -> E4M3 bytes and their scale; with a NaN among them
// the scale and every byte (0x7F, any sign) are NaN.  All 32 lanes call it.
__device__ __forceinline__ void store_fp8(const NormParams &p, int64_t row, int chunk, bool in, int nb,
                                          const float (&f)[8]) {
  const float amax = half_warp_amax_nan(f);
  const bool fast = amax >= 0x1p-120f && amax <= 3.4028234e38f;
  const float scale[1] = {fast ? div448_fast(amax) : __fdiv_rn(amax, 448.0f)};
  const bool zero[1] = {amax == 0.0f};
  const float r[1] = {zero[0] ? 1.0f : __frcp_rn(scale[0])};
  const float v[1][8] = {{f[0], f[1], f[2], f[3], f[4], f[5], f[6], f[7]}};
  uint2 q[1];
  quantise_blocks<1>(v, scale, r, zero, q);
  if (!in) return;
  *reinterpret_cast<uint2 *>(p.y_q + row * p.H + (int64_t)chunk * 8) = q[0];
  if ((chunk & 15) == 0) {
    const int blk = chunk >> 4;
    p.y_scale[p.scale_t ? (int64_t)blk * p.N + row : row * nb + blk] = scale[0];
  }
}

template <int C, int WPR, bool RES, bool FP8, int WARPS = kNormWarps>
__global__ void __launch_bounds__(32 * WARPS, C == 1 ? 6 : 32 / WARPS)
norm_kernel(NormParams p) {
  constexpr int kRows = WARPS / WPR;
  __shared__ float s_sum[2][WARPS];
  __shared__ uint32_t s_most[WARPS];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c0 = (warp % WPR) * 32 + lane, cpr = p.H / 8, nb = (p.H + 127) / 128;
  pdl_wait_for_previous();
  int buf = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * kRows; row0 < p.N; row0 += (int64_t)gridDim.x * kRows) {
    const int64_t row = row0 + warp / WPR;
    uint4 s[C];
    if (RES) {
      uint4 r[C];
#pragma unroll
      for (int u = 0; u < C; ++u) {
        const int c = c0 + u * WPR * 32;
        const bool in = row < p.N && c < cpr;
        s[u] = in ? load16(p.x, row * cpr + c) : make_uint4(0, 0, 0, 0);
        r[u] = in ? load16(p.residual, row * cpr + c) : make_uint4(0, 0, 0, 0);
      }
#pragma unroll
      for (int u = 0; u < C; ++u) {
        const int c = c0 + u * WPR * 32;
        s[u] = add8(s[u], r[u]);
        if (p.sum && row < p.N && c < cpr) reinterpret_cast<uint4 *>(p.sum)[row * cpr + c] = s[u];
      }
    } else {
#pragma unroll
      for (int u = 0; u < C; ++u) {
        const int c = c0 + u * WPR * 32;
        s[u] = row < p.N && c < cpr ? load16(p.x, row * cpr + c) : make_uint4(0, 0, 0, 0);
      }
    }
    float eps = p.eps;
    if (p.eps < kSmallEps) lift_row<C, WPR>(s, eps, s_most, warp);
    float sq = 0.0f;
#pragma unroll
    for (int u = 0; u < C; ++u) {
      float f[8];
      unpack8(s[u], f);
#pragma unroll
      for (int i = 0; i < 8; ++i) sq = fmaf(f[i], f[i], sq);
    }
    const float rstd = rsqrtf(row_sum<WPR>(sq, s_sum[buf], warp) / (float)p.H + eps);
    buf ^= 1;
#pragma unroll
    for (int u = 0; u < C; ++u) {
      const int c = c0 + u * WPR * 32;
      const bool in = row < p.N && c < cpr;
      float f[8], g[8];
      unpack8(s[u], f);
      unpack8(load_gain(p.gain, c, cpr), g);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = f[i] * rstd * g[i];
      if ((!FP8 || p.y) && in) reinterpret_cast<uint4 *>(p.y)[row * cpr + c] = pack8(f);
      if (FP8) store_fp8(p, row, c, in, nb, f);
    }
  }
}

// Rows of any length: a block reads its row twice.
template <bool RES, bool FP8>
__global__ void __launch_bounds__(kNormThreads)
norm_long_kernel(NormParams p) {
  __shared__ float s_sum[2][kNormWarps];
  __shared__ uint32_t s_most[kNormWarps];
  const int warp = threadIdx.x >> 5;
  const int cpr = p.H / 8, nb = (p.H + 127) / 128;
  pdl_wait_for_previous();
  int buf = 0;
  for (int64_t row = blockIdx.x; row < p.N; row += gridDim.x) {
    const auto read = [&](int c) {
      uint4 s = reinterpret_cast<const uint4 *>(p.x)[row * cpr + c];
      if (RES) s = add8(s, reinterpret_cast<const uint4 *>(p.residual)[row * cpr + c]);
      return s;
    };
    float lift = 1.0f;
    if (p.eps < kSmallEps) {
      uint32_t m = 0;
      for (int c = threadIdx.x; c < cpr; c += kNormThreads) m = most8(m, read(c));
      lift = row_lift(row_most<kNormWarps>(m, s_most, warp), p.eps);
    }
    float sq = 0.0f;
#pragma unroll 4
    for (int c = threadIdx.x; c < cpr; c += kNormThreads) {
      float f[8];
      unpack8(read(c), f);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float v = f[i] * lift;
        sq = fmaf(v, v, sq);
      }
    }
    const float rstd = rsqrtf(row_sum<kNormWarps>(sq, s_sum[buf], warp) / (float)p.H + p.eps * lift * lift);
    buf ^= 1;
    for (int cb = 0; cb < cpr; cb += kNormThreads) {      // all lanes, for the half-warps' maxima
      const int c = cb + threadIdx.x;
      const bool in = c < cpr;
      float f[8], g[8];
      const uint4 s = in ? read(c) : make_uint4(0, 0, 0, 0);
      unpack8(s, f);
      unpack8(in ? __ldg(reinterpret_cast<const uint4 *>(p.gain) + c) : make_uint4(0, 0, 0, 0), g);
#pragma unroll
      for (int i = 0; i < 8; ++i) f[i] = f[i] * lift * rstd * g[i];
      if (RES && p.sum && in) reinterpret_cast<uint4 *>(p.sum)[row * cpr + c] = s;
      if ((!FP8 || p.y) && in) reinterpret_cast<uint4 *>(p.y)[row * cpr + c] = pack8(f);
      if (FP8) store_fp8(p, row, c, in, nb, f);
    }
  }
}

// LIFT: eps is below kSmallEps.  A variant of its own, since this kernel has no
// register left: with the branch and the factor in the one kernel 2048 x 16384 took 60.8
// us, so 53.5; 8192 x 4096 51.8, so 49.6.
template <int C, int WPR, bool DSUM, bool LIFT, int WARPS = kNormWarps>
__global__ void __launch_bounds__(32 * WARPS, 16 / WARPS)
norm_backward_kernel(NormBackwardParams p) {
  constexpr int kRows = WARPS / WPR;
  __shared__ float s_sum[2][2][WARPS];
  __shared__ uint32_t s_most[LIFT ? WARPS : 1];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int c0 = (warp % WPR) * 32 + lane, cpr = p.H / 8;
  pdl_wait_for_previous();
  float acc[C][8];
#pragma unroll
  for (int u = 0; u < C; ++u)
#pragma unroll
    for (int i = 0; i < 8; ++i) acc[u][i] = 0.0f;
  int buf = 0;
  for (int64_t row0 = (int64_t)blockIdx.x * kRows; row0 < p.N; row0 += (int64_t)gridDim.x * kRows) {
    const int64_t row = row0 + warp / WPR;
    uint4 s[C], dy[C], ds[C];
#pragma unroll
    for (int u = 0; u < C; ++u) {
      const int c = c0 + u * WPR * 32;
      const bool in = row < p.N && c < cpr;
      s[u] = in ? load16(p.sum, row * cpr + c) : make_uint4(0, 0, 0, 0);
      dy[u] = in ? load16(p.d_y, row * cpr + c) : make_uint4(0, 0, 0, 0);
      if (DSUM) ds[u] = in ? load16(p.d_sum, row * cpr + c) : make_uint4(0, 0, 0, 0);
    }
    float eps = p.eps, lift = 1.0f;
    if (LIFT) lift = lift_row<C, WPR>(s, eps, s_most, warp);
    float sq = 0.0f, dot = 0.0f;
#pragma unroll
    for (int u = 0; u < C; ++u) {
      float f[8], d[8], g[8];
      unpack8(s[u], f);
      unpack8(dy[u], d);
      unpack8(load_gain(p.gain, c0 + u * WPR * 32, cpr), g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        sq = fmaf(f[i], f[i], sq);
        dot = fmaf(d[i] * g[i], f[i], dot);
      }
    }
    // both sums behind one barrier
    sq = warp_sum(sq);
    dot = warp_sum(dot);
    if (WPR > 1) {
      if (lane == 0) {
        s_sum[buf][0][warp] = sq;
        s_sum[buf][1][warp] = dot;
      }
      __syncthreads();
      sq = dot = 0.0f;
#pragma unroll
      for (int i = 0; i < WPR; ++i) {
        sq += s_sum[buf][0][warp / WPR * WPR + i];
        dot += s_sum[buf][1][warp / WPR * WPR + i];
      }
      buf ^= 1;
    }
    const float rstd = rsqrtf(sq / (float)p.H + eps);
    const float mean = dot * rstd / (float)p.H;             // of g u
#pragma unroll
    for (int u = 0; u < C; ++u) {
      const int c = c0 + u * WPR * 32;
      float f[8], d[8], g[8], e[8];
      unpack8(s[u], f);
      unpack8(dy[u], d);
      unpack8(load_gain(p.gain, c0 + u * WPR * 32, cpr), g);
      if (DSUM) unpack8(ds[u], e);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float un = f[i] * rstd;
        if (row < p.N) acc[u][i] = fmaf(d[i], un, acc[u][i]);
        f[i] = d[i] * g[i] - un * mean;
        if (LIFT) f[i] *= lift;
        f[i] *= rstd;
        if (DSUM) f[i] += e[i];
      }
      if (row < p.N && c < cpr) reinterpret_cast<uint4 *>(p.d_x)[row * cpr + c] = pack8(f);
    }
  }
  // the block's share of d_gain: its row groups' in their order
  if (kRows > 1) {
    __shared__ float s_acc[kRows > 1 ? kRows - 1 : 1][WPR * 32 * C * 8];
    const int group = warp / WPR, at = c0 * 8;
    if (group > 0)
#pragma unroll
      for (int u = 0; u < C; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) s_acc[group - 1][u * WPR * 256 + at + i] = acc[u][i];
    __syncthreads();
    if (group > 0) return;
#pragma unroll
    for (int k = 0; k < kRows - 1; ++k)
#pragma unroll
      for (int u = 0; u < C; ++u)
#pragma unroll
        for (int i = 0; i < 8; ++i) acc[u][i] += s_acc[k][u * WPR * 256 + at + i];
  }
#pragma unroll
  for (int u = 0; u < C; ++u) {
    const int c = c0 + u * WPR * 32;
    if (c < cpr) {
      float4 *q = reinterpret_cast<float4 *>(p.part + (int64_t)blockIdx.x * p.H) + 2 * c;
      q[0] = make_float4(acc[u][0], acc[u][1], acc[u][2], acc[u][3]);
      q[1] = make_float4(acc[u][4], acc[u][5], acc[u][6], acc[u][7]);
    }
  }
}

// Rows of any length: a block reads its row twice and keeps its share of
// d_gain in the workspace.
template <bool DSUM>
__global__ void __launch_bounds__(kNormThreads)
norm_backward_long_kernel(NormBackwardParams p) {
  __shared__ float s_sum[2][2][kNormWarps];
  __shared__ uint32_t s_most[kNormWarps];
  const int warp = threadIdx.x >> 5, cpr = p.H / 8;
  float4 *part = reinterpret_cast<float4 *>(p.part + (int64_t)blockIdx.x * p.H);
  pdl_wait_for_previous();
  int buf = 0;
  for (int64_t row = blockIdx.x; row < p.N; row += gridDim.x) {
    const uint4 *s = reinterpret_cast<const uint4 *>(p.sum) + row * cpr;
    const uint4 *dy = reinterpret_cast<const uint4 *>(p.d_y) + row * cpr;
    const uint4 *gain = reinterpret_cast<const uint4 *>(p.gain);
    float lift = 1.0f;
    if (p.eps < kSmallEps) {
      uint32_t m = 0;
      for (int c = threadIdx.x; c < cpr; c += kNormThreads) m = most8(m, s[c]);
      lift = row_lift(row_most<kNormWarps>(m, s_most, warp), p.eps);
    }
    float sq = 0.0f, dot = 0.0f;
#pragma unroll 4
    for (int c = threadIdx.x; c < cpr; c += kNormThreads) {
      float f[8], d[8], g[8];
      unpack8(s[c], f);
      unpack8(dy[c], d);
      unpack8(__ldg(gain + c), g);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float v = f[i] * lift;
        sq = fmaf(v, v, sq);
        dot = fmaf(d[i] * g[i], v, dot);
      }
    }
    sq = row_sum<kNormWarps>(sq, s_sum[buf][0], warp);
    dot = row_sum<kNormWarps>(dot, s_sum[buf][1], warp);
    buf ^= 1;
    const float rstd = rsqrtf(sq / (float)p.H + p.eps * lift * lift);
    const float mean = dot * rstd / (float)p.H;
    for (int c = threadIdx.x; c < cpr; c += kNormThreads) {
      float f[8], d[8], g[8], e[8];
      unpack8(s[c], f);
      unpack8(dy[c], d);
      unpack8(__ldg(gain + c), g);
      if (DSUM) unpack8(reinterpret_cast<const uint4 *>(p.d_sum)[row * cpr + c], e);
      float4 a[2] = {make_float4(0, 0, 0, 0), make_float4(0, 0, 0, 0)};
      if (row != (int64_t)blockIdx.x) {
        a[0] = part[2 * c];
        a[1] = part[2 * c + 1];
      }
      float *acc = reinterpret_cast<float *>(a);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float un = f[i] * lift * rstd;
        acc[i] = fmaf(d[i], un, acc[i]);
        f[i] = rstd * ((d[i] * g[i] - un * mean) * lift);
        if (DSUM) f[i] += e[i];
      }
      part[2 * c] = a[0];
      part[2 * c + 1] = a[1];
      reinterpret_cast<uint4 *>(p.d_x)[row * cpr + c] = pack8(f);
    }
  }
}

struct GainParams {
  const float *part;           // [parts][H]
  float *d_gain;               // [H]
  int parts, H;
};
constexpr int kGainThreads = 1024;

// 32 columns a block: each warp adds every 32nd block's share, then the warps'
// sums are added in their order.
__global__ void __launch_bounds__(kGainThreads)
norm_gain_kernel(GainParams p) {
  constexpr int kWarps = kGainThreads / 32;
  __shared__ float s[kWarps][33];
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int col = blockIdx.x * 32 + lane;
  pdl_wait_for_previous();
  float v = 0.0f;
  if (col < p.H) {
#pragma unroll 8
    for (int i = warp; i < p.parts; i += kWarps) v += __ldg(p.part + (int64_t)i * p.H + col);
  }
  s[warp][lane] = v;
  __syncthreads();
  if (warp == 0 && col < p.H) {
    float t = 0.0f;
#pragma unroll
    for (int i = 0; i < kWarps; ++i) t += s[i][lane];
    p.d_gain[col] = t;
  }
}

template <int C, int WPR, bool RES, bool FP8, int WARPS = kNormWarps>
cudaError_t launch_rows(const NormParams &p, cudaStream_t stream) {
  const auto kern = norm_kernel<C, WPR, RES, FP8, WARPS>;
  return launch_after_previous(kern, persistent_grid((const void *)kern, 32 * WARPS, (int64_t)p.N * WPR),
                               32 * WARPS, p, stream);
}

template <bool RES, bool FP8>
cudaError_t launch_width(const NormParams &p, cudaStream_t stream) {
  const int cpr = p.H / 8;
  if (cpr <= 32) return launch_rows<1, 1, RES, FP8>(p, stream);
  if (cpr <= 64) return launch_rows<2, 1, RES, FP8>(p, stream);
  if (cpr <= 128) return launch_rows<4, 1, RES, FP8>(p, stream);
  if (cpr <= 256) return launch_rows<4, 2, RES, FP8>(p, stream);
  if (cpr <= 512) return launch_rows<4, 4, RES, FP8>(p, stream);
  if (cpr <= 1024) return launch_rows<4, 8, RES, FP8>(p, stream);
  if (cpr <= 2048) return launch_rows<4, 16, RES, FP8, 16>(p, stream);
  const auto kern = norm_long_kernel<RES, FP8>;
  return launch_after_previous(
      kern, persistent_grid((const void *)kern, kNormThreads, (int64_t)p.N * kNormWarps), kNormThreads, p,
      stream);
}

int backward_blocks(const void *kern, int threads, int64_t warps) {
  const int g = persistent_grid(kern, threads, warps);
  return g < kNormMaxBlocks ? g : kNormMaxBlocks;
}

template <int C, int WPR, bool DSUM, int WARPS = kNormWarps>
cudaError_t launch_backward_rows(const NormBackwardParams &p, int &parts, cudaStream_t stream) {
  const auto kern = p.eps < kSmallEps ? norm_backward_kernel<C, WPR, DSUM, true, WARPS>
                                      : norm_backward_kernel<C, WPR, DSUM, false, WARPS>;
  parts = backward_blocks((const void *)kern, 32 * WARPS, (int64_t)p.N * WPR);
  return launch_after_previous(kern, parts, 32 * WARPS, p, stream);
}

template <bool DSUM>
cudaError_t launch_backward_width(const NormBackwardParams &p, int &parts, cudaStream_t stream) {
  const int cpr = p.H / 8;
  if (cpr <= 32) return launch_backward_rows<1, 1, DSUM>(p, parts, stream);
  if (cpr <= 64) return launch_backward_rows<2, 1, DSUM>(p, parts, stream);
  if (cpr <= 128) return launch_backward_rows<4, 1, DSUM>(p, parts, stream);
  if (cpr <= 256) return launch_backward_rows<4, 2, DSUM>(p, parts, stream);
  if (cpr <= 512) return launch_backward_rows<4, 4, DSUM>(p, parts, stream);
  if (cpr <= 1024) return launch_backward_rows<4, 8, DSUM>(p, parts, stream);
  if (cpr <= 2048) return launch_backward_rows<4, 16, DSUM, 16>(p, parts, stream);
  const auto kern = norm_backward_long_kernel<DSUM>;
  parts = backward_blocks((const void *)kern, kNormThreads, (int64_t)p.N * kNormWarps);
  return launch_after_previous(kern, parts, kNormThreads, p, stream);
}

}  // namespace

cudaError_t launch_norm(const NormParams &p, cudaStream_t stream) {
  if (p.y_q) return p.residual ? launch_width<true, true>(p, stream) : launch_width<false, true>(p, stream);
  return p.residual ? launch_width<true, false>(p, stream) : launch_width<false, false>(p, stream);
}

cudaError_t launch_norm_backward(const NormBackwardParams &p, float *d_gain, cudaStream_t stream) {
  GainParams g;
  g.part = p.part;
  g.d_gain = d_gain;
  g.H = p.H;
  g.parts = 0;
  if (p.N > 0) {
    const cudaError_t e = p.d_sum ? launch_backward_width<true>(p, g.parts, stream)
                                  : launch_backward_width<false>(p, g.parts, stream);
    if (e != cudaSuccess) return e;
  }
  return launch_after_previous(norm_gain_kernel, (p.H + 31) / 32, kGainThreads, g, stream);
}

}  // namespace moe
