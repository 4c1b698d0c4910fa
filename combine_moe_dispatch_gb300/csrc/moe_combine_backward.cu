// moe_combine_backward.cu -- the combine's backward pass, down to the
// router's logits.
//
// What it computes, for token g with gradient dy[g] and its routed entries k
// (row (e, s) = (idx[g,k], slot_of[g,k]) of the experts' outputs):
//   d_expert_y[e][s] = w[g,k] dy[g]
//   d_weights[g,k]   = <dy[g], expert_y[e][s]>
//   d_logits[g,idx]  = w[g,k] (d_weights[g,k] - sum_j w[g,j] d_weights[g,j])
// The last line is the softmax's backward pass over the K chosen logits, with
// d_weights = 0 for an entry that was left out afterwards (slot_of = -1): its
// logit is in the softmax's denominator and gets -w sum_j w_j d_weights_j.
// The logits that were not chosen get 0.
//
// How: WPT warps share a token.  Each lane reads 16 bytes of dy once and, for
// a group of KG entries, the same 16 bytes of every expert row, so that KG x U
// loads are in flight before the first product; it writes w dy to the same
// rows as it goes.  One pass: every byte is read and written once.  The dot
// products stay in registers (binary32, one accumulator per entry and lane),
// are summed over the lanes by shuffles and over the warps through shared
// memory, always in the same order.
#include <cuda_bf16.h>

#include "moe_train.cuh"

namespace moe {

constexpr int kBackThreads = 256;
constexpr int kBackWarps = kBackThreads / 32;

namespace {

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}

template <int KG, int U, int WPT, int MINB>
__global__ void __launch_bounds__(kBackThreads, MINB)
combine_backward_kernel(CombineBackwardParams p) {
  constexpr int kTokens = kBackWarps / WPT;       // tokens per block at a time
  constexpr unsigned kFull = 0xFFFFFFFFu;
  __shared__ float s_dot[kBackWarps][kMaxTopK];
  __shared__ int32_t s_status;
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
  const int sub = warp % WPT;                     // this warp among its token's
  const int cpr = p.H / 8;                        // 16-byte chunks per row
  pdl_wait_for_previous();
  if (threadIdx.x == 0) s_status = read_status(p.hdr);
  __syncthreads();
  if (s_status != MOE_OK) return;
  for (int64_t g0 = (int64_t)blockIdx.x * kTokens; g0 < p.N; g0 += (int64_t)gridDim.x * kTokens) {
    const int64_t g = g0 + warp / WPT;
    const bool on = g < p.N;
    int e_l = -1, s_l = -1;
    float w_l = 0.0f;
    if (on && lane < p.K) {
      e_l = __ldg(p.topk_idx + g * p.K + lane);
      s_l = __ldg(p.slot_of + g * p.K + lane);
      w_l = __ldg(p.topk_weights + g * p.K + lane);
    }
    const bool routed = on && lane < p.K && s_l != -1;
    const bool e_ok = e_l >= 0 && e_l < p.E;
    const bool ok = routed && e_ok && s_l >= 0 && s_l < p.cap;
    if (sub == 0 && routed && !ok)
      report_status(p.hdr, e_ok ? MOE_ERR_CAPACITY : MOE_ERR_BAD_EXPERT);
    const unsigned okmask = __ballot_sync(kFull, ok);
    const bool left_out = on && lane < p.K && s_l == -1 && e_ok;
    const unsigned chosen = okmask | __ballot_sync(kFull, left_out);
    for (int kb = 0; kb < p.K; kb += KG) {
      float dot[KG];
      int64_t off[KG];
      float w[KG];
      bool use[KG];
#pragma unroll
      for (int j = 0; j < KG; ++j) {
        const int k = kb + j;
        const int e = __shfl_sync(kFull, e_l, k & 31), s = __shfl_sync(kFull, s_l, k & 31);
        w[j] = __shfl_sync(kFull, w_l, k & 31);
        use[j] = k < p.K && ((okmask >> (k & 31)) & 1u);
        off[j] = use[j] ? ((int64_t)e * p.cap + s) * p.H : 0;
        dot[j] = 0.0f;
      }
      if (on)
        for (int c0 = sub * 32 * U + lane; c0 < cpr; c0 += WPT * 32 * U) {
          uint4 dy[U], v[U][KG];
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int c = c0 + 32 * u;
            dy[u] = c < cpr ? __ldg(reinterpret_cast<const uint4 *>(p.d_y + g * p.H) + c)
                            : make_uint4(0, 0, 0, 0);
#pragma unroll
            for (int j = 0; j < KG; ++j)
              v[u][j] = use[j] && c < cpr
                            ? __ldcs(reinterpret_cast<const uint4 *>(p.expert_y + off[j]) + c)
                            : make_uint4(0, 0, 0, 0);
          }
#pragma unroll
          for (int u = 0; u < U; ++u) {
            const int c = c0 + 32 * u;
            const uint32_t d[4] = {dy[u].x, dy[u].y, dy[u].z, dy[u].w};
#pragma unroll
            for (int j = 0; j < KG; ++j) {
              const uint32_t y[4] = {v[u][j].x, v[u][j].y, v[u][j].z, v[u][j].w};
              uint32_t o[4];
#pragma unroll
              for (int i = 0; i < 4; ++i) {
                const float dl = bf16_lo(d[i]), dh = bf16_hi(d[i]);
                dot[j] = fmaf(dl, bf16_lo(y[i]), dot[j]);
                dot[j] = fmaf(dh, bf16_hi(y[i]), dot[j]);
                o[i] = pack2(w[j] * dl, w[j] * dh);
              }
              if (use[j] && c < cpr)
                __stcs(reinterpret_cast<uint4 *>(p.d_expert_y + off[j]) + c,
                       make_uint4(o[0], o[1], o[2], o[3]));
            }
          }
        }
#pragma unroll
      for (int j = 0; j < KG; ++j) {
        float v = dot[j];
#pragma unroll
        for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(kFull, v, d);
        if (lane == 0 && kb + j < p.K) s_dot[warp][kb + j] = v;
      }
    }
    if (WPT == 1) __syncwarp();
    else __syncthreads();
    // the token's first warp: lane k has entry k
    if (on && p.d_logits)
      for (int e = sub * 32 + lane; e < p.E; e += WPT * 32) p.d_logits[g * p.E + e] = 0.0f;
    if (on && sub == 0) {
      float dw = 0.0f;
      if (ok)
        for (int i = 0; i < WPT; ++i) dw += s_dot[warp + i][lane];
      if (lane < p.K) p.d_weights[g * p.K + lane] = dw;
      if (p.d_logits) {
        // Entries of the softmax: the routed ones, and those left out of a token
        // that has others.  A token with nothing routed (padding, say) has y = 0
        // whatever its logits are: its weights may be anything, and count as 0.
        const float wk = ok || (left_out && okmask != 0u) ? w_l : 0.0f;
        float mean = 0.0f;
        for (int k = 0; k < p.K; ++k) {
          const float term = __shfl_sync(kFull, wk, k), dk = __shfl_sync(kFull, dw, k);
          if ((okmask >> k) & 1u) mean = fmaf(term, dk, mean);
        }
        // an expert chosen twice gets the sum of its entries
        const float own = wk * (dw - mean);
        float sum = 0.0f;
        for (int k = 0; k < p.K; ++k) {
          const int ek = __shfl_sync(kFull, e_l, k);
          const float dk = __shfl_sync(kFull, own, k);
          if (((chosen >> k) & 1u) && ek == e_l) sum += dk;
        }
        s_dot[warp][lane] = sum;                  // written after the row's zeros, below
      }
    }
    if (p.d_logits) {
      if (WPT == 1) __syncwarp();
      else __syncthreads();
      if (sub == 0 && (ok || left_out)) p.d_logits[g * p.E + e_l] = s_dot[warp][lane];
    }
    // s_dot is written again in the next round
    if (WPT == 1) __syncwarp();
    else __syncthreads();
  }
}

template <int KG, int U, int WPT, int MINB>
cudaError_t launch_variant(const CombineBackwardParams &p, cudaStream_t stream) {
  const auto kern = combine_backward_kernel<KG, U, WPT, MINB>;
  const int grid = persistent_grid((const void *)kern, kBackThreads, (int64_t)p.N * WPT);
  return launch_after_previous(kern, grid, kBackThreads, p, stream);
}

// Rows of up to 2048 elements take one warp per token, longer ones the block's
// 8 warps.  Measured, one warp and eight, us:
//   K  H      16 tokens   64          256         1024         8192
//   2  256    2.5  2.5    2.5  2.5    2.7  2.7    3.0  4.8     7.3  28.4
//   2  2048   4.2  2.5    4.3  2.6    4.4  2.8    6.6  6.6    29.3  39.2
//   8  256    3.9  3.1    3.9  3.2    4.0  3.5    4.2  11.2   17.4  75.5
//   8  1024   6.1  3.3    6.2  3.3    6.4  3.9    9.9  14.1   50.4  91.0
//   8  2048   8.8  3.7    8.9  3.7    9.1  4.5   16.8  16.5   95.6  113.7
//   8  7168   128 tokens: 31.6  9.1                          327   311
// The rule is made for tokens that fill the SMs; up to a few hundred eight warps
// would be faster at every H from 1024 on.
template <int KG, int U, int MINB>
cudaError_t launch_rows(const CombineBackwardParams &p, cudaStream_t stream) {
  if (p.H / 8 > 256) return launch_variant<KG, U, kBackWarps, MINB>(p, stream);
  return launch_variant<KG, U, 1, MINB>(p, stream);
}

}  // namespace

// Entries loaded at a time, chunks per lane and resident blocks per SM, by K.
// Measured: K = 2, 4096 tokens, H = 4096: 2 chunks at 4 blocks 29.3 us, 1 at 4
// 31.9, 4 at 3 42.2.  K = 4, 1024 tokens, H = 2048: 3 blocks 10.7 us, 2 blocks
// 11.9 (eight warps per token).  K = 8, 8192 tokens, H = 7168 (1.9 GB): 1 chunk
// at 2 blocks 311 us, 6.45 TB/s, 95 % of the measured bandwidth; 2 chunks 351,
// 3 blocks (80 registers, which spill) 358.
cudaError_t launch_combine_backward(const CombineBackwardParams &p, cudaStream_t stream) {
  if (p.K <= 2) return launch_rows<2, 2, 4>(p, stream);
  if (p.K <= 4) return launch_rows<4, 2, 3>(p, stream);
  return launch_rows<8, 1, 2>(p, stream);
}

}  // namespace moe
