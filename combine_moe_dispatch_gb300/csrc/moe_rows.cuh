// moe_rows.cuh -- the populated rows of the experts' padded buffers, numbered
// through: shared by the kernels that work on those rows alone.
#pragma once

#include "moe_common.cuh"

#ifdef __CUDACC__
namespace moe {

// Exclusive prefix of clamp(count[e], 0, cap) over e into out[0..E], by the
// whole block of THREADS (any E).  Ends with a block barrier.
template <int THREADS>
__device__ void count_prefix(const int32_t *count, int E, int cap, int32_t *out) {
  __shared__ int32_t s_warp[THREADS / 32];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int per = (E + THREADS - 1) / THREADS;     // consecutive entries per thread
  const int e0 = tid * per;
  int local = 0;
  for (int i = 0; i < per; ++i) {
    const int e = e0 + i;
    if (e < E) local += min(max(__ldg(count + e), 0), cap);
  }
  int incl = local;
#pragma unroll
  for (int off = 1; off < 32; off <<= 1) {
    const int v = __shfl_up_sync(0xFFFFFFFFu, incl, off);
    if (lane >= off) incl += v;
  }
  if (lane == 31) s_warp[warp] = incl;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < warp; ++w) before += s_warp[w];
  int run = before + incl - local;
  for (int i = 0; i < per; ++i) {
    const int e = e0 + i;
    if (e < E) {
      out[e] = run;
      run += min(max(__ldg(count + e), 0), cap);
    }
  }
  if (tid == THREADS - 1) out[E] = run;
  __syncthreads();
}

// The expert whose populated rows hold row number rg: the last e with
// prefix[e] <= rg.
__device__ __forceinline__ int populated_expert(const int32_t *s_prefix, int E, int rg) {
  int lo = 0, hi = E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (s_prefix[mid] <= rg) lo = mid;
    else hi = mid;
  }
  return lo;
}

}  // namespace moe
#endif
