// moe_clip.cu -- global gradient norm over many tensors, and clipping.
//
// What it computes:
//   norm = sqrt(sum over all tensors and elements of g^2)
//   out  = g * min(1, max_norm / (norm + 1e-6)), in g's type
//
// How: the tensors are cut into chunks of 32 KB at 16-byte boundaries of
// their own addresses, and a persistent grid takes the chunks of up to
// kClipBatch tensors in turn (the table of tensors travels in the kernel's
// parameters, so nothing is copied or allocated).  The norm's kernel sums a
// chunk's squares in binary32 per thread (64 bf16 or 32 fp32 elements; in
// binary64 where they leave binary32's range) and everything above that in
// binary64; each block leaves one partial sum, and the last block to finish
// adds them in a fixed order, so that the norm does not depend on the order
// in which blocks run.  The second kernel scales; it
// takes the chunks in the opposite order, so that it begins with what the
// first one read last and the L2 (129 MB) still holds: of 344 MB it reads 264
// from memory, of 204 MB 125.  In place with a coefficient of 1 it writes nothing.
//
// Measured: 476 M gradients (1 GB, mostly bf16) 474 us, 1.01 GB read twice
// and written once at 6.4 TB/s, 94 % of the measured bandwidth; 300 tensors of
// 1000 to 4 M (344 MB) 171 us where the host's list does not take longer (it does
// through the Python binding: 190 us); up to 4 MB 7 us, two launches.  One cluster of 8
// blocks that does both in one launch took 11 us at 64 KB and 21 us at 2 MB
// (eight SMs read too slowly), and was not kept.
#include <cuda_bf16.h>

#include "moe_train.cuh"

namespace moe {

namespace {

constexpr int kClipThreads = 256;
constexpr int kGroupBytes = 16;
constexpr int kChunkGroups = 2048;            // 16-byte groups per chunk: 32 KB, 8 per thread
constexpr int kClipBatch = 512;               // tensors per launch
constexpr float kClipEps = 1e-6f;

struct ClipTensor {
  const void *grad;
  void *out;
  int64_t numel;
};

template <int BATCH>
struct ClipParams {
  ClipTensor t[BATCH];
  int64_t first[BATCH];                       // chunks before this tensor
  uint32_t f32[BATCH / 32];                   // bit i: tensor i is fp32
  int num;
  int64_t chunks;
  ClipHeader *hdr;
  double *partial;                            // [grid]
  float *norm;
  float max_norm;
  int begin, end;                             // first and last batch of the call
};

// The chunk's tensor: the last one whose first chunk is not after it.
template <int BATCH>
__device__ __forceinline__ int tensor_of(const ClipParams<BATCH> &p, int64_t chunk) {
  int lo = 0, hi = p.num;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (p.first[mid] <= chunk) lo = mid;
    else hi = mid;
  }
  return lo;
}

// A chunk's place: groups [g0, g1) of 16 bytes from the aligned address at
// or below the tensor's first element, which is element `lead` of group 0.
template <typename T>
struct Chunk {
  static constexpr int VE = kGroupBytes / (int)sizeof(T);
  const T *base;
  int64_t lead, end, g0, g1;                  // elements [lead, end) exist
  __device__ __forceinline__ Chunk(const ClipTensor &t, int64_t index) {
    const uintptr_t a = reinterpret_cast<uintptr_t>(t.grad);
    lead = (int64_t)((a & (kGroupBytes - 1)) / sizeof(T));
    base = static_cast<const T *>(t.grad) - lead;
    end = lead + t.numel;
    const int64_t groups = (end + VE - 1) / VE;
    g0 = index * kChunkGroups;
    g1 = g0 + kChunkGroups < groups ? g0 + kChunkGroups : groups;
  }
  __device__ __forceinline__ bool whole(int64_t g) const {
    return g * VE >= lead && (g + 1) * VE <= end;
  }
};

__device__ __forceinline__ float to_float(float v) { return v; }
__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ void store_as(float *q, float v) { *q = v; }
__device__ __forceinline__ void store_as(__nv_bfloat16 *q, float v) { *q = __float2bfloat16_rn(v); }

__device__ __forceinline__ float squares(const uint4 &v, float) {
  const float a = __uint_as_float(v.x), b = __uint_as_float(v.y);
  const float c = __uint_as_float(v.z), d = __uint_as_float(v.w);
  return fmaf(a, a, fmaf(b, b, fmaf(c, c, d * d)));
}
__device__ __forceinline__ float squares(const uint4 &v, __nv_bfloat16) {
  const uint32_t w[4] = {v.x, v.y, v.z, v.w};
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    s = fmaf(bf16_lo(w[i]), bf16_lo(w[i]), s);
    s = fmaf(bf16_hi(w[i]), bf16_hi(w[i]), s);
  }
  return s;
}

// `zeros`: the thread's part holds nothing but +0 (told for whole chunks alone).
template <typename T>
__device__ __forceinline__ float chunk_squares(const ClipTensor &t, int64_t index, bool &zeros) {
  const Chunk<T> c(t, index);
  constexpr int U = kChunkGroups / kClipThreads;
  float s = 0.0f;
  if (c.whole(c.g0) && c.whole(c.g0 + kChunkGroups - 1)) {
    const uint4 *in4 = reinterpret_cast<const uint4 *>(c.base) + c.g0 + threadIdx.x;
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = __ldg(in4 + u * kClipThreads);
#pragma unroll
    for (int u = 0; u < U; ++u) s += squares(v[u], T());
    if (s == 0.0f) {
      uint32_t any = 0;
#pragma unroll
      for (int u = 0; u < U; ++u) any |= v[u].x | v[u].y | v[u].z | v[u].w;
      zeros = any == 0;
    }
    return s;
  }
  for (int64_t g = c.g0 + threadIdx.x; g < c.g1; g += kClipThreads) {
    if (c.whole(g)) {
      s += squares(__ldg(reinterpret_cast<const uint4 *>(c.base) + g), T());
    } else {
      for (int64_t i = max(g * c.VE, c.lead); i < min((g + 1) * c.VE, c.end); ++i) {
        const float x = to_float(c.base[i]);
        s = fmaf(x, x, s);
      }
    }
  }
  return s;
}

// The same in binary64, for a thread whose sum left the range in which binary32
// squares are sums of normal numbers: values past 2^64 or so, or all below 2^-58.
// Not the norm's usual path, so that it may read the chunk again (600 M values near
// 1e-30: 2.2 ms, near 1 or all 0: 0.19).
template <typename T>
__device__ __noinline__ double chunk_squares_wide(const ClipTensor &t, int64_t index) {
  const Chunk<T> c(t, index);
  double s = 0.0;
  for (int64_t g = c.g0 + threadIdx.x; g < c.g1; g += kClipThreads) {
    for (int64_t i = max(g * c.VE, c.lead); i < min((g + 1) * c.VE, c.end); ++i) {
      const double x = (double)to_float(c.base[i]);
      s = fma(x, x, s);
    }
  }
  return s;
}

template <typename T>
__device__ __forceinline__ double chunk_sum(const ClipTensor &t, int64_t index) {
  bool zeros = false;
  const float s = chunk_squares<T>(t, index, zeros);
  // 64 squares and sums that are subnormal lose 2^-150 each: 2^-34 of such a sum
  return zeros || (s >= 0x1p-110f && s < INFINITY) ? (double)s : chunk_squares_wide<T>(t, index);
}

__device__ __forceinline__ double block_sum(double v, double *s_part) {
#pragma unroll
  for (int d = 16; d > 0; d >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, d);
  if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = v;
  __syncthreads();
  double r = 0.0;
  if (threadIdx.x == 0)
    for (int i = 0; i < kClipThreads / 32; ++i) r += s_part[i];
  return r;                                   // thread 0 has it
}

// As written: a norm that is NaN gives a coefficient that is NaN.
__device__ __forceinline__ float coefficient(float max_norm, float norm) {
  const float c = max_norm / (norm + kClipEps);
  return c > 1.0f ? 1.0f : c;
}

template <int BATCH>
__global__ void __launch_bounds__(kClipThreads, 4)
clip_norm_kernel(const __grid_constant__ ClipParams<BATCH> p) {
  __shared__ double s_part[kClipThreads / 32];
  __shared__ bool s_last;
  pdl_wait_for_previous();
  double sum = 0.0;
  for (int64_t c = blockIdx.x; c < p.chunks; c += gridDim.x) {
    const int i = tensor_of(p, c);
    const bool f32 = (p.f32[i >> 5] >> (i & 31)) & 1u;
    sum += f32 ? chunk_sum<float>(p.t[i], c - p.first[i]) : chunk_sum<__nv_bfloat16>(p.t[i], c - p.first[i]);
  }
  sum = block_sum(sum, s_part);
  if (threadIdx.x == 0) {
    p.partial[blockIdx.x] = sum;
    __threadfence();
    s_last = atomicAdd(&p.hdr->done, 1u) == gridDim.x - 1;
    __threadfence();
  }
  __syncthreads();
  if (!s_last) return;
  double all = 0.0;
  for (int i = threadIdx.x; i < (int)gridDim.x; i += kClipThreads)
    all += *reinterpret_cast<volatile double *>(p.partial + i);
  all = block_sum(all, s_part);
  if (threadIdx.x == 0) {
    if (!p.begin) all += p.hdr->total;
    p.hdr->total = all;
    p.hdr->done = 0;
    if (p.end) {
      const float norm = (float)sqrt(all);
      *p.norm = norm;
      p.hdr->coef = coefficient(p.max_norm, norm);
    }
  }
}

template <typename T>
__device__ __forceinline__ uint4 scaled(const uint4 &v, float coef) {
  uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    if (sizeof(T) == 4) {
      w[i] = __float_as_uint(__uint_as_float(w[i]) * coef);
    } else {
      const __nv_bfloat162 b = __floats2bfloat162_rn(bf16_lo(w[i]) * coef, bf16_hi(w[i]) * coef);
      w[i] = *reinterpret_cast<const uint32_t *>(&b);
    }
  }
  return make_uint4(w[0], w[1], w[2], w[3]);
}

template <typename T>
__device__ __forceinline__ void chunk_scale(const ClipTensor &t, int64_t index, float coef) {
  const Chunk<T> c(t, index);
  constexpr int U = kChunkGroups / kClipThreads;
  T *out = static_cast<T *>(t.out) - c.lead;
  const bool vec = (reinterpret_cast<uintptr_t>(out) & (kGroupBytes - 1)) == 0;
  if (vec && c.whole(c.g0) && c.whole(c.g0 + kChunkGroups - 1)) {
    // a chunk inside the tensor: nothing to check per group
    const uint4 *in4 = reinterpret_cast<const uint4 *>(c.base) + c.g0 + threadIdx.x;
    uint4 *out4 = reinterpret_cast<uint4 *>(out) + c.g0 + threadIdx.x;
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u) v[u] = __ldcs(in4 + u * kClipThreads);
#pragma unroll
    for (int u = 0; u < U; ++u) __stcs(out4 + u * kClipThreads, scaled<T>(v[u], coef));
    return;
  }
  for (int64_t g = c.g0 + threadIdx.x; g < c.g1; g += kClipThreads) {
    if (vec && c.whole(g)) {
      reinterpret_cast<uint4 *>(out)[g] = scaled<T>(reinterpret_cast<const uint4 *>(c.base)[g], coef);
    } else {
      for (int64_t i = max(g * c.VE, c.lead); i < min((g + 1) * c.VE, c.end); ++i)
        store_as(out + i, to_float(c.base[i]) * coef);
    }
  }
}

template <int BATCH>
__global__ void __launch_bounds__(kClipThreads, 4)
clip_scale_kernel(const __grid_constant__ ClipParams<BATCH> p) {
  pdl_wait_for_previous();
  const float coef = p.hdr->coef;
  for (int64_t k = blockIdx.x; k < p.chunks; k += gridDim.x) {
    const int64_t c = p.chunks - 1 - k;
    const int i = tensor_of(p, c);
    const ClipTensor &t = p.t[i];
    if (coef == 1.0f && t.out == t.grad) continue;
    if ((p.f32[i >> 5] >> (i & 31)) & 1u) chunk_scale<float>(t, c - p.first[i], coef);
    else chunk_scale<__nv_bfloat16>(t, c - p.first[i], coef);
  }
}

int64_t chunks_of(const moe_grad_tensor &t) {
  const int64_t size = t.dtype == MOE_DTYPE_FP32 ? 4 : 2;
  const int64_t bytes = (int64_t)(reinterpret_cast<uintptr_t>(t.grad) & (kGroupBytes - 1)) + t.numel * size;
  return (bytes + (int64_t)kChunkGroups * kGroupBytes - 1) / ((int64_t)kChunkGroups * kGroupBytes);
}

template <int BATCH>
cudaError_t launch_batches(const moe_grad_tensor *tensors, int num, float max_norm, float *norm,
                           void *workspace, cudaStream_t stream) {
  ClipParams<BATCH> p;
  p.hdr = static_cast<ClipHeader *>(workspace);
  p.partial = reinterpret_cast<double *>(static_cast<char *>(workspace) + sizeof(ClipHeader));
  p.norm = norm;
  p.max_norm = max_norm;
  const int64_t most = (int64_t)device_sm_count() * 4;
  const int64_t cap = most < kClipMaxBlocks ? most : kClipMaxBlocks;
  const int batches = num > 0 ? (num + BATCH - 1) / BATCH : 1;
  for (int k = 0; k < 2 * batches; ++k) {
    // the scaling pass takes the batches backwards too
    const bool scale = k >= batches;
    const int at = (scale ? 2 * batches - 1 - k : k) * BATCH;
    if (k != batches || batches > 1) {        // one batch: the norm's table serves both
      const int n = num - at < BATCH ? num - at : BATCH;
      p.chunks = 0;
      p.num = 0;
      for (int i = 0; i < BATCH / 32; ++i) p.f32[i] = 0;
      for (int i = 0; i < n; ++i) {
        const moe_grad_tensor &t = tensors[at + i];
        if (t.numel == 0) continue;
        p.t[p.num] = ClipTensor{t.grad, t.out, t.numel};
        p.first[p.num] = p.chunks;
        if (t.dtype == MOE_DTYPE_FP32) p.f32[p.num >> 5] |= 1u << (p.num & 31);
        p.chunks += chunks_of(t);
        ++p.num;
      }
    }
    p.begin = k == 0;
    p.end = k == batches - 1;
    const int64_t grid = p.chunks < cap ? p.chunks : cap;
    if (scale && grid == 0) continue;
    const cudaError_t e = launch_after_previous(scale ? clip_scale_kernel<BATCH> : clip_norm_kernel<BATCH>,
                                                (int)(grid < 1 ? 1 : grid), kClipThreads, p, stream);
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

size_t clip_workspace_bytes() {
  return sizeof(ClipHeader) + sizeof(double) * kClipMaxBlocks;
}

cudaError_t launch_clip(const moe_grad_tensor *tensors, int num, float max_norm, float *norm,
                        void *workspace, cudaStream_t stream) {
  // the table of tensors is copied with every launch: no larger than needed
  if (num <= 32) return launch_batches<32>(tensors, num, max_norm, norm, workspace, stream);
  if (num <= 128) return launch_batches<128>(tensors, num, max_norm, norm, workspace, stream);
  return launch_batches<kClipBatch>(tensors, num, max_norm, norm, workspace, stream);
}

}  // namespace moe
