// moe_mxfp4.cu -- quantisation to MXFP4 and back, of rows where they stand and
// of tokens on their way to their experts.
//
// What it computes (OCP Microscaling Formats 1.0), for each block of 32
// elements of a row:
//   X = 2^(floor(log2 amax) - 2),  q = e2m1(x / X)  (nearest, ties to even, at
//   most 6),  and back  x = q X.
// X is a power of two, so that x / X is exact and q is rounded once; dequantised
// values are exact in bf16.  The scale is read from the exponent field of the
// block's largest magnitude, found on the bf16 bit patterns as integers (an
// infinity or a NaN is above every number there, and makes the block NaN).
//
// How: bound by memory.  A warp takes a segment of a row, U chunks of 32 x 16
// bytes, 4 lanes to a block: the maximum is two shuffles, a lane's 8 elements
// are 4 bytes, a half-warp's 4 scale bytes one word.  The dispatch reads a
// token once and writes the bytes and scales to its K rows.  Rows from an
// expert's count on are not touched.
#include "moe_mxfp4.cuh"

namespace moe {

namespace {

constexpr int kMxThreads = 256;
constexpr unsigned kFull = 0xFFFFFFFFu;

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// A lane's 8 elements of a block that 4 lanes share -> their bytes and the
// half-warp's word of 4 scales.  All 32 lanes call it.
struct Quantised {
  uint32_t q, scales;
};
__device__ __forceinline__ Quantised quantise8(const uint4 &v) {
  constexpr uint32_t kMag = 0x7FFF7FFFu;
  uint32_t m = max_u16x2(max_u16x2(v.x & kMag, v.y & kMag), max_u16x2(v.z & kMag, v.w & kMag));
  m = max_u16x2(m, __shfl_xor_sync(kFull, m, 1));
  m = max_u16x2(m, __shfl_xor_sync(kFull, m, 2));
  const uint32_t byte = mx_scale(max(m & 0xFFFFu, m >> 16) >> 7);
  const float inv = mx_inverse(byte);
  // a NaN times 0 would still be a NaN: such a block's elements become 0 here
  const uint32_t keep = byte == 255u ? 0u : 0xFFFFFFFFu;
  const uint32_t w[4] = {v.x & keep, v.y & keep, v.z & keep, v.w & keep};
  float f[8];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    f[2 * i] = bf16_lo(w[i]) * inv;
    f[2 * i + 1] = bf16_hi(w[i]) * inv;
  }
  Quantised r;
  r.q = e2m1x8(f);
  uint32_t s = byte << (8 * ((threadIdx.x >> 2) & 3));
  s |= __shfl_xor_sync(kFull, s, 4);
  s |= __shfl_xor_sync(kFull, s, 8);
  r.scales = s;
  return r;
}

__device__ __forceinline__ bool plan_failed(const WsHeader *hdr) {
  return hdr && read_status(hdr) != MOE_OK;
}
__device__ __forceinline__ int rows_below(const int32_t *counts, int e, int rows) {
  return counts ? min(max(__ldg(counts + e), 0), rows) : rows;
}

// Walks (expert, row, segment) with a constant stride without divisions.
struct RowCursor {
  int e, row, seg;
  int de, drow, dseg;
  __device__ __forceinline__ RowCursor(int64_t task, int64_t stride, int rows, int segs) {
    const int64_t r = task / segs, dr = stride / segs;
    seg = (int)(task - r * segs);
    dseg = (int)(stride - dr * segs);
    e = (int)(r / rows);
    row = (int)(r - (int64_t)e * rows);
    de = (int)(dr / rows);
    drow = (int)(dr - (int64_t)de * rows);
  }
  __device__ __forceinline__ void next(int rows, int segs) {
    seg += dseg;
    if (seg >= segs) {
      seg -= segs;
      ++row;
    }
    row += drow;
    e += de;
    if (row >= rows) {
      row -= rows;
      ++e;
    }
  }
};

template <int U>
__global__ void __launch_bounds__(kMxThreads)
quant_kernel(QuantParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t warp0 = ((int64_t)blockIdx.x * kMxThreads + threadIdx.x) >> 5;
  const int64_t nwarps = ((int64_t)gridDim.x * kMxThreads) >> 5;
  const Mxfp4Rows &m = p.out;
  const int cpr = m.cols / 8, segs = (cpr + 32 * U - 1) / (32 * U);
  pdl_wait_for_previous();
  if (plan_failed(p.hdr)) return;
  RowCursor c(warp0, nwarps, m.rows, segs);
  for (; c.e < p.E; c.next(m.rows, segs)) {
    if (c.row >= rows_below(p.counts, c.e, m.rows)) continue;
    const int64_t row = (int64_t)c.e * m.rows + c.row;
    const uint4 *src = reinterpret_cast<const uint4 *>(p.src) + row * cpr;
    const int c0 = c.seg * 32 * U + lane;
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      v[u] = c0 + 32 * u < cpr ? __ldcs(src + c0 + 32 * u) : make_uint4(0, 0, 0, 0);
    uint32_t *q = reinterpret_cast<uint32_t *>(m.q) + row * cpr;
    uint8_t *tiles = m.scale + expert_tiles(m, c.e);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const Quantised r = quantise8(v[u]);
      const int at = c0 + 32 * u;
      if (at < cpr) q[at] = r.q;
      if ((lane & 15) == 0 && at < cpr)
        *reinterpret_cast<uint32_t *>(tiles + scale_word(m, c.row, at >> 4)) = r.scales;
    }
  }
}

// Two E2M1 of a byte -> floats.
__device__ __forceinline__ float2 e2m1x2_to_float(uint32_t byte) {
  uint32_t h;
  asm("{\n\t.reg .b8 a;\n\tcvt.u8.u32 a, %1;\n\tcvt.rn.f16x2.e2m1x2 %0, a;\n\t}" : "=r"(h) : "r"(byte));
  float2 r;
  asm("{\n\t.reg .b16 lo, hi;\n\tmov.b32 {lo, hi}, %2;\n\t"
      "cvt.f32.f16 %0, lo;\n\tcvt.f32.f16 %1, hi;\n\t}" : "=f"(r.x), "=f"(r.y) : "r"(h));
  return r;
}

template <int U>
__global__ void __launch_bounds__(kMxThreads)
dequant_kernel(DequantParams p) {
  const int lane = threadIdx.x & 31;
  const int64_t warp0 = ((int64_t)blockIdx.x * kMxThreads + threadIdx.x) >> 5;
  const int64_t nwarps = ((int64_t)gridDim.x * kMxThreads) >> 5;
  const Mxfp4Rows &m = p.in;
  const int cpr = m.cols / 8, segs = (cpr + 32 * U - 1) / (32 * U);
  pdl_wait_for_previous();
  if (plan_failed(p.hdr)) return;
  RowCursor c(warp0, nwarps, m.rows, segs);
  for (; c.e < p.E; c.next(m.rows, segs)) {
    if (c.row >= rows_below(p.counts, c.e, m.rows)) continue;
    const int64_t row = (int64_t)c.e * m.rows + c.row;
    const uint32_t *q = reinterpret_cast<const uint32_t *>(m.q) + row * cpr;
    const uint8_t *tiles = m.scale + expert_tiles(m, c.e);
    const int c0 = c.seg * 32 * U + lane;
    uint32_t v[U], s[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = c0 + 32 * u;
      const bool in = at < cpr;
      v[u] = in ? __ldcs(q + at) : 0u;
      s[u] = in ? __ldg(tiles + scale_word(m, c.row, at >> 4) + ((at >> 2) & 3)) : 0u;
    }
    uint4 *out = reinterpret_cast<uint4 *>(p.out) + row * cpr;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int at = c0 + 32 * u;
      const float x = s[u] == 255u ? __uint_as_float(0x7FC00000u)
                                   : __uint_as_float(s[u] ? s[u] << 23 : 1u << 22);
      uint32_t o[4];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const float2 f = e2m1x2_to_float((v[u] >> (8 * i)) & 0xFFu);
        // exact in bf16: the upper halves are the values
        o[i] = __byte_perm(__float_as_uint(f.x * x), __float_as_uint(f.y * x), 0x7632);
      }
      if (at < cpr) __stcs(out + at, make_uint4(o[0], o[1], o[2], o[3]));
    }
  }
}

template <int U>
__global__ void __launch_bounds__(kMxThreads)
dispatch_mxfp4_kernel(DispatchMxfp4Params p) {
  const int lane = threadIdx.x & 31;
  const int64_t warp0 = ((int64_t)blockIdx.x * kMxThreads + threadIdx.x) >> 5;
  const int64_t nwarps = ((int64_t)gridDim.x * kMxThreads) >> 5;
  const Mxfp4Rows &m = p.out;
  const int cpr = m.cols / 8, segs = (cpr + 32 * U - 1) / (32 * U);
  const int64_t ntasks = (int64_t)p.N * segs;
  pdl_wait_for_previous();
  if (plan_failed(p.hdr)) return;
  TaskCursor cur(warp0, nwarps, segs);
  for (int64_t task = warp0; task < ntasks; task += nwarps, cur = cur.next()) {
    const int64_t g = cur.g;
    int e_l = -1, s_l = -1;
    if (lane < p.K) {
      e_l = __ldg(p.topk_idx + g * p.K + lane);
      s_l = __ldg(p.slot_of + g * p.K + lane);
    }
    const int c0 = cur.seg * 32 * U + lane;
    uint4 v[U];
#pragma unroll
    for (int u = 0; u < U; ++u)
      v[u] = c0 + 32 * u < cpr ? __ldcs(reinterpret_cast<const uint4 *>(p.x) + g * cpr + c0 + 32 * u)
                               : make_uint4(0, 0, 0, 0);
    Quantised r[U];
#pragma unroll
    for (int u = 0; u < U; ++u) r[u] = quantise8(v[u]);
    const bool routed = lane < p.K && s_l != -1;
    const bool e_ok = e_l >= 0 && e_l < p.E;
    const bool ok = routed && e_ok && s_l >= 0 && s_l < m.rows;
    if (cur.seg == 0 && routed && !ok) report_status(p.hdr, e_ok ? MOE_ERR_CAPACITY : MOE_ERR_BAD_EXPERT);
    for (unsigned left = __ballot_sync(kFull, ok); left != 0; left &= left - 1) {
      const int k = __ffs(left) - 1;
      const int e = __shfl_sync(kFull, e_l, k), s = __shfl_sync(kFull, s_l, k);
      uint32_t *q = reinterpret_cast<uint32_t *>(m.q) + ((int64_t)e * m.rows + s) * cpr;
      uint8_t *tiles = m.scale + expert_tiles(m, e);
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int at = c0 + 32 * u;
        if (at < cpr) q[at] = r[u].q;
        if ((lane & 15) == 0 && at < cpr)
          *reinterpret_cast<uint32_t *>(tiles + scale_word(m, s, at >> 4)) = r[u].scales;
      }
    }
  }
}

// Chunks per lane: as many as the row has, 4 at most.
int chunks(int cols) {
  const int w = (cols / 8 + 31) / 32;
  return w >= 4 ? 4 : w >= 2 ? 2 : 1;
}

template <typename P>
cudaError_t launch_rows(void (*kern)(P), int64_t rows, int cols, int U, const P &p, cudaStream_t stream) {
  const int64_t tasks = rows * ((cols / 8 + 32 * U - 1) / (32 * U));
  return launch_after_previous(kern, persistent_grid((const void *)kern, kMxThreads, tasks), kMxThreads, p,
                               stream);
}

}  // namespace

cudaError_t launch_quant_mxfp4(const QuantParams &p, cudaStream_t stream) {
  const int64_t rows = (int64_t)p.E * p.out.rows;
  const int U = chunks(p.out.cols);
  const auto kern = U == 4 ? quant_kernel<4> : U == 2 ? quant_kernel<2> : quant_kernel<1>;
  return launch_rows(kern, rows, p.out.cols, U, p, stream);
}

cudaError_t launch_dequant_mxfp4(const DequantParams &p, cudaStream_t stream) {
  const int64_t rows = (int64_t)p.E * p.in.rows;
  const int U = chunks(p.in.cols);
  const auto kern = U == 4 ? dequant_kernel<4> : U == 2 ? dequant_kernel<2> : dequant_kernel<1>;
  return launch_rows(kern, rows, p.in.cols, U, p, stream);
}

cudaError_t launch_dispatch_mxfp4(const DispatchMxfp4Params &p, cudaStream_t stream) {
  const int U = chunks(p.out.cols);
  const auto kern = U == 4 ? dispatch_mxfp4_kernel<4> : U == 2 ? dispatch_mxfp4_kernel<2> : dispatch_mxfp4_kernel<1>;
  return launch_rows(kern, p.N, p.out.cols, U, p, stream);
}

}  // namespace moe
