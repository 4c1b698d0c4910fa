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
// How: bound by memory.  A lane takes a whole block: 64 bytes of bf16 as two
// 32-byte accesses (four of 16 where the array is not aligned to 32), 16 bytes of
// codes, no exchange for the maximum; four neighbouring lanes join their scale
// bytes into one word.  Lanes are dealt out over the rows' blocks, each row's
// rounded up to whole words of 4, so that short rows fill the warps as long ones
// do; a lane has kUnroll blocks in flight.  Where counts say which rows exist,
// those are numbered through by a prefix sum in shared memory, so that empty
// places cost nothing.  The dispatch reads a token's block once and writes its
// bytes and scales to its K rows.
//
// Measured on GB300 (copy 6.78 TB/s): 939.5 M elements of gate and up weights
// quantised in 347 us (6.9 TB/s), read back in 395 (6.0 TB/s); with one block in
// flight per lane both 778 us together, with two 743, with four 757.  Rows by counts,
// 8192 of 7168 over 256 experts: quantised in 28.8 us, read back in 29.1, 148 MB each
// (5.1 TB/s; 65536 rows 197 and 206 us, 6 TB/s).  DeepSeek-V3-shaped decode dispatch,
// 1024 tokens to 8 rows each, x from memory: 13.2 us for 46 MB, not memory but a chain
// of latencies (x, then the routes in rounds of four); 8192 tokens 81 us, 4.5 TB/s.
// With four lanes to a block (two shuffles for the maximum, 4-byte stores) weights
// there and back took 872 us, decode's dispatch and its rows read back 47, now 37.5.
#include "moe_mxfp4.cuh"
#include "moe_rows.cuh"

namespace moe {

namespace {

constexpr int kMxThreads = 256;
constexpr int kUnroll = 2;
constexpr int kRoutes = 4;     // of a token, loaded together
constexpr unsigned kFull = 0xFFFFFFFFu;

__device__ __forceinline__ uint32_t max_u16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.u16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}

// A block's 64 bytes of bf16, WIDE: 32-byte aligned.
template <bool WIDE>
__device__ __forceinline__ void load_block(const uint16_t *p, uint32_t (&w)[16]) {
  if (WIDE) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      asm volatile("ld.global.cs.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                   : "=r"(w[8 * i]), "=r"(w[8 * i + 1]), "=r"(w[8 * i + 2]), "=r"(w[8 * i + 3]),
                     "=r"(w[8 * i + 4]), "=r"(w[8 * i + 5]), "=r"(w[8 * i + 6]), "=r"(w[8 * i + 7])
                   : "l"(p + 16 * i));
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const uint4 v = __ldcs(reinterpret_cast<const uint4 *>(p) + i);
      w[4 * i] = v.x;
      w[4 * i + 1] = v.y;
      w[4 * i + 2] = v.z;
      w[4 * i + 3] = v.w;
    }
  }
}
template <bool WIDE>
__device__ __forceinline__ void store_block(uint16_t *p, const uint32_t (&w)[16]) {
  if (WIDE) {
#pragma unroll
    for (int i = 0; i < 2; ++i)
      asm volatile("st.global.cs.v8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(w[8 * i]),
                   "r"(w[8 * i + 1]), "r"(w[8 * i + 2]), "r"(w[8 * i + 3]), "r"(w[8 * i + 4]),
                   "r"(w[8 * i + 5]), "r"(w[8 * i + 6]), "r"(w[8 * i + 7]), "l"(p + 16 * i)
                   : "memory");
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i)
      __stcs(reinterpret_cast<uint4 *>(p) + i,
             make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]));
  }
}

// A block -> its codes, and the word of scales of its 4 lanes.  All 32 lanes
// call it.
struct Quantised {
  uint4 q;
  uint32_t scales;
};
__device__ __forceinline__ Quantised quantise(const uint32_t (&w)[16]) {
  constexpr uint32_t kMag = 0x7FFF7FFFu;
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 16; ++i) m = max_u16x2(m, w[i] & kMag);
  const uint32_t byte = mx_scale(max(m & 0xFFFFu, m >> 16) >> 7);
  const float inv = mx_inverse(byte);
  // a NaN times 0 would still be a NaN: such a block's elements become 0 here
  const uint32_t keep = byte == 255u ? 0u : 0xFFFFFFFFu;
  uint32_t q[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float f[8];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      const uint32_t v = w[4 * i + k] & keep;
      f[2 * k] = bf16_lo(v) * inv;
      f[2 * k + 1] = bf16_hi(v) * inv;
    }
    q[i] = e2m1x8(f);
  }
  Quantised r;
  r.q = make_uint4(q[0], q[1], q[2], q[3]);
  uint32_t s = byte << (8 * (threadIdx.x & 3));
  s |= __shfl_xor_sync(kFull, s, 1);
  s |= __shfl_xor_sync(kFull, s, 2);
  r.scales = s;
  return r;
}

// Whether the plan before failed, one answer for the whole warp: another block may
// set the word while it is read (a dispatch's, on an entry out of range), and lanes
// that left alone would be missing at the exchanges that follow.  One lane reads.
__device__ __forceinline__ bool plan_failed(const WsHeader *hdr) {
  int32_t st = MOE_OK;
  if (hdr && (threadIdx.x & 31) == 0) st = read_status(hdr);
  return __shfl_sync(kFull, st, 0) != MOE_OK;
}

// A lane's place among the rows' blocks, `nbp` to a row, and how it moves on by
// the grid's lanes.
struct Place {
  int64_t row;
  int b;
};
struct Steps {
  int64_t rows;
  int blocks, nbp;
  __device__ __forceinline__ Steps(int64_t lanes, int nbp_)
      : rows(lanes / nbp_), blocks((int)(lanes % nbp_)), nbp(nbp_) {}
  __device__ __forceinline__ void next(Place &p) const {
    p.row += rows;
    p.b += blocks;
    if (p.b >= nbp) {
      p.b -= nbp;
      ++p.row;
    }
  }
};
__device__ __forceinline__ Place first_place(int nbp) {
  const int64_t at = (int64_t)blockIdx.x * kMxThreads + threadIdx.x;
  return Place{at / nbp, (int)(at % nbp)};
}
__device__ __forceinline__ int64_t grid_lanes() { return (int64_t)gridDim.x * kMxThreads; }

// Calls body(experts, rows, blocks, exists, blocks of a row) for kUnroll places of
// every lane at a time until the warp has none left: rows of the experts' buffers,
// the populated ones alone with counts.  Without counts the grid's lanes go through
// the places side by side.  With them each thread block has a stretch of its own, so that a
// lane's next expert is this one or the next few: looked up from the start for
// every place, the rows of the DeepSeek-V3-shaped decode took 27 us to read back.
// After a failed plan there are none.
template <bool COUNTED, typename Body>
__device__ __forceinline__ void for_rows(const Mxfp4Rows &m, const int32_t *counts, const WsHeader *hdr, int E,
                                         const Body &body) {
  __shared__ int32_t s_prefix[COUNTED ? kMaxExperts + 1 : 1];
  __shared__ int32_t s_status;
  const int nb = m.cols / 32, nbp = (nb + 3) & ~3;
  if (COUNTED) {
    if (threadIdx.x == 0) s_status = hdr ? read_status(hdr) : MOE_OK;
    count_prefix<kMxThreads>(counts, E, m.rows, s_prefix);   // ends with a barrier
    if (s_status != MOE_OK) return;
    const int total = s_prefix[E];
    const int64_t places = (int64_t)total * nbp, share = (places + gridDim.x - 1) / gridDim.x;
    const int64_t rounds = (share + kMxThreads - 1) / kMxThreads;
    const int64_t at = (int64_t)blockIdx.x * rounds * kMxThreads + threadIdx.x;
    const Steps steps(kMxThreads, nbp);
    Place p{at / nbp, (int)(at % nbp)};
    int ex = p.row < total ? populated_expert(s_prefix, E, (int)p.row) : 0;
    for (int64_t i = 0; i < rounds && __any_sync(kFull, p.row < total); i += kUnroll) {
      int e[kUnroll], row[kUnroll], b[kUnroll];
      bool in[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        in[u] = p.row < total && i + u < rounds;
        const int r = in[u] ? (int)p.row : 0;
        if (in[u])
          while (s_prefix[ex + 1] <= r) ++ex;
        e[u] = ex;
        b[u] = p.b;
        row[u] = in[u] ? r - s_prefix[ex] : 0;
        steps.next(p);
      }
      body(e, row, b, in, nb);
    }
  } else {
    if (plan_failed(hdr)) return;
    const int64_t total = (int64_t)E * m.rows;
    const Steps steps(grid_lanes(), nbp);
    Place p = first_place(nbp);
    while (__any_sync(kFull, p.row < total)) {
      int e[kUnroll], row[kUnroll], b[kUnroll];
      bool in[kUnroll];
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        in[u] = p.row < total;
        const unsigned r = in[u] ? (unsigned)p.row : 0u;
        b[u] = p.b;
        e[u] = (int)(r / (unsigned)m.rows);
        row[u] = (int)(r - (unsigned)e[u] * (unsigned)m.rows);
        steps.next(p);
      }
      body(e, row, b, in, nb);
    }
  }
}

template <bool COUNTED, bool WIDE>
__global__ void __launch_bounds__(kMxThreads)
quant_kernel(QuantParams p) {
  pdl_wait_for_previous();
  const Mxfp4Rows &m = p.out;
  for_rows<COUNTED>(m, p.counts, p.hdr, p.E, [&](const int (&e)[kUnroll], const int (&row)[kUnroll],
                                                 const int (&b)[kUnroll], const bool (&in)[kUnroll], int nb) {
    uint32_t w[kUnroll][16];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      if (in[u] && b[u] < nb) {
        load_block<WIDE>(p.src + ((int64_t)e[u] * m.rows + row[u]) * m.cols + b[u] * 32, w[u]);
      } else {
#pragma unroll
        for (int i = 0; i < 16; ++i) w[u][i] = 0u;
      }
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const Quantised r = quantise(w[u]);
      if (!in[u]) continue;
      const int64_t at = ((int64_t)e[u] * m.rows + row[u]) * nb + b[u];
      if (b[u] < nb) reinterpret_cast<uint4 *>(m.q)[at] = r.q;
      if ((b[u] & 3) == 0)
        *reinterpret_cast<uint32_t *>(m.scale + expert_tiles(m, e[u]) + scale_word(m, row[u], b[u] >> 2)) = r.scales;
    }
  });
}

// The 8 E2M1 of a word times x -> 8 bf16.  The products are exact in bf16: their
// upper halves are the values.
__device__ __forceinline__ void dequantise8(uint32_t q, float x, uint32_t (&o)[4]) {
  uint32_t h[4];
  asm("{\n\t.reg .b8 a, b, c, d;\n\t"
      "mov.b32 {a, b, c, d}, %4;\n\t"
      "cvt.rn.f16x2.e2m1x2 %0, a;\n\t"
      "cvt.rn.f16x2.e2m1x2 %1, b;\n\t"
      "cvt.rn.f16x2.e2m1x2 %2, c;\n\t"
      "cvt.rn.f16x2.e2m1x2 %3, d;\n\t}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(q));
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    float lo, hi;
    asm("{\n\t.reg .b16 l, h;\n\tmov.b32 {l, h}, %2;\n\t"
        "cvt.f32.f16 %0, l;\n\tcvt.f32.f16 %1, h;\n\t}" : "=f"(lo), "=f"(hi) : "r"(h[i]));
    o[i] = __byte_perm(__float_as_uint(lo * x), __float_as_uint(hi * x), 0x7632);
  }
}

template <bool COUNTED, bool WIDE>
__global__ void __launch_bounds__(kMxThreads)
dequant_kernel(DequantParams p) {
  pdl_wait_for_previous();
  const Mxfp4Rows &m = p.in;
  for_rows<COUNTED>(m, p.counts, p.hdr, p.E, [&](const int (&e)[kUnroll], const int (&row)[kUnroll],
                                                 const int (&b)[kUnroll], const bool (&in)[kUnroll], int nb) {
    uint4 q[kUnroll];
    uint32_t s[kUnroll];
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const bool is = in[u] && b[u] < nb;
      const int64_t at = ((int64_t)e[u] * m.rows + row[u]) * nb + b[u];
      q[u] = is ? __ldcs(reinterpret_cast<const uint4 *>(m.q) + at) : make_uint4(0, 0, 0, 0);
      s[u] = is ? __ldg(m.scale + expert_tiles(m, e[u]) + scale_word(m, row[u], b[u] >> 2) + (b[u] & 3)) : 0u;
    }
#pragma unroll
    for (int u = 0; u < kUnroll; ++u) {
      const float x = s[u] == 255u ? __uint_as_float(0x7FC00000u)
                                   : __uint_as_float(s[u] ? s[u] << 23 : 1u << 22);
      const uint32_t c[4] = {q[u].x, q[u].y, q[u].z, q[u].w};
      uint32_t w[16];
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        uint32_t o[4];
        dequantise8(c[i], x, o);
#pragma unroll
        for (int k = 0; k < 4; ++k) w[4 * i + k] = o[k];
      }
      if (in[u] && b[u] < nb)
        store_block<WIDE>(p.out + ((int64_t)e[u] * m.rows + row[u]) * m.cols + b[u] * 32, w);
    }
  });
}

template <bool WIDE>
__global__ void __launch_bounds__(kMxThreads)
dispatch_mxfp4_kernel(DispatchMxfp4Params p) {
  const Mxfp4Rows &m = p.out;
  const int nb = m.cols / 32, nbp = (nb + 3) & ~3;
  const Steps steps(grid_lanes(), nbp);
  Place c = first_place(nbp);
  pdl_wait_for_previous();
  if (plan_failed(p.hdr)) return;
  for (; __any_sync(kFull, c.row < p.N); steps.next(c)) {
    const bool in = c.row < p.N;
    const int64_t g = in ? c.row : 0;
    uint32_t w[16];
    if (in && c.b < nb) {
      load_block<WIDE>(p.x + g * m.cols + c.b * 32, w);
    } else {
#pragma unroll
      for (int i = 0; i < 16; ++i) w[i] = 0u;
    }
    const Quantised r = quantise(w);
    for (int k0 = 0; in && k0 < p.K; k0 += kRoutes) {
      int e[kRoutes], s[kRoutes];
#pragma unroll
      for (int j = 0; j < kRoutes; ++j) {
        const bool is = k0 + j < p.K;
        e[j] = is ? __ldg(p.topk_idx + g * p.K + k0 + j) : -1;
        s[j] = is ? __ldg(p.slot_of + g * p.K + k0 + j) : -1;
      }
#pragma unroll
      for (int j = 0; j < kRoutes; ++j) {
        if (s[j] == -1) continue;            // not routed
        const bool e_ok = e[j] >= 0 && e[j] < p.E;
        if (!e_ok || s[j] < 0 || s[j] >= m.rows) {
          if (c.b == 0) report_status(p.hdr, e_ok ? MOE_ERR_CAPACITY : MOE_ERR_BAD_EXPERT);
          continue;
        }
        if (c.b < nb) reinterpret_cast<uint4 *>(m.q)[((int64_t)e[j] * m.rows + s[j]) * nb + c.b] = r.q;
        if ((c.b & 3) == 0)
          *reinterpret_cast<uint32_t *>(m.scale + expert_tiles(m, e[j]) + scale_word(m, s[j], c.b >> 2)) = r.scales;
      }
    }
  }
}

// `rows` rows of m.cols elements, `unroll` blocks of a lane at a time.
template <typename P>
cudaError_t launch(void (*kern)(P), int64_t rows, int cols, int unroll, const P &p, cudaStream_t stream) {
  const int64_t lanes = rows * ((cols / 32 + 3) & ~3);
  const int64_t warps = (lanes + 32 * unroll - 1) / (32 * unroll);
  return launch_after_previous(kern, persistent_grid((const void *)kern, kMxThreads, warps), kMxThreads, p,
                               stream);
}
bool wide(const void *p) { return (uintptr_t)p % 32 == 0; }

}  // namespace

cudaError_t launch_quant_mxfp4(const QuantParams &p, cudaStream_t stream) {
  const auto kern = p.counts ? (wide(p.src) ? quant_kernel<true, true> : quant_kernel<true, false>)
                             : (wide(p.src) ? quant_kernel<false, true> : quant_kernel<false, false>);
  return launch(kern, (int64_t)p.E * p.out.rows, p.out.cols, kUnroll, p, stream);
}

cudaError_t launch_dequant_mxfp4(const DequantParams &p, cudaStream_t stream) {
  const auto kern = p.counts ? (wide(p.out) ? dequant_kernel<true, true> : dequant_kernel<true, false>)
                             : (wide(p.out) ? dequant_kernel<false, true> : dequant_kernel<false, false>);
  return launch(kern, (int64_t)p.E * p.in.rows, p.in.cols, kUnroll, p, stream);
}

cudaError_t launch_dispatch_mxfp4(const DispatchMxfp4Params &p, cudaStream_t stream) {
  const auto kern = wide(p.x) ? dispatch_mxfp4_kernel<true> : dispatch_mxfp4_kernel<false>;
  return launch(kern, p.N, p.out.cols, 1, p, stream);
}

}  // namespace moe
