// moe_tc.cuh -- PTX helpers of the experts' products (moe_ffn.cu and
// moe_ffn_mxfp4.cu): TMA tile
// copies, tcgen05 matrix instructions on a pair of SMs, tensor memory, and
// cluster-scope mbarriers.
#pragma once

#include "moe_common.cuh"

#ifdef __CUDACC__
namespace moe {
namespace tc {

// --- cluster addresses and mbarriers ---
// The shared::cluster address of `local` (a shared::cta address) in CTA `rank`.
__device__ __forceinline__ uint32_t map_rank(uint32_t local, uint32_t rank) {
  uint32_t r;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(local), "r"(rank));
  return r;
}
__device__ __forceinline__ void mbar_init_at(uint32_t bar, uint32_t count) {
  asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(bar), "r"(count) : "memory");
}
// Arrive once for the whole warp, announcing `bytes`.
__device__ __forceinline__ void mbar_expect_warp(uint32_t bar, uint32_t bytes) {
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xFFFFFFFF;\n\t"
               "@e mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;\n\t}" ::"r"(bar), "r"(bytes)
               : "memory");
}
__device__ __forceinline__ void mbar_arrive_local(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(bar) : "memory");
}
// Arrive once for the whole warp on a barrier of any CTA of the cluster; what
// the lanes have read stays read, their stores are not released.
__device__ __forceinline__ void mbar_arrive_warp_at(uint32_t bar) {
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xFFFFFFFF;\n\t"
               "@e mbarrier.arrive.shared::cluster.b64 _, [%0];\n\t}" ::"r"(bar) : "memory");
}
// Arrive on a barrier of any CTA of the cluster, announcing `bytes`; nothing
// else is released.
__device__ __forceinline__ void mbar_expect_at(uint32_t bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.relaxed.cluster.shared::cluster.b64 _, [%0], %1;" ::"r"(bar),
               "r"(bytes) : "memory");
}
// 16 bytes into the shared memory of any CTA of the cluster; they complete on
// `bar` of the same CTA.
__device__ __forceinline__ void store_async(uint32_t dst, const uint4 &v, uint32_t bar) {
  asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v4.b32 [%0], {%1, %2, %3, %4}, [%5];"
               ::"r"(dst), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w), "r"(bar) : "memory");
}
// Arrive on a barrier of any CTA of the cluster.  Orders tcgen05 reads (after
// fence_before), not ordinary stores to memory that another CTA reads.
__device__ __forceinline__ void mbar_arrive_remote(uint32_t bar) {
  asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
  uint32_t ok;
  asm volatile("{\n\t.reg .pred p;\n\t"
               "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n\t"
               "selp.u32 %0, 1, 0, p;\n\t}"
               : "=r"(ok) : "r"(bar), "r"(parity) : "memory");
  return ok != 0;
}
// --- TMA ---
__device__ __forceinline__ void prefetch_map(const void *map) {
  asm volatile("prefetch.tensormap [%0];" ::"l"(map) : "memory");
}
// Copies and matrix instructions take their operands from the warp's uniform
// registers.  In a branch that one lane takes alone the compiler moves each
// operand there anew, about 70 cycles more per instruction (four matrix
// instructions of 256 x 256 x 16: 595 cycles instead of the 512 they take).  So
// whole warps run the loops that issue them, and these helpers pick the lane.

// A tile into this CTA's shared memory; its bytes complete on `bar`, which
// may lie in either CTA of the pair.  Called by a whole warp.
__device__ __forceinline__ void tma_load_pair(uint32_t dst, const void *map, uint32_t bar, int c0,
                                              int c1, int c2, int c3) {
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xFFFFFFFF;\n\t"
               "@e cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes "
               "[%0], [%1, {%3, %4, %5, %6}], [%2];\n\t}"
               ::"r"(dst), "l"(map), "r"(bar), "r"(c0), "r"(c1), "r"(c2), "r"(c3) : "memory");
}
// A copy of the tensor map `map` in global memory at `out` whose dimension 1
// has `rows` elements; `tmp` is 128 bytes of this CTA's shared memory.  Called
// by a whole warp.  A reader in a later kernel calls map_acquire first.
__device__ __forceinline__ void map_with_rows(void *out, const void *map, uint8_t *tmp, uint32_t rows) {
  const int lane = threadIdx.x & 31;
  reinterpret_cast<uint32_t *>(tmp)[lane] = static_cast<const uint32_t *>(map)[lane];
  __syncwarp();
  const uint32_t t = smem_u32(tmp);
  if (lane == 0)
    asm volatile("tensormap.replace.tile.global_dim.shared::cta.b1024.b32 [%0], 1, %1;" ::"r"(t), "r"(rows)
                 : "memory");
  __syncwarp();
  asm volatile("tensormap.cp_fenceproxy.global.shared::cta.tensormap::generic.release.gpu.sync.aligned "
               "[%0], [%1], 128;" ::"l"(out), "r"(t) : "memory");
  __syncwarp();
}
__device__ __forceinline__ void map_acquire(const void *map) {
  asm volatile("fence.proxy.tensormap::generic.acquire.gpu [%0], 128;" ::"l"(map) : "memory");
}
__device__ __forceinline__ void tma_store(const void *map, uint32_t src, int c0, int c1, int c2,
                                          int c3) {
  asm volatile("cp.async.bulk.tensor.4d.global.shared::cta.bulk_group [%0, {%2, %3, %4, %5}], [%1];"
               ::"l"(map), "r"(src), "r"(c0), "r"(c1), "r"(c2), "r"(c3) : "memory");
}
__device__ __forceinline__ void store_commit() {
  asm volatile("cp.async.bulk.commit_group;" ::: "memory");
}
template <int LEFT>
__device__ __forceinline__ void store_wait_read() {
  asm volatile("cp.async.bulk.wait_group.read %0;" ::"n"(LEFT) : "memory");
}
__device__ __forceinline__ void store_wait_all() {
  asm volatile("cp.async.bulk.wait_group 0;" ::: "memory");
}
// Between ordinary accesses to global memory and asynchronous copies of it.
__device__ __forceinline__ void fence_async_global() {
  asm volatile("fence.proxy.async.global;" ::: "memory");
}
__device__ __forceinline__ void fence_async_smem() {
  asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
}

// --- tensor memory ---
__device__ __forceinline__ void tmem_alloc_pair(uint32_t smem_slot, uint32_t cols) {
  asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_slot),
               "r"(cols) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
}
__device__ __forceinline__ void tmem_free_pair(uint32_t addr, uint32_t cols) {
  asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(addr), "r"(cols));
}
__device__ __forceinline__ void fence_before() {
  asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void fence_after() {
  asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}
// 32 columns of this warp's 32 lanes: v[i] = column i of the thread's lane.
__device__ __forceinline__ void tmem_ld32(uint32_t (&v)[32], uint32_t addr) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]),
        "=r"(v[7]), "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]),
        "=r"(v[14]), "=r"(v[15]), "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]),
        "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]),
        "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(addr));
}
__device__ __forceinline__ void tmem_ld_wait() {
  asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// --- matrix instructions ---
// Instruction descriptor of kind::f16: fp32 accumulator, bf16 operands,
// each operand K-major or (bit 15: A, bit 16: B) with its rows contiguous.
__host__ __device__ constexpr uint32_t instr_desc(uint32_t m, uint32_t n, bool a_mn, bool b_mn) {
  return (1u << 4) | (1u << 7) | (1u << 10) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) |
         ((n >> 3) << 17) | ((m >> 4) << 24);
}
// Shared-memory descriptor, 128-byte swizzle.  K-major: rows of 128 bytes,
// 1024 bytes from one group of 8 rows to the next (the stride field).
// MN-major: 64 consecutive rows' elements of one k are a 128-byte line, 8 k
// are 1024 bytes (the stride field), the next 64 rows are `leading` bytes on.
__device__ __forceinline__ uint64_t smem_desc(uint32_t addr, uint32_t leading) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(leading >> 4) << 16) |
         ((uint64_t)(1024u >> 4) << 32) | (1ull << 46) | (2ull << 61);
}
// A stage's products on both CTAs of the pair, by a whole warp: D (+)= A B^T
// over `steps` (1 to 4) times 16 k, `astep` and `bstep` apart in the
// descriptors; then arrive on `done`, at that offset in both CTAs, when they
// and everything before them are finished.  Between the instructions it asks
// whether phases `p0` of barrier `bar0` and `p1` of `bar1` are over; reading a
// barrier takes about 200 cycles beside the tensor cores' own reads, which
// pass while the instructions run.
struct Asked {
  uint32_t first, second;
};
__device__ __forceinline__ Asked mma_stage(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                           uint32_t accumulate, uint32_t steps, uint64_t astep,
                                           uint64_t bstep, uint32_t done, uint32_t bar0, uint32_t p0,
                                           uint32_t bar1, uint32_t p1) {
  Asked r;
  asm volatile("{\n\t.reg .pred e, e1, e2, e3, c, q0, q1;\n\t"
               ".reg .b64 a1, b1, a2, b2, a3, b3;\n\t"
               "elect.sync _|e, 0xFFFFFFFF;\n\t"
               "setp.ne.u32 c, %6, 0;\n\t"
               "setp.gt.and.u32 e1, %7, 1, e;\n\t"
               "setp.gt.and.u32 e2, %7, 2, e;\n\t"
               "setp.gt.and.u32 e3, %7, 3, e;\n\t"
               "add.s64 a1, %3, %8;\n\tadd.s64 b1, %4, %9;\n\t"
               "add.s64 a2, a1, %8;\n\tadd.s64 b2, b1, %9;\n\t"
               "add.s64 a3, a2, %8;\n\tadd.s64 b3, b2, %9;\n\t"
               "@e tcgen05.mma.cta_group::2.kind::f16 [%2], %3, %4, %5, c;\n\t"
               "mbarrier.test_wait.parity.shared::cta.b64 q0, [%11], %12;\n\t"
               "mbarrier.test_wait.parity.shared::cta.b64 q1, [%13], %14;\n\t"
               "@e1 tcgen05.mma.cta_group::2.kind::f16 [%2], a1, b1, %5, 1;\n\t"
               "@e2 tcgen05.mma.cta_group::2.kind::f16 [%2], a2, b2, %5, 1;\n\t"
               "@e3 tcgen05.mma.cta_group::2.kind::f16 [%2], a3, b3, %5, 1;\n\t"
               "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
               "[%10], %15;\n\t"
               "selp.u32 %0, 1, 0, q0;\n\t"
               "selp.u32 %1, 1, 0, q1;\n\t}"
               : "=r"(r.first), "=r"(r.second)
               : "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate), "r"(steps), "l"(astep), "l"(bstep),
                 "r"(done), "r"(bar0), "r"(p0), "r"(bar1), "r"(p1), "h"((uint16_t)3)
               : "memory");
  return r;
}
// Arrive on the barrier at this offset in both CTAs once every earlier matrix
// instruction of this warp is done.
__device__ __forceinline__ void mma_commit_pair(uint32_t bar) {
  asm volatile("{\n\t.reg .pred e;\n\telect.sync _|e, 0xFFFFFFFF;\n\t"
               "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
               "[%0], %1;\n\t}" ::"r"(bar), "h"((uint16_t)3) : "memory");
}

// --- block-scaled 4-bit matrix instructions ---
// Instruction descriptor of kind::mxf4: fp32 accumulator, E2M1 operands, K-major,
// UE8M0 scales, 64 k.  Which two of a column's four scale bytes an instruction
// takes stands in bits 4 and 29 (0: the first two, 2: the last two).
__host__ __device__ constexpr uint32_t instr_desc_mx(uint32_t m, uint32_t n) {
  return (1u << 7) | (1u << 10) | ((n >> 3) << 17) | (1u << 23) | ((m >> 4) << 24);
}
// Shared-memory descriptor of a tile of scales: 32 lanes of 16 bytes, no swizzle,
// 128 bytes from one group of 8 lanes to the next.
__device__ __forceinline__ uint64_t scale_desc(uint32_t addr) {
  return (uint64_t)((addr >> 4) & 0x3FFFu) | ((uint64_t)(128u >> 4) << 16) | ((uint64_t)(128u >> 4) << 32) |
         (1ull << 46);
}
// A stage's scales into tensor memory on both CTAs of the pair, each from its
// own shared memory, by a whole warp: two tiles of A's 128 rows, one for each 128
// k, into columns [to, to + 4) and [to + 4, to + 8), and `tiles` (1 to 3) of B's,
// 128 rows each, into [to + 8, to + 20) and [to + 20, to + 32), 4 columns a
// tile.  In shared memory the tiles of 128 k follow one another, those of the next
// 128 rows come after.  `second_k`: the stage has more than 128 k.  Called by the
// warp that issues the matrix instructions: the tensor core takes one thread's copies
// and instructions in the order of their issue, so that the columns are written again
// for the next stage without a wait.
__device__ __forceinline__ void load_scales(uint32_t to, uint64_t a, uint64_t b, uint32_t second_k,
                                            uint32_t tiles) {
  asm volatile("{\n\t.reg .pred e, ek, e1, e2, f1, f2;\n\t"
               ".reg .b32 t;\n\t"
               ".reg .b64 s;\n\t"
               "elect.sync _|e, 0xFFFFFFFF;\n\t"
               "setp.ne.and.u32 ek, %3, 0, e;\n\t"
               "setp.gt.and.u32 e1, %4, 1, e;\n\t"
               "setp.gt.and.u32 e2, %4, 2, e;\n\t"
               "setp.gt.and.u32 f1, %4, 1, ek;\n\t"
               "setp.gt.and.u32 f2, %4, 2, ek;\n\t"
               "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [%0], %1;\n\t"
               "add.u32 t, %0, 8;\n\t"
               "@e tcgen05.cp.cta_group::2.32x128b.warpx4 [t], %2;\n\t"
               "add.u32 t, %0, 12;\n\tadd.s64 s, %2, 64;\n\t"
               "@e1 tcgen05.cp.cta_group::2.32x128b.warpx4 [t], s;\n\t"
               "add.u32 t, %0, 16;\n\tadd.s64 s, %2, 128;\n\t"
               "@e2 tcgen05.cp.cta_group::2.32x128b.warpx4 [t], s;\n\t"
               "add.u32 t, %0, 4;\n\tadd.s64 s, %1, 32;\n\t"
               "@ek tcgen05.cp.cta_group::2.32x128b.warpx4 [t], s;\n\t"
               "add.u32 t, %0, 20;\n\tadd.s64 s, %2, 32;\n\t"
               "@ek tcgen05.cp.cta_group::2.32x128b.warpx4 [t], s;\n\t"
               "add.u32 t, %0, 24;\n\tadd.s64 s, %2, 96;\n\t"
               "@f1 tcgen05.cp.cta_group::2.32x128b.warpx4 [t], s;\n\t"
               "add.u32 t, %0, 28;\n\tadd.s64 s, %2, 160;\n\t"
               "@f2 tcgen05.cp.cta_group::2.32x128b.warpx4 [t], s;\n\t}"
               ::"r"(to), "l"(a), "l"(b), "r"(second_k), "r"(tiles) : "memory");
}
// mma_stage for kind::mxf4, after load_scales(scales, ...): `steps` (1 to 4) times
// 64 k.  The product's first column is row 0 of B's first tile of scales, or with
// `skip` 2 row 64: a column of scales holds those of 32 rows.
__device__ __forceinline__ Asked mma_stage_mx(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc,
                                              uint32_t scales, uint32_t skip, uint32_t accumulate,
                                              uint32_t steps, uint32_t done, uint32_t bar0, uint32_t p0, uint32_t bar1,
                                              uint32_t p1) {
  Asked r;
  asm volatile("{\n\t.reg .pred e, e1, e2, e3, c, q0, q1;\n\t"
               ".reg .b64 a1, b1, a2, b2, a3, b3;\n\t"
               ".reg .b32 odd, sb, sa1, sb1;\n\t"
               "elect.sync _|e, 0xFFFFFFFF;\n\t"
               "setp.ne.u32 c, %7, 0;\n\t"
               "setp.gt.and.u32 e1, %8, 1, e;\n\t"
               "setp.gt.and.u32 e2, %8, 2, e;\n\t"
               "setp.gt.and.u32 e3, %8, 3, e;\n\t"
               "or.b32 odd, %5, 0x40000020;\n\t"
               "add.u32 sa1, %6, 4;\n\tadd.u32 sb, %6, %15;\n\tadd.u32 sb, sb, 8;\n\tadd.u32 sb1, sb, 12;\n\t"
               "add.s64 a1, %3, 2;\n\tadd.s64 b1, %4, 2;\n\t"
               "add.s64 a2, %3, 4;\n\tadd.s64 b2, %4, 4;\n\t"
               "add.s64 a3, %3, 6;\n\tadd.s64 b3, %4, 6;\n\t"
               "@e tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%2], %3, %4, %5, [%6], [sb], c;\n\t"
               "mbarrier.test_wait.parity.shared::cta.b64 q0, [%10], %11;\n\t"
               "mbarrier.test_wait.parity.shared::cta.b64 q1, [%12], %13;\n\t"
               "@e1 tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%2], a1, b1, odd, [%6], [sb], 1;\n\t"
               "@e2 tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%2], a2, b2, %5, [sa1], [sb1], 1;\n\t"
               "@e3 tcgen05.mma.cta_group::2.kind::mxf4.block_scale.scale_vec::2X [%2], a3, b3, odd, [sa1], [sb1], 1;\n\t"
               "@e tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 "
               "[%9], %14;\n\t"
               "selp.u32 %0, 1, 0, q0;\n\t"
               "selp.u32 %1, 1, 0, q1;\n\t}"
               : "=r"(r.first), "=r"(r.second)
               : "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(scales), "r"(accumulate), "r"(steps), "r"(done),
                 "r"(bar0), "r"(p0), "r"(bar1), "r"(p1), "h"((uint16_t)3), "r"(skip)
               : "memory");
  return r;
}

}  // namespace tc
}  // namespace moe
#endif
