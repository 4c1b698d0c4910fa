// moe_ffn.cu -- the experts' gated feed-forward over the dispatched rows, and
// its backward pass, as grouped matrix products on the tensor cores.
//
// What it computes, for expert e and its count[e] rows x:
//   h = x Wgu^T (gate | up),  a = SiLU(gate) * up,  y = a Wd^T
// and, from dy and the kept h, with s = sigmoid(gate):
//   da = dy Wd,  dgate = da up s (1 + gate (1 - s)),  dup = da gate s,
//   dx = dh Wgu,  dWgu = dh^T x,  dWd = dy^T a.
//
// How: one launch of pair_kernel<KIND> forward, kForward (a, then y), and two
// backward, kActGrad (da, and from it a and dh) and kRest (dx, dWgu and dWd).  A cluster
// of two CTAs (the two SMs of a pair) computes a tile of 256 rows x up to 256
// columns with tcgen05.mma.cta_group::2: each CTA stages its half of both
// operands (128 rows of A, half the columns of B, 64 k at a time) by TMA in a
// ring of 6 stages, a warp of the leading CTA issues the matrix instructions,
// and the accumulators stay in tensor memory, two tiles deep, so that the
// eight epilogue warps of each CTA write one tile while the next is multiplied.
//  - Products over the hidden or intermediate size ("row products") put the
//    weights' output features on the 256-row side and the expert's tokens on
//    the column side: the column count of a matrix instruction can be any
//    multiple of 32, so an expert with 40 tokens costs 64 columns and not a
//    whole tile of 256.  An expert's tokens are cut into equal tiles of at
//    most 256.  Gate and up of the same 64 features are the two halves of a
//    CTA's 128 rows, so that a is computed from both in binary32 and h need
//    not be written.
//  - Weight gradients contract over the expert's tokens; both operands are
//    then read with the contraction as the outer dimension (MN-major
//    shared-memory tiles).  Rows past count[e] are not the expert's and may
//    hold anything, NaN included: kActGrad writes, for every expert, tensor
//    maps that end at its count, and the copies fill the rest of the last
//    block of 64 tokens with zeros.  (Zeroing that block in shared memory
//    instead took about 2000 cycles per tile: dWgu of the Mixtral-shaped batch
//    1310 us, now 1220.)
//  - Few tiles and a long contraction (few tokens): the tiles of the last,
//    partial round are cut into parts whose sums are joined, see choose_split.
//  - Forward, a tile of y needs all of its rows of a.  Its first copy waits, with
//    a limit, until a counter says that every tile of a is written.  Units come
//    from a counter in order, so that those that are waited for are with pairs
//    that run, and wait for nothing themselves.  Two launches against one: 61 odd
//    rows 10.3 and 8.9 us, ten rows over 95 experts 28.4 and 25.6, 128 rows of one
//    expert 36.6 and 34.1, one token 117.7 and 114.9; batch and decode the same.
//    The backward pass in one launch as well: 128 rows 11.7 and 10.6 us, batch
//    sizes the same, but uneven experts 207 (two launches) and 214, few rows of
//    many experts 271 and 288, so that it stays at two.  Bringing Wd into the L2
//    during the wait: one token 111.9 us without, 113.2 and 115.5 with 12 and 40
//    blocks a tile.
// Counts are read on the device: nothing waits for the host, and the call can
// be captured in a CUDA graph.  Tiles go to the pairs in order, as they get
// free: what runs at one time is then a stretch of the list, whose operands
// the L2 holds.  Dealt out round robin instead, pairs whose tiles were
// narrower ran ahead (backward of the Mixtral-shaped batch 4.06 ms, now 3.78).
//
// Rounding: the operands are bf16, every product and sum is accumulated in
// binary32; a, dh and the results are rounded to bf16 once each (the matrix
// instructions take 16-bit operands; the kept h is never re-rounded).
//
// What bounds it, measured on GB300 (copy 6.78 TB/s; bf16 products of the library
// 1.94 PFLOP/s the best of ten, 1.71 for seconds, under the power limit):
//  - Mixtral-shaped batch (8192 rows over 8 experts, H 4096, I 14336): forward
//    1.79 to 1.87 ms (1.54 to 1.61 PFLOP/s), backward 3.70 to 3.85 (1.50 to
//    1.56).  At 2048 rows over 2 experts the tensor pipe is active 94 % of kRest's
//    cycles, 80 % of kActGrad's (its epilogue reads h) and 85 % of the forward
//    pass's (its ends, and the wait between a and y).  At 8192 rows the clock,
//    1.32 to 1.36 GHz at 1.37 kW, is what the power limit leaves.
//  - DeepSeek-V3-shaped decode (256 experts, 32 rows each, 22.5 GB of weights):
//    3.32 ms, 6.86 TB/s: the weights' reading.  One token over two experts of
//    the Mixtral shape: 113 to 116 us for 705 MB.
//  - Weight gradients of experts with few rows: not established.  64 experts of 128
//    rows, 2.1 GB of dWgu, are written at 5 TB/s.  kRest of 31 experts with 5000
//    rows (H 2048, I 1000) takes 147 us from cold caches, moves 0.70 GB to and from
//    memory (4.8 TB/s) and keeps the tensor pipe active 33 % of the cycles: neither is
//    at its limit.  Its tiles multiply for 2 to 3 blocks and then store 256 x 256
//    values through one staging buffer per warp, which is the likely bound.
//  - Tiny calls: latency, about 5 us a launch from the end of the one before:
//    status and counts, the first copies, the products, the epilogue.
//  - Few tiles: the last round.  Dense, H 7168, I 2048 (88 MB of weights, 13 us):
//    1 row 30.1 us, 128 rows 34.1, 1024 rows 64.5 (46.6 of operations); y of 128
//    rows is 28 tiles on 76 pairs, and no cut is priced below none.  dx alone is
//    not cut: one token of two Mixtral-shaped experts 137 us for 705 MB.
#include <mutex>

#include "moe_ffn.cuh"
#include "moe_pairs.cuh"

namespace moe {

namespace {

constexpr int kPairThreads = 384;      // warps: 0 TMA, 1 MMA, 2 maps, 3 scheduling, 4-11 epilogue
constexpr int kStages = 6;
constexpr int kBlockK = 64;            // one 128-byte swizzled line of bf16
constexpr uint32_t kHalfBytes = 128 * kBlockK * 2;       // a CTA's half of one operand: 16 KB
constexpr uint32_t kStageBytes = 2 * kHalfBytes;
constexpr uint32_t kStagingBytes = 2 * 16384;            // epilogue, one buffer per group
constexpr uint32_t kBarOff = kStages * kStageBytes + kStagingBytes;
constexpr uint32_t kRingOff = kBarOff + 256;
constexpr uint32_t kMapOff = kRingOff + kRing * 64;      // kActGrad: a tensor map being written
constexpr uint32_t kPairSmem = kMapOff + 128 + 1024;     // + alignment slack
static_assert(kPairSmem <= 232448, "shared memory of one CTA");

struct Job {
  CUtensorMap a;
  CUtensorMap b[4];        // row products: boxes of 16, 32, 64 and 128 tokens
  CUtensorMap out;         // weight gradients: stored by TMA
  uint16_t *o0, *o1;       // row products: outputs (gate and up: a, h or null; kActGrad: a, dh)
  const uint16_t *h;       // kActGrad: kept gate | up
  int M, N, K;             // features; weight gradients: output columns; row products: contraction
  int mt;                  // tiles of 256 accumulator rows (gate and up: of 128 features); 0: no job
  int a_wide, b_wide;      // MN-major operands: a copy brings 128 rows (else 64) x 64 k
};

// The operands of the weight gradients, dh and x of dWgu, dy and a of dWd: their
// tensor maps, and those that end at each expert's count, [4][E] in the
// workspace.  Written by kActGrad, read by kRest.
constexpr int kRowMaps = 4;
template <int KIND>
struct RowMaps {};
template <>
struct RowMaps<kActGrad> {
  CUtensorMap whole[kRowMaps];
};

template <int KIND>
struct PairParams {
  static constexpr int kKind = KIND, kBlock = kBlockK;
  static constexpr int kTileStep = 32, kExpertGroups = 1;
  static constexpr int kJobs = KIND == kRest ? 3 : KIND == kForward ? 2 : 1;
  Job job[kJobs];          // kForward: a, y; kRest: dx, dWgu, dWd
  const int32_t *counts;   // [E], or null (cap rows each)
  WsHeader *hdr;
  float *part;             // partial sums of split contractions
  uint32_t *tickets;       // finished parts, 4 bits for each split tile and CTA of the pair
  UnitCounter *units;
  CUtensorMap *row_maps;   // [4][E], or null
  RowMaps<KIND> maps;
  int E, cap;
};

__device__ __forceinline__ uint2 pack4(const float (&v)[4]) {
  return make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
}
__device__ __forceinline__ void unpack4(const uint2 &w, float (&v)[4]) {
  v[0] = bf16_lo(w.x);
  v[1] = bf16_hi(w.x);
  v[2] = bf16_lo(w.y);
  v[3] = bf16_hi(w.y);
}

template <int KIND>
__global__ void __launch_bounds__(kPairThreads, 1) __cluster_dims__(2, 1, 1)
pair_kernel(const __grid_constant__ PairParams<KIND> p) {
  constexpr bool kAMn = KIND == kActGrad || KIND == kRest;
  extern __shared__ uint8_t smem_raw[];
  const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t *smem_p = smem_raw + (smem - smem_u32(smem_raw));
  // the same value in every lane, and known to be
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_cta_rank();

  const uint32_t staging = smem + kStages * kStageBytes;
  const uint32_t bars = smem + kBarOff;
  const uint32_t full = bars, empty = bars + 8 * kStages;
  const uint32_t tm_full = bars + 16 * kStages, tm_empty = tm_full + 16;
  const uint32_t tm_slot = tm_empty + 16;
  // barriers of the ring of tiles
  const uint32_t rec_full = bars + 192, rec_empty = bars + 224;
  Tile *ring = reinterpret_cast<Tile *>(smem_p + kRingOff);
  volatile uint32_t *last_in = reinterpret_cast<uint32_t *>(smem_p + kBarOff + 16 * kStages + 40);

  if (threadIdx.x == 0) {
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init_at(full + 8 * s, 1);     // the leader's arrival, and the bytes of both CTAs
      tc::mbar_init_at(empty + 8 * s, 1);    // the commit of the stage's instructions
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init_at(tm_full + 8 * b, 1);
      tc::mbar_init_at(tm_empty + 8 * b, 2 * kEpiWarps);   // the epilogue warps of both CTAs
    }
    for (int r = 0; r < kRing; ++r) {
      tc::mbar_init_at(rec_full + 8 * r, 1);
      // in the leader: TMA and epilogue of both CTAs, and the MMA warp
      tc::mbar_init_at(rec_empty + 8 * r, 2 * (kEpiWarps + 1) + 1);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  } else if (threadIdx.x == 32 && p.job[0].mt > 0) {
    tc::prefetch_map(&p.job[0].a);
    tc::prefetch_map(&p.job[0].b[0]);
    if (KIND == kForward) tc::prefetch_map(&p.job[PairParams<KIND>::kJobs - 1].a);
  }
  if (warp == 2) tc::tmem_alloc_pair(tm_slot, kTmemCols);
  tc::fence_before();
  __syncthreads();
  cluster_arrive_relaxed();              // the barriers' initial values are released above
  cluster_wait();
  tc::fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem_p + kBarOff + 16 * kStages + 32);

  pdl_allow_dependents();
  pdl_wait_for_previous();
  // After a plan error, or a wait of an earlier launch that ran out, no tile is
  // computed and nothing is written.  The block's threads decide together: both
  // words may change under them when another pair's wait runs out.
  const uint64_t tmo = p.hdr->timeout_ns;
  const StatusWords words = read_status_words(p.hdr);
  const bool broken = (words.flags & kFfnBroken) != 0;
  const bool live = __syncthreads_and(words.status == MOE_OK && !broken);
  if (broken && threadIdx.x == 0) report_status(p.hdr, MOE_ERR_TIMEOUT);
  const uint64_t limit = tmo ? tmo : kDefaultTimeoutNs;
  bool ok = true;
  Tile t;
  Feed feed(ring, rec_full, tc::map_rank(rec_empty, 0), limit);

  if (warp == 3) {
    // ---- scheduling: one warp of the leader takes units and announces their
    // tiles to both CTAs.  (The first counts are read together with the status.)
    // Where no tile waits for another pair's, the pair's first unit is its own
    // number, and each CTA finds it; in kForward a unit belongs to a pair that
    // runs, since others will wait for it.
    constexpr bool kOwnFirst = KIND != kForward;
    Schedule<PairParams<KIND>> sched(p);
    const uint32_t peer_full = tc::map_rank(rec_full, 1), peer_ring = tc::map_rank(smem + kRingOff, 1);
    int64_t unit = blockIdx.x >> 1;
    bool written = false;                    // kForward: all of a
    const uint32_t epoch = KIND == kForward && rank == 0 ? __ldcg(&p.units->epoch) & 1u : 0u;
    uint32_t c = 0;
    for (; live && (kOwnFirst || rank == 0); ++c) {
      const uint32_t s = c % kRing;
      if (c > 0 || !kOwnFirst) {
        // A unit is taken as late as its tile allows: once the record 2 or
        // kRing before it has been read by every warp of both CTAs.
        const uint32_t ahead = c > 0 && t.nk >= kLongTile ? 2 : kRing;
        if (c >= ahead) {
          const uint32_t r = c - ahead;
          ok = __all_sync(0xFFFFFFFFu, wait_bar(rec_empty + 8 * (r % kRing), (r / kRing) & 1u, limit));
          if (!ok) break;
        }
        // one tile of y for each pair until all of a is written: a second one
        // would be missing where a pair is still busy with a (one token 132
        // us, now 115; 32 rows over eight such experts 451 and 420)
        if (KIND == kForward && c > 0 && t.need != 0 && !written) {
          written = ok =
              __all_sync(0xFFFFFFFFu, wait_count(p.units->ready + epoch, (uint32_t)t.need, limit));
          if (!ok) break;
        }
        unsigned long long n = 0;
        if (lane == 0) n = atomicAdd(&p.units->next, 1ull);
        unit = (kOwnFirst ? gridDim.x >> 1 : 0) + (int64_t)__shfl_sync(0xFFFFFFFFu, n, 0);
      }
      t.valid = sched.find(unit, t);
      t.epoch = epoch;
      if (lane == 0) {
        ring[s] = t;
        tc::mbar_arrive_local(rec_full + 8 * s);
      }
      if (c > 0 || !kOwnFirst) {
        __syncwarp();
        if (lane == 0) tc::mbar_expect_at(peer_full + 8 * s, sizeof(Tile));
        if (lane < 4)
          tc::store_async(peer_ring + s * (uint32_t)sizeof(Tile) + lane * 16,
                          reinterpret_cast<const uint4 *>(ring + s)[lane], peer_full + 8 * s);
      }
      if (!t.valid || rank != 0) break;
    }
    // the other CTA's arrivals for the records before the last (number c) land
    // before this one may exit
    if (live && rank == 0)
      for (uint32_t r = c < kRing ? 0 : c - kRing + 1; ok && r < c; ++r)
        ok = __all_sync(0xFFFFFFFFu, wait_bar(rec_empty + 8 * (r % kRing), (r / kRing) & 1u, limit));
    if (rank == 0 && lane == 0 &&
        atomicAdd(&p.units->done, 1u) == (gridDim.x >> 1) - 1) {
      // every pair knows this launch's epoch by now: the next one counts in the
      // other counter, which nobody uses any more
      p.units->next = 0;
      p.units->done = 0;
      if (KIND == kForward) {
        p.units->ready[epoch ^ 1u] = 0;
        p.units->epoch = epoch ^ 1u;
      }
    }
  } else if (live && warp == 0) {
    // ---- TMA: both CTAs load their halves; bytes complete on the leader's barrier
    int s = 0;
    uint32_t ph = 0;
    const uint32_t full0 = tc::map_rank(full, 0);
    const CUtensorMap *held = nullptr;       // kRest: the maps acquired last
    bool written = false;                    // kForward: all of a
    while (ok && feed.next_uniform<kCopyWords>(t, ok)) {
      const Job &j = p.job[KIND != kActGrad ? t.job : 0];
      const bool weight = KIND == kRest && t.job > 0;
      const uint32_t half_n = t.n >> 1;
      const int bsel = half_n <= 16 ? 0 : half_n <= 32 ? 1 : half_n <= 64 ? 2 : 3;
      const uint32_t bytes = kHalfBytes + (weight ? kHalfBytes : (16u << bsel) * 128u);
      const int m0 = t.m * 256 + (int)rank * 128, n0 = t.n0 + (int)(rank * half_n);
      const CUtensorMap *map_a = &j.a, *map_b = &j.b[bsel];
      if (weight) {                          // the expert's own maps, which end at its count
        map_a = p.row_maps + (int64_t)(2 * (t.job - 1)) * p.E + t.e;
        map_b = map_a + p.E;
        if (map_a != held && t.nk > 0) {
          tc::map_acquire(map_a);
          tc::map_acquire(map_b);
          held = map_a;
        }
      }
      if (KIND == kForward && t.need != 0 && !written) {
        written = ok = __all_sync(0xFFFFFFFFu, wait_count(p.units->ready + t.epoch, (uint32_t)t.need, limit));
        if (!ok) break;
      }
      // 64 gate rows and the same 64 features of up in one copy, or 128 features
      const int a0 = KIND == kForward && t.job == 0 ? t.m * 128 + (int)rank * 64 : m0;
      // 128 rows of an MN-major operand from row r on: 64 rows a copy, or all
      const auto load_mn = [&](uint32_t dst, const CUtensorMap *map, int wide, uint32_t bar, int r, int k0) {
        if (wide) {
          tc::tma_load_pair(dst, map, bar, 0, k0, r >> 6, t.e);
        } else {
          tc::tma_load_pair(dst, map, bar, r, k0, 0, t.e);
          tc::tma_load_pair(dst + 8192, map, bar, r + 64, k0, 0, t.e);
        }
      };
      for (int kb = 0; kb < t.nk; ++kb) {
        ok = __all_sync(0xFFFFFFFFu, wait_bar(empty + 8 * s, ph ^ 1u, limit));
        if (!ok) break;
        const uint32_t sa = smem + s * kStageBytes, sb = sa + kHalfBytes;
        const int k0 = (t.k0 + kb) * kBlockK;
        const uint32_t bar = full0 + 8 * s;
        if (rank == 0) tc::mbar_expect_warp(full + 8 * s, 2 * bytes);
        if (kAMn)
          load_mn(sa, map_a, j.a_wide, bar, m0, k0);
        else
          tc::tma_load_pair(sa, map_a, bar, k0, a0, 0, t.e);
        if (weight)
          load_mn(sb, map_b, j.b_wide, bar, n0, k0);
        else
          tc::tma_load_pair(sb, map_b, bar, k0, n0, 0, t.e);
        if (++s == kStages) {
          s = 0;
          ph ^= 1u;
        }
      }
    }
    // the last commits on this CTA's barriers land before it may exit
    for (int i = 0; ok && i < kStages; ++i) {
      ok = __all_sync(0xFFFFFFFFu, wait_bar(empty + 8 * s, ph ^ 1u, limit));
      if (++s == kStages) {
        s = 0;
        ph ^= 1u;
      }
    }
  } else if (live && warp == 1 && rank == 0) {
    // ---- matrix instructions, one warp of the leading CTA.  What it needs
    // next (the next stage, tile and accumulator) is asked for while the
    // instructions of a stage run, so that the tensor cores have work meanwhile.
    int s = 0;
    uint32_t ph = 0, it = 0;
    bool stage_ready = false, acc_ready = false;
    const uint64_t desc_a0 = tc::smem_desc(smem, kAMn ? 8192u : 16u);
    const uint64_t desc_b0 = tc::smem_desc(smem + kHalfBytes, 16u);
    bool more = feed.next_uniform<kMathWords>(t, ok);
    while (ok && more) {
      if (t.nk == 0) {
        more = feed.next_uniform<kMathWords>(t, ok);
        continue;
      }
      const bool bmn = KIND == kRest && t.job > 0;
      const uint32_t buf = it & 1u;
      const uint32_t d = tmem + buf * kTileCols;
      const uint32_t idesc = tc::instr_desc(256, t.n, kAMn, bmn);
      // 16 k on: 32 bytes of a K-major line, 16 lines (2048 bytes) MN-major
      constexpr uint64_t astep = kAMn ? 128 : 2;
      const uint64_t bstep = bmn ? 128 : 2;
      const uint64_t desc_b = desc_b0 + (bmn ? (uint64_t)((8192u - 16u) >> 4) << 16 : 0);
      // the last block of a weight gradient: no more than its tokens need
      const int tail_rows = bmn ? (t.rows & (kBlockK - 1)) : 0;
      if (!acc_ready)
        ok = __all_sync(0xFFFFFFFFu, wait_bar(tm_empty + 8 * buf, ((it >> 1) & 1u) ^ 1u, limit));
      acc_ready = false;
      tc::fence_after();
      Feed::Raw next_raw;
      bool have = false;                     // the next tile's record is being read
      for (int kb = 0; ok && kb < t.nk; ++kb) {
        if (!stage_ready) {
          ok = __all_sync(0xFFFFFFFFu, wait_bar(full + 8 * s, ph, limit));
          if (!ok) break;
        }
        const bool last = kb == t.nk - 1;
        const uint32_t steps = last && tail_rows != 0 ? (tail_rows + 15) >> 4 : kBlockK / 16;
        tc::fence_after();
        const uint64_t at = (uint64_t)(s * (kStageBytes >> 4));
        const uint32_t stage = empty + 8 * s;
        if (++s == kStages) {
          s = 0;
          ph ^= 1u;
        }
        // the last block asks for the next accumulator, the others for the next record
        const uint32_t bar1 = last || have ? tm_empty + 8 * (buf ^ 1u) : feed.full + 8 * feed.s;
        const uint32_t p1 = last || have ? (((it + 1) >> 1) & 1u) ^ 1u : feed.ph;
        const tc::Asked r = tc::mma_stage(d, desc_a0 + at, desc_b + at, idesc, kb > 0, steps, astep, bstep,
                                          stage, full + 8 * s, ph, bar1, p1);
        stage_ready = __all_sync(0xFFFFFFFFu, r.first);
        const bool second = __all_sync(0xFFFFFFFFu, r.second);
        if (last) {
          acc_ready = second;
        } else if (!have && second) {
          have = true;
          next_raw = feed.read();
        }
      }
      if (ok) tc::mma_commit_pair(tm_full + 8 * buf);
      if (ok) more = have ? feed.spread<kMathWords>(next_raw, t) : feed.next_uniform<kMathWords>(t, ok);
      ++it;
    }
    // the other CTA's arrivals for both accumulators land before this one may exit
    for (int i = 0; ok && i < 2; ++i, ++it)
      ok = __all_sync(0xFFFFFFFFu, wait_bar(tm_empty + 8 * (it & 1u), ((it >> 1) & 1u) ^ 1u, limit));
  } else if (live && warp == 2 && KIND == kActGrad) {
    // ---- the weight gradients' tensor maps: each block writes some experts'
    if constexpr (KIND == kActGrad) {
      if (p.row_maps)
        for (int i = blockIdx.x; i < kRowMaps * p.E; i += gridDim.x) {
          const int e = i % p.E, rows = rows_of(p, e);
          if (rows > 0)                      // an expert without rows has nothing to copy
            tc::map_with_rows(p.row_maps + i, &p.maps.whole[i / p.E], smem_p + kMapOff, (uint32_t)rows);
        }
    }
  } else if (live && warp >= 4) {
    // ---- epilogue: tensor memory -> registers -> shared memory -> results
    uint32_t it = 0;
    const int wq = warp & 3, grp = (warp - 4) >> 2, tid = (threadIdx.x - 128) & 127;
    const uint32_t empty0 = tc::map_rank(tm_empty, 0);
    uint8_t *const stage_p = smem_p + kStages * kStageBytes + grp * 16384;
    const uint32_t stage_u = staging + grp * 16384;
    while (true) {
      const bool more = feed.next(t, ok);
      const uint32_t buf = it & 1u;
      const Job &j = p.job[KIND != kActGrad ? t.job : 0];
      const bool gate = KIND == kForward && t.job == 0;
      // a thread's place in the staged chunk: 4 features of rows r8, r8 + 8, ...
      const int i4 = tid & 15, r8 = tid >> 4;
      const int f0 = gate ? t.m * 128 + (int)rank * 64 + 4 * i4
                                     : t.m * 256 + (int)rank * 128 + 4 * i4;
      const int64_t row0 = (int64_t)t.e * p.cap + t.n0;
      uint2 g[4][2], u[4][2];                // kActGrad: kept gate and up of a chunk
      const auto load_h = [&](int c) {
#pragma unroll
        for (int r = 0; r < 4; ++r)
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
            if (c + r * 8 + r8 < t.cols && f0 + 64 * hf < j.M) {
              const uint16_t *q = j.h + (row0 + c + r * 8 + r8) * 2 * j.M + f0 + 64 * hf;
              g[r][hf] = *reinterpret_cast<const uint2 *>(q);
              u[r][hf] = *reinterpret_cast<const uint2 *>(q + j.M);
            }
      };
      // one token's 4 + 4 features: sums lo, hi -> results
      const auto emit = [&](int tok, int r, const float4 &lo4, const float4 &hi4) {
        const float lo[4] = {lo4.x, lo4.y, lo4.z, lo4.w}, hi[4] = {hi4.x, hi4.y, hi4.z, hi4.w};
        const int64_t row = row0 + tok;
        if (gate) {                          // lo: gate, hi: up of the same features
          if (f0 < j.M) {
            float a[4];
#pragma unroll
            for (int k = 0; k < 4; ++k) a[k] = lo[k] * sigmoid(lo[k]) * hi[k];
            *reinterpret_cast<uint2 *>(j.o0 + row * j.M + f0) = pack4(a);
            if (j.o1) {
              *reinterpret_cast<uint2 *>(j.o1 + row * 2 * j.M + f0) = pack4(lo);
              *reinterpret_cast<uint2 *>(j.o1 + row * 2 * j.M + j.M + f0) = pack4(hi);
            }
          }
        } else if (KIND == kActGrad) {
#pragma unroll
          for (int hf = 0; hf < 2; ++hf)
            if (f0 + 64 * hf < j.M) {
              float gv[4], uv[4], a[4], dg[4], du[4];
              unpack4(g[r][hf], gv);
              unpack4(u[r][hf], uv);
#pragma unroll
              for (int k = 0; k < 4; ++k) {
                const float da = hf ? hi[k] : lo[k];
                const float sg = sigmoid(gv[k]), silu = gv[k] * sg;
                a[k] = silu * uv[k];
                du[k] = da * silu;
                dg[k] = da * uv[k] * (sg + silu * (1.0f - sg));
              }
              *reinterpret_cast<uint2 *>(j.o0 + row * j.M + f0 + 64 * hf) = pack4(a);
              uint16_t *q = j.o1 + row * 2 * j.M + f0 + 64 * hf;
              *reinterpret_cast<uint2 *>(q) = pack4(dg);
              *reinterpret_cast<uint2 *>(q + j.M) = pack4(du);
            }
        } else {
          if (f0 < j.M) *reinterpret_cast<uint2 *>(j.o0 + row * j.M + f0) = pack4(lo);
          if (f0 + 64 < j.M) *reinterpret_cast<uint2 *>(j.o0 + row * j.M + f0 + 64) = pack4(hi);
        }
      };
      if (more && t.nk > 0) {
        if (KIND == kActGrad) load_h(grp * 32);          // while the tile is multiplied
        ok = wait_bar(tm_full + 8 * buf, (it >> 1) & 1u, limit);
        tc::fence_after();
      }
      // all the warps agree to go on, and are done with the staging buffers
      ok = named_sync_and(3, 32 * kEpiWarps, ok);
      if (!ok || !more) break;
      const uint32_t src = tmem + ((uint32_t)(wq * 32) << 16) + buf * kTileCols;
      const auto release = [&] {             // this warp has read its part of the accumulator
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_remote(empty0 + 8 * buf);
      };
      bool wrote = true;                     // this was the tile's last part
      if (KIND == kRest && t.job > 0) {
        // each warp on its own: 32 rows x 64 columns of bf16, swizzled, stored by TMA
        const int m0 = t.m * 256 + (int)rank * 128 + wq * 32;
        if (t.nk > 0 && grp * 64 >= t.n) release();
        for (int c = grp * 64; c < t.n; c += 128) {
          uint32_t v[32], w[32];
#pragma unroll
          for (int hf = 0; hf < 2; ++hf) {
            if (t.nk > 0 && c + hf * 32 < t.n) {
              tc::tmem_ld32(v, src + c + hf * 32);
              tc::tmem_ld_wait();
            } else {
#pragma unroll
              for (int q = 0; q < 32; ++q) v[q] = 0u;
            }
#pragma unroll
            for (int q = 0; q < 16; ++q)
              w[hf * 16 + q] = pack2(__uint_as_float(v[2 * q]), __uint_as_float(v[2 * q + 1]));
          }
          if (t.nk > 0 && c + 128 >= t.n) release();
          // this warp's last store has read the buffer
          if (lane == 0) tc::store_wait_read<0>();
          __syncwarp();
          uint8_t *q = stage_p + wq * 4096 + lane * 128;
#pragma unroll
          for (int k = 0; k < 8; ++k)
            *reinterpret_cast<uint4 *>(q + ((k ^ (lane & 7)) * 16)) =
                make_uint4(w[4 * k], w[4 * k + 1], w[4 * k + 2], w[4 * k + 3]);
          tc::fence_async_smem();
          __syncwarp();
          if (lane == 0) {
            if (m0 < j.M && t.n0 + c < j.N)
              tc::tma_store(&j.out, stage_u + wq * 4096, t.n0 + c, m0, 0, t.e);
            tc::store_commit();
          }
        }
      } else if (KIND != kRest && t.split > 1) {
        // A part of a split contraction leaves its sums in the workspace
        // ([tile][part][CTA][column][128 features]); the last part to finish
        // adds all of them, in the order of the parts.
        const int64_t size = (int64_t)t.part_cols * 128;
        const float *part = p.part + (t.slot * t.split * 2 + (int)rank) * size;
        float *own = p.part + ((t.slot * t.split + t.part) * 2 + (int)rank) * size;
        for (int c = grp * 32; c < t.n; c += 64) {
          uint32_t v[32];
          tc::tmem_ld32(v, src + c);
          tc::tmem_ld_wait();
#pragma unroll
          for (int q = 0; q < 32; ++q)
            __stcg(own + (c + q) * 128 + wq * 32 + lane, __uint_as_float(v[q]));
        }
        release();
        __threadfence();
        named_sync(3, 32 * kEpiWarps);
        if (threadIdx.x == 128) {
          const uint32_t ticket = t.slot * 2 + rank, shift = 4 * (ticket & 7);
          const uint32_t before = atomicAdd(p.tickets + (ticket >> 3), 1u << shift);
          const bool last = ((before >> shift) & 15u) == (uint32_t)t.split - 1;
          if (last) atomicSub(p.tickets + (ticket >> 3), (uint32_t)t.split << shift);
          *last_in = last;
          __threadfence();
        }
        named_sync(3, 32 * kEpiWarps);
        wrote = *last_in != 0;
        if (wrote)
          for (int c = grp * 32; c < t.n; c += 64) {
            float4 lo[4], hi[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) lo[r] = hi[r] = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 2
            for (int s = 0; s < t.split; ++s)
#pragma unroll
              for (int r = 0; r < 4; ++r) {
                const float *q = part + s * 2 * size + (c + r * 8 + r8) * 128 + 4 * i4;
                const float4 a = __ldcg(reinterpret_cast<const float4 *>(q));
                const float4 b = __ldcg(reinterpret_cast<const float4 *>(q + 64));
                lo[r] = make_float4(lo[r].x + a.x, lo[r].y + a.y, lo[r].z + a.z, lo[r].w + a.w);
                hi[r] = make_float4(hi[r].x + b.x, hi[r].y + b.y, hi[r].z + b.z, hi[r].w + b.w);
              }
            if (KIND == kActGrad && c > grp * 32) load_h(c);
#pragma unroll
            for (int r = 0; r < 4; ++r)
              if (c + r * 8 + r8 < t.cols) emit(c + r * 8 + r8, r, lo[r], hi[r]);
          }
      } else {
        if (grp * 32 >= t.n) release();
        float *st = reinterpret_cast<float *>(stage_p);
        for (int c = grp * 32; c < t.n; c += 64) {
          uint32_t v[32];
          tc::tmem_ld32(v, src + c);
          tc::tmem_ld_wait();
          if (c + 64 >= t.n) release();
          if (c > grp * 32) named_sync(1 + grp, 128);      // the last chunk has been read
#pragma unroll
          for (int q = 0; q < 32; ++q) st[q * 128 + wq * 32 + lane] = __uint_as_float(v[q]);
          named_sync(1 + grp, 128);
#pragma unroll
          for (int r = 0; r < 4; ++r) {
            const int tok = r * 8 + r8;
            if (c + tok < t.cols)
              emit(c + tok, r, *reinterpret_cast<const float4 *>(st + tok * 128 + 4 * i4),
                   *reinterpret_cast<const float4 *>(st + tok * 128 + 64 + 4 * i4));
          }
          if (KIND == kActGrad && c + 64 < t.n) load_h(c + 64);
        }
      }
      if (gate && wrote) {
        // half a tile of a is written, for copies of other CTAs to read
        tc::fence_async_global();
        __threadfence();
        named_sync(3, 32 * kEpiWarps);
        if (threadIdx.x == 128) {
          __threadfence();
          atomicAdd(p.units->ready + t.epoch, 1u);
        }
      }
      if (t.nk > 0) ++it;
    }
    if (KIND == kRest && lane == 0) tc::store_wait_all();
  }

  if (!ok) {
    // a wait ran out: report it, and give the copies and products that are
    // already issued (microseconds of work) time to land before the exit
    if (lane == 0) {
      atomicOr(&p.hdr->debug_flags, kFfnBroken);
      report_status(p.hdr, MOE_ERR_TIMEOUT);
      for (int i = 0; i < 1000; ++i) __nanosleep(10000);
    }
  }
  // Neither CTA leaves while the other may still use its shared or tensor
  // memory or its barriers.  The cluster barrier orders nothing: every arrival,
  // copy and commit that comes from the other CTA has been waited for above, by
  // the warp that needed it or, where nobody did (records and accumulators that
  // are free, the last stages' commits), by their owner at its end.  A barrier
  // that releases instead: backward of 128 rows 12.3 us, so 12.0.
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  cluster_arrive_relaxed();
  cluster_wait();
  tc::fence_after();
  if (warp == 2) tc::tmem_free_pair(tmem, kTmemCols);
}

// --- host --------------------------------------------------------------------

// bf16 elements [d3][d2][d1][d0], `s1`, `s2` and `s3` elements apart; boxes of
// deep x rows x 64 elements, 128-byte swizzle.
bool encode(CUtensorMap *m, const void *base, int64_t d0, int64_t d1, int64_t d2, int64_t d3,
            int64_t s1, int64_t s2, int64_t s3, int rows, int deep) {
  const EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)d0, (cuuint64_t)d1, (cuuint64_t)d2, (cuuint64_t)d3};
  const cuuint64_t strides[3] = {(cuuint64_t)s1 * 2, (cuuint64_t)s2 * 2, (cuuint64_t)s3 * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)rows, (cuuint32_t)deep, 1};
  const cuuint32_t step[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void *>(base), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// A dense array [d3][d2][d1][d0].
bool make_map(CUtensorMap *m, const void *base, int64_t d0, int64_t d1, int64_t d2, int64_t d3,
              int rows, int deep = 1) {
  return encode(m, base, d0, d1, d2, d3, d0, d0 * d1, d0 * d1 * d2, rows, deep);
}

// An operand stored [E][k][width], its contraction dimension k outside: one
// copy brings 64 k of 128 rows, as two blocks of 64 rows, where the width is
// whole blocks (*wide: a block must not run into the next row of the array),
// else two copies bring 64 rows each.
bool make_map_mn(CUtensorMap *m, int *wide, const void *base, int64_t width, int64_t k, int64_t E) {
  *wide = width % 128 == 0;
  if (*wide) return encode(m, base, 64, k, width / 64, E, width, 64, k * width, 64, 2);
  return make_map(m, base, width, k, 1, E, 64);
}

template <int KIND>
cudaError_t launch_pair(const PairParams<KIND> &p, int64_t tiles, cudaStream_t stream) {
  static std::once_flag once[64];
  int dev = 0;
  cudaGetDevice(&dev);
  cudaError_t attr = cudaSuccess;
  std::call_once(once[dev & 63], [&] {
    attr = cudaFuncSetAttribute(pair_kernel<KIND>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                (int)kPairSmem);
  });
  if (attr != cudaSuccess) return attr;
  int64_t most = device_sm_count() / 2;
  if (most > kMaxPairs) most = kMaxPairs;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)(2 * (tiles < most ? tiles : most)));
  cfg.blockDim = dim3(kPairThreads);
  cfg.dynamicSmemBytes = kPairSmem;
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, pair_kernel<KIND>, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

template <int KIND>
PairParams<KIND> base_params(const FfnParams &f) {
  PairParams<KIND> p = {};
  p.counts = f.counts;
  p.hdr = f.hdr;
  p.part = f.part;
  p.tickets = f.hdr->reserved + kTicketWord;
  p.units = reinterpret_cast<UnitCounter *>(f.hdr->reserved + kUnitWord);
  p.row_maps = f.dw_gate_up || f.dw_down ? static_cast<CUtensorMap *>(f.row_maps) : nullptr;
  p.E = f.E;
  p.cap = f.cap;
  return p;
}

// Boxes of the tokens' operand: those that tiles of at most cap tokens use.
bool token_maps(Job &j, const void *rows, int64_t width, int64_t cap, int64_t E) {
  for (int i = 0; i < 4; ++i) {
    if (!make_map(&j.b[i], rows, width, cap, 1, E, 16 << i)) return false;
    if (cap <= (32 << i)) break;
  }
  return true;
}

// Units of a row product: its most tiles, each in up to kMaxSplit parts.
int64_t units(const Job &j, const FfnParams &f) {
  const int64_t nk = cdiv(j.K, kBlockK);
  return j.mt * f.E * cdiv(f.cap, kTileCols) * (nk < 16 ? 1 : kMaxSplit);
}

}  // namespace

FfnScratch ffn_scratch(int64_t E, int64_t cap, int64_t H, int64_t I) {
  const int64_t mt = cdiv(I, 128) > cdiv(H, 256) ? cdiv(I, 128) : cdiv(H, 256);
  const int64_t most = mt * E * cdiv(cap, kTileCols) * kMaxSplit;
  const int64_t cols = cap < kTileCols ? (cap + 31) / 32 * 32 : kTileCols;
  FfnScratch s;
  s.maps_off = (size_t)((most < kMaxPairs ? most : kMaxPairs) * cols) * 256 * sizeof(float);
  // the caller's workspace is aligned to 16 bytes, a tensor map to 128
  s.total = s.maps_off + 128 + (size_t)(kRowMaps * E) * sizeof(CUtensorMap);
  return s;
}

cudaError_t launch_ffn(const FfnParams &f, cudaStream_t stream) {
  PairParams<kForward> p = base_params<kForward>(f);
  Job &gu = p.job[0], &d = p.job[1];
  if (!make_map(&gu.a, f.w_gate_up, f.H, f.I, 2, f.E, 64, 2) || !token_maps(gu, f.x, f.H, f.cap, f.E) ||
      !make_map(&d.a, f.w_down, f.I, f.H, 1, f.E, 128) || !token_maps(d, f.act, f.I, f.cap, f.E))
    return cudaErrorInvalidValue;
  gu.o0 = f.act;
  gu.o1 = f.h;
  gu.M = f.I;
  gu.K = f.H;
  gu.mt = (int)cdiv(f.I, 128);
  d.o0 = f.y;
  d.M = f.H;
  d.K = f.I;
  d.mt = (int)cdiv(f.H, 256);
  return launch_pair<kForward>(p, units(gu, f) + units(d, f), stream);
}

cudaError_t launch_ffn_backward(const FfnParams &f, cudaStream_t stream) {
  const int64_t I2 = 2 * (int64_t)f.I;
  // what the weight gradients contract: dh and x, dy and a
  const void *operand[kRowMaps] = {f.dh, f.x, f.dy, f.act};
  const int64_t width[kRowMaps] = {I2, f.H, f.H, f.I};
  int wide[kRowMaps];
  {
    PairParams<kActGrad> p = base_params<kActGrad>(f);       // dh and a
    Job &j = p.job[0];
    if (!make_map_mn(&j.a, &j.a_wide, f.w_down, f.I, f.H, f.E) || !token_maps(j, f.dy, f.H, f.cap, f.E))
      return cudaErrorInvalidValue;
    for (int i = 0; i < kRowMaps; ++i)
      if (!make_map_mn(&p.maps.whole[i], &wide[i], operand[i], width[i], f.cap, f.E))
        return cudaErrorInvalidValue;
    j.o0 = f.act;
    j.o1 = f.dh;
    j.h = f.h;
    j.M = f.I;
    j.K = f.H;
    j.mt = (int)cdiv(f.I, 256);
    const cudaError_t e = launch_pair<kActGrad>(p, units(j, f), stream);
    if (e != cudaSuccess) return e;
  }
  // dx first: its tiles have the longest contraction
  PairParams<kRest> p = base_params<kRest>(f);
  int64_t tiles = 0;
  if (f.dx) {
    Job &j = p.job[0];
    if (!make_map_mn(&j.a, &j.a_wide, f.w_gate_up, f.H, I2, f.E) || !token_maps(j, f.dh, I2, f.cap, f.E))
      return cudaErrorInvalidValue;
    j.o0 = f.dx;
    j.M = f.H;
    j.K = (int)I2;
    j.mt = (int)cdiv(f.H, 256);
    tiles += j.mt * f.E * cdiv(f.cap, kTileCols);
  }
  for (int w = 0; w < 2; ++w) {
    uint16_t *out = w ? f.dw_down : f.dw_gate_up;
    if (!out) continue;
    Job &j = p.job[1 + w];
    const int64_t M = width[2 * w], N = width[2 * w + 1];
    if (!make_map(&j.out, out, N, M, 1, f.E, 32)) return cudaErrorInvalidValue;
    j.a_wide = wide[2 * w];
    j.b_wide = wide[2 * w + 1];
    j.M = (int)M;
    j.N = (int)N;
    j.mt = (int)cdiv(M, 256);
    tiles += j.mt * cdiv(N, kTileCols) * f.E;
  }
  return tiles > 0 ? launch_pair<kRest>(p, tiles, stream) : cudaSuccess;
}

}  // namespace moe
