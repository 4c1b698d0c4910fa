// moe_ffn_mxfp4.cu -- the experts' gated feed-forward on 4-bit operands, as
// grouped block-scaled matrix products on the tensor cores.
//
// What it computes, for expert e and its count[e] rows x, all operands MXFP4
// (blocks of 32 elements with a power of two each):
//   h = x Wgu^T (gate | up),  a = SiLU(gate) * up,  a4 = MXFP4(a),  y = a4 Wd^T.
//
// How: one launch.  The order of the work, the pairs of CTAs and their warps' roles
// are moe_ffn.cu's (moe_pairs.cuh): weights' output features on the 256-row side,
// the expert's tokens on the column side, a ring of stages filled by TMA,
// tcgen05.mma.cta_group::2, accumulators in tensor memory two tiles deep, eight
// epilogue warps.  What 4 bits change:
//  - A stage is 256 k (128 bytes of a row, as 64 k of bf16 are): 16 KB of weights
//    per CTA, up to 16 KB of tokens, 1 KB of the weights' scales and up to 3 KB of
//    the tokens'.  The scales stand in memory in the tiles that a copy into tensor
//    memory takes (tcgen05.cp), so that they come by TMA and go on without passing
//    through registers.  Both CTAs need the scales of all the tile's tokens.
//  - Gate and up of the same 64 features are the two halves of a CTA's 128 rows;
//    their scales lie so in memory (MOE_MXFP4_GATE_UP).
//  - Scales take 32 columns of tensor memory, which leaves 480 for two
//    accumulators of 256: they overlap by 32 columns.  The epilogue reads those
//    first, and the next tile starts when it has.  Tiles of up to 224 columns do
//    not overlap.
//  - a is quantised where it is computed: through shared memory a lane gets 16
//    features of one token, so that a block is two lanes.
//  - Tiles are four times shorter in time than bf16's, so that what happens once a
//    tile counts.  A warp of its own waits for the stores of a and publishes
//    them; the two epilogue groups agree only where a tile is cut; an expert's
//    tokens are dealt out to its tiles in steps of 64 (a last tile of a few tokens
//    takes 0.2 us a stage however few they are, a full one 0.28).  Batch of 8192
//    rows, step by step: four features a lane and a maximum over eight lanes 536 us;
//    no fence in the epilogue 479; lanes per token 447; groups apart and weights of y
//    ahead of its wait 441; even tiles 433; whole sectors of codes 424.
//  - Tiles of y wait for a of their own group of experts, of seven, instead of all of
//    a (31 uneven experts 43.8 us, so 39.1; GroupCounter, kLongY).
//
// Rounding: products of E2M1 numbers and powers of two, summed in binary32; a is
// rounded to MXFP4 from binary32, y to bf16, once each.
//
// What bounds it, measured on GB300 (copy 6.78 TB/s):
//  - DeepSeek-V3-shaped decode (256 experts, 32 rows each, 6.0 GB of 4-bit
//    weights): 887 us, 6.9 TB/s: the weights' reading (bf16: 3325 us).
//  - Mixtral-shaped batch (8192 rows over 8 experts, H 4096, I 14336): 412 to 430
//    us alone, 6.7 to 7.0 PFLOP/s; 466 to 483 after some tenths of a second, when
//    the power limit lowers the clock (bf16: 1.79 to 1.87 ms).  The products alone,
//    nothing copied and no results written, take 360 of 415 us, 318 ns for each of a
//    pair's 1132 stages: 300 us of instructions (512 cycles a stage), 0.6 us between
//    two tiles, 9 us until the first is multiplied, and y's last round, in which half
//    of the pairs have no tile.  Without the copies 369 us, without the results 382,
//    without the products 323: the three delay one another by 55 us, on what is not
//    established.  (A full stage is 72 KB a pair: 15 TB/s from the L2 on average.)
//    Tensor pipe active 68 % of the cycles at a quarter of the rows.
//  - One token over two Mixtral-shaped experts (187 MB): 40.5 us, of 27.6: the
//    second expert's wait between a and y, and joining y's parts, 4 to 5 us each,
//    and the start.  Bringing Wd into the L2 during the wait changed nothing.
//  - Many tokens and contractions below about 3700: the epilogue, 3 to 4 us for a
//    tile of a of 256 x 256, as long as 11 to 14 stages.  65536 rows over 128 experts,
//    H 2048, I 768: 210 us, 118 without its results; 8192 rows over 16, H and I 2048:
//    59 and 43.  More epilogue warps (12 or 16) were slower.
//  - Tiny calls: latency, as moe_ffn.cu.
#include <mutex>

#include "moe_mxfp4.cuh"
#include "moe_pairs.cuh"

namespace moe {

namespace {

constexpr int kGroups = 2;             // of four epilogue warps; each takes every kGroups-th chunk of columns
constexpr int kOutWarps = 4 * kGroups;
constexpr int kThreads = 128 + 32 * kOutWarps;     // warps: 0 TMA, 1 MMA, 2 publishing, 3 scheduling, then the epilogue
constexpr int kStages = 5;
constexpr int kBlockK = 256;           // one 128-byte swizzled line of 4-bit elements
constexpr uint32_t kHalfBytes = 128 * 128;               // a CTA's half of one operand: 16 KB
constexpr uint32_t kScaleOff = 2 * kHalfBytes;           // A's scales: 2 tiles, one for each 128 k
constexpr uint32_t kScaleStage = 2 * kScaleTileBytes;
constexpr uint32_t kStageBytes = kScaleOff + 4 * kScaleStage;   // and B's: 2, 4 or 6 tiles
// Epilogue: 32 tokens of gate and up for each group, 128 features in a row, which
// 16-byte reads of different tokens find in different banks.
constexpr int kStagedRow = 132;
constexpr uint32_t kStagingBytes = kGroups * 32 * kStagedRow * 4;
constexpr uint32_t kBarOff = kStages * kStageBytes + kStagingBytes;
constexpr uint32_t kRingOff = kBarOff + 256;
constexpr uint32_t kSmem = kRingOff + kRing * 64 + 1024;        // + alignment slack
static_assert(kSmem <= 232448, "shared memory of one CTA");
static_assert(kStageBytes % 1024 == 0, "swizzled tiles start on 1024 bytes");
// Tensor memory: the scales, then two accumulators of 256 columns that share
// kShared of them.
constexpr uint32_t kAcc0 = 32, kAcc1 = 256;
constexpr int kShared = (int)(kAcc0 + kTileCols - kAcc1);       // a multiple of the epilogue's chunks of 32
constexpr int kApart = kTileCols - kShared;                     // tiles of so many columns share none
// Tiles announced ahead, less than the ring holds: one taken early cannot go to a
// pair that is free sooner, one taken late comes too late.  Measured with 2, 3 and
// 4: one token 41.9, 42.3 and 43.3 us, the Mixtral-shaped batch 462, 428 and 428 (all
// of a waited for).
constexpr uint32_t kAhead = 3;
static_assert(kAhead <= kRing, "a record's place is free when it is written");
// Blocks of a tile of y from which on a pair holds one alone until all of a is
// written: its second one would be missing where a pair is still busy with a, but
// begins sooner.  Measured holding and not, 8 experts, H 4096, with 64, 1024, 2048 and
// 4096 rows: 9 blocks 31.2 and 27.2, 35.6 and 31.7, 44.9 and 39.5 us; 16 blocks 43.6
// and 41.5, 48.5 and 46.1, 61.7 and 58.6; 24 blocks 58.1 and 55.5, 63.3 and 60.8, 78.8
// and 79.1, 110.2 and 106.6; 28 blocks 62.9 and 64.6, 69.0 and 71.2, 87.5 and 89.8, 125.2
// and 122.3; 40 blocks 87.1 and 90.1, 94.6 and 100.9, 117.5 and 124.5, 172.4 and 172.2;
// 56 blocks 117 and 121, 126 and 134, 157 and 170, 259 and 261.  (48 blocks go either
// way by 1 %.)  H 7168, 64 and 1024 rows: 16 blocks 68.1 and 63.3, 75.2 and 70.3; 28
// blocks 103.3 and 108.3, 111.2 and 115.4.  8 blocks (DeepSeek-V3-shaped), 64 rows over
// 256 experts 214 and 206, decode 895 and 887; 4 blocks, 31 uneven experts 44.5 and
// 39.1; one token the same at every length.
constexpr int kLongY = 28;
static_assert(kShared == 32, "the epilogue reads the shared columns as one chunk");

// Words of a tile's record that the matrix instructions need.
constexpr uint32_t kMxWords = kMathWords | kN0 | kK0;

// Row tiles of scales that a tile's columns lie in: its first is row 0 or 64 of one.
__device__ __forceinline__ int scale_tiles(const Tile &t) { return ((t.n0 & 64) + t.n + 127) >> 7; }

struct MxJob {
  CUtensorMap a, a_scale;
  CUtensorMap b[4], b_scale[3];        // boxes of 16, 32, 64 and 128 tokens; of 1, 2 and 3 row tiles of scales
  uint8_t *q, *scale;                  // gate and up: a4
  uint16_t *out;                       // y
  int M, K, N;                         // features, contraction; N is not used
  int mt;                              // tiles of 256 accumulator rows (gate and up: of 128 features)
  int row_tiles, block_tiles;          // of a4's scales
};

// What is written of a, by groups of experts, so that the first experts' tiles of y
// need not wait for the last experts' a.  In the header's reserved words past the
// tickets; the counters of the other epoch are 0 between launches.
constexpr int kGroupWord = kTicketWord + kMaxPairs * 2 * 4 / 32;
// Seven groups are what those words hold.  Measured with 1 (all of a), 2, 4 and 7:
// 31 uneven experts 43.8, 40.0, 39.5 and 39.1 us; 64 rows over 256 experts 211, 205, 205
// and 206; decode 891, 885, 886 and 887; one token 42.4, 41.3, 40.7 and 40.7; 4096 rows
// over 128 experts (H 2048, I 768) 66.9, 64.3, 64.9 and 66.5.
struct GroupCounter {
  uint32_t epoch;                      // which of `ready` counts this launch's
  uint32_t ready[2][7];                // CTAs' halves of tiles of a that are written
};
static_assert(kGroupWord * 4 + sizeof(GroupCounter) <= sizeof(WsHeader::reserved), "the groups fit");

struct MxParams {
  static constexpr int kKind = kForward, kBlock = kBlockK, kJobs = 2, kExpertGroups = 7;
  static constexpr int kTileStep = 64;   // block scales come 128 rows at a time, from row 0 or 64 on
  MxJob job[kJobs];                    // a, y
  const int32_t *counts;               // [E], or null (cap rows each)
  WsHeader *hdr;
  float *part;                         // partial sums of split contractions
  uint32_t *tickets;                   // finished parts, 4 bits for each split tile and CTA of the pair
  UnitCounter *units;
  GroupCounter *groups;
  int E, cap;
};

__global__ void __launch_bounds__(kThreads, 1) __cluster_dims__(2, 1, 1)
ffn_mxfp4_kernel(const __grid_constant__ MxParams p) {
  extern __shared__ uint8_t smem_raw[];
  const uint32_t smem = (smem_u32(smem_raw) + 1023u) & ~1023u;
  uint8_t *smem_p = smem_raw + (smem - smem_u32(smem_raw));
  // the same value in every lane, and known to be
  const int warp = __shfl_sync(0xFFFFFFFFu, threadIdx.x >> 5, 0), lane = threadIdx.x & 31;
  const uint32_t rank = cluster_cta_rank();

  const uint32_t bars = smem + kBarOff;
  const uint32_t full = bars, empty = bars + 8 * kStages;
  const uint32_t tm_full = bars + 16 * kStages, tm_empty = tm_full + 16, tm_shared = tm_empty + 16;
  const uint32_t tm_slot = tm_shared + 16;
  constexpr uint32_t kSlotOff = kBarOff + 16 * kStages + 48, kLastOff = kSlotOff + 8;
  static_assert(kLastOff + 8 <= kBarOff + 144 && 144 + 8 * kRing <= 192, "the barriers fit");
  // barriers of the ring of tiles: announced, read by all, results written
  const uint32_t rec_done = bars + 144;
  const uint32_t rec_full = bars + 192, rec_empty = bars + 224;
  Tile *ring = reinterpret_cast<Tile *>(smem_p + kRingOff);
  volatile uint32_t *gave_up = reinterpret_cast<uint32_t *>(smem_p + kLastOff + 4);
  volatile uint32_t *last_in = reinterpret_cast<uint32_t *>(smem_p + kLastOff);

  if (threadIdx.x == 0) {
    *gave_up = 0u;
    for (int s = 0; s < kStages; ++s) {
      tc::mbar_init_at(full + 8 * s, 1);     // the leader's arrival, and the bytes of both CTAs
      tc::mbar_init_at(empty + 8 * s, 1);    // the commit of the stage's instructions
    }
    for (int b = 0; b < 2; ++b) {
      tc::mbar_init_at(tm_full + 8 * b, 1);
      tc::mbar_init_at(tm_empty + 8 * b, 2 * kOutWarps);   // the epilogue warps of both CTAs
      tc::mbar_init_at(tm_shared + 8 * b, 2 * kOutWarps);
    }
    for (int r = 0; r < kRing; ++r) {
      tc::mbar_init_at(rec_full + 8 * r, 1);
      // in the leader: TMA, publishing and epilogue of both CTAs, and the MMA warp
      tc::mbar_init_at(rec_empty + 8 * r, 2 * (kOutWarps + 2) + 1);
      tc::mbar_init_at(rec_done + 8 * r, kOutWarps);
    }
    asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
  } else if (threadIdx.x == 32) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      tc::prefetch_map(&p.job[j].a);
      tc::prefetch_map(&p.job[j].a_scale);
    }
    tc::prefetch_map(&p.job[0].b[0]);
    tc::prefetch_map(&p.job[0].b_scale[0]);
  }
  if (warp == 2) tc::tmem_alloc_pair(tm_slot, kTmemCols);
  tc::fence_before();
  __syncthreads();
  cluster_arrive_relaxed();              // the barriers' initial values are released above
  cluster_wait();
  tc::fence_after();
  const uint32_t tmem = *reinterpret_cast<volatile uint32_t *>(smem_p + kSlotOff);

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
    // tiles to both CTAs.  A unit belongs to a pair that runs, since others will
    // wait for it.
    Schedule<MxParams> sched(p);
    const uint32_t peer_full = tc::map_rank(rec_full, 1), peer_ring = tc::map_rank(smem + kRingOff, 1);
    int written = -1;                        // the group of the last tile of y whose a is there, or all
    const uint32_t epoch = rank == 0 ? __ldcg(&p.groups->epoch) & 1u : 0u;
    uint32_t c = 0;
    for (; live && rank == 0; ++c) {
      const uint32_t s = c % kRing;
      // A unit is taken once the record kAhead before it has been read by every
      // warp of both CTAs.
      if (c >= kAhead) {
        const uint32_t r = c - kAhead;
        ok = __all_sync(0xFFFFFFFFu, wait_bar(rec_empty + 8 * (r % kRing), (r / kRing) & 1u, limit));
        if (!ok) break;
      }
      // One tile of y for each pair until its a is written, or, where y's tiles are
      // long, all of a: a second one would be missing where a pair is still busy
      // with a.
      if (c > 0 && t.need != 0) {
        if (t.nk >= kLongY) {
          for (int g = 0; ok && written < 0 && g < MxParams::kExpertGroups; ++g)
            ok = __all_sync(0xFFFFFFFFu, wait_count(&p.groups->ready[epoch][g], (uint32_t)sched.count_group(g), limit));
          written = 0;
        } else if (group_of(p, t.e) != written) {
          written = group_of(p, t.e);
          ok = __all_sync(0xFFFFFFFFu, wait_count(&p.groups->ready[epoch][written], (uint32_t)t.need, limit));
        }
        if (!ok) break;
      }
      unsigned long long n = 0;
      if (lane == 0) n = atomicAdd(&p.units->next, 1ull);
      t.valid = sched.find((int64_t)__shfl_sync(0xFFFFFFFFu, n, 0), t);
      t.epoch = epoch;
      if (lane == 0) {
        ring[s] = t;
        tc::mbar_arrive_local(rec_full + 8 * s);
      }
      __syncwarp();
      if (lane == 0) tc::mbar_expect_at(peer_full + 8 * s, sizeof(Tile));
      if (lane < 4)
        tc::store_async(peer_ring + s * (uint32_t)sizeof(Tile) + lane * 16,
                        reinterpret_cast<const uint4 *>(ring + s)[lane], peer_full + 8 * s);
      if (!t.valid) break;
    }
    // the other CTA's arrivals for the records before the last (number c) land
    // before this one may exit
    if (live && rank == 0)
      for (uint32_t r = c < kRing ? 0 : c - kRing + 1; ok && r < c; ++r)
        ok = __all_sync(0xFFFFFFFFu, wait_bar(rec_empty + 8 * (r % kRing), (r / kRing) & 1u, limit));
    if (rank == 0 && lane == 0 && atomicAdd(&p.units->done, 1u) == (gridDim.x >> 1) - 1) {
      // every pair knows this launch's epoch by now: the next one counts in the
      // other counters, which nobody uses any more
      p.units->next = 0;
      p.units->done = 0;
      for (int g = 0; g < MxParams::kExpertGroups; ++g) p.groups->ready[epoch ^ 1u][g] = 0;
      p.groups->epoch = epoch ^ 1u;
    }
  } else if (live && warp == 0) {
    // ---- TMA: both CTAs load their halves; bytes complete on the leader's barrier
    int s = 0;
    uint32_t ph = 0;
    const uint32_t full0 = tc::map_rank(full, 0);
    int written = -1;                        // the group of the last tile of y whose a is there
    while (ok && feed.next_uniform<kCopyWords>(t, ok)) {
      const MxJob &j = p.job[t.job];
      const uint32_t half_n = t.n >> 1;
      const int bsel = half_n <= 16 ? 0 : half_n <= 32 ? 1 : half_n <= 64 ? 2 : 3;
      const int tiles = scale_tiles(t);
      const uint32_t bytes = kHalfBytes + (16u << bsel) * 128u + (1u + tiles) * kScaleStage;
      const int n0 = t.n0 + (int)(rank * half_n), rt = t.m * 2 + (int)rank;
      // 64 gate rows and the same 64 features of up in one copy, or 128 features
      const int a0 = rt * (t.job == 0 ? 64 : 128);
      // A group's first tile of y takes its first stages' weights before it waits for
      // the group's a.
      const int early = t.need != 0 && group_of(p, t.e) != written ? min(t.nk, kStages) : 0;
      for (int kb = 0; ok && kb < early; ++kb) {
        const int at = s + kb < kStages ? s + kb : s + kb - kStages;
        ok = __all_sync(0xFFFFFFFFu, wait_bar(empty + 8 * at, ph ^ (s + kb < kStages ? 1u : 0u), limit));
        if (!ok) break;
        const uint32_t sa = smem + at * kStageBytes;
        if (rank == 0) tc::mbar_expect_warp(full + 8 * at, 2 * bytes);
        tc::tma_load_pair(sa, &j.a, full0 + 8 * at, (t.k0 + kb) * 128, a0, 0, t.e);
        tc::tma_load_pair(sa + kScaleOff, &j.a_scale, full0 + 8 * at, 0, 2 * (t.k0 + kb), rt, t.e);
      }
      if (!ok) break;
      if (early > 0) {
        written = group_of(p, t.e);
        ok = __all_sync(0xFFFFFFFFu, wait_count(&p.groups->ready[t.epoch][written], (uint32_t)t.need, limit));
        if (!ok) break;
      }
      for (int kb = 0; kb < t.nk; ++kb) {
        const uint32_t sa = smem + s * kStageBytes;
        const int k = t.k0 + kb;
        const uint32_t bar = full0 + 8 * s;
        if (kb >= early) {
          ok = __all_sync(0xFFFFFFFFu, wait_bar(empty + 8 * s, ph ^ 1u, limit));
          if (!ok) break;
          if (rank == 0) tc::mbar_expect_warp(full + 8 * s, 2 * bytes);
          tc::tma_load_pair(sa, &j.a, bar, k * 128, a0, 0, t.e);
          tc::tma_load_pair(sa + kScaleOff, &j.a_scale, bar, 0, 2 * k, rt, t.e);
        }
        tc::tma_load_pair(sa + kHalfBytes, &j.b[bsel], bar, k * 128, n0, 0, t.e);
        tc::tma_load_pair(sa + kScaleOff + kScaleStage, &j.b_scale[tiles - 1], bar, 0, 2 * k, t.n0 >> 7, t.e);
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
    // An answer takes about 200 cycles, more beside the epilogue's shared-memory
    // traffic: it is looked at one stage later, and the stage that is asked for is
    // the one after next (asked for the next and looked at at once, an iteration
    // took longer than the stage's instructions).
    int s = 0, s2 = 1;                       // this stage, the next one
    uint32_t ph = 0, ph2 = 0, it = 0;
    uint32_t ready = 0, ready_next = 0;      // answers: this stage, the next one
    bool acc_ready = false;
    int before = 0;                          // columns of the tile before
    const uint64_t desc_a0 = tc::smem_desc(smem, 16u), desc_b0 = tc::smem_desc(smem + kHalfBytes, 16u);
    const uint64_t desc_sa0 = tc::scale_desc(smem + kScaleOff);
    const uint64_t desc_sb0 = tc::scale_desc(smem + kScaleOff + kScaleStage);
    bool more = feed.next_uniform<kMxWords>(t, ok);
    while (ok && more) {
      const uint32_t buf = it & 1u;
      const uint32_t d = tmem + (buf ? kAcc1 : kAcc0);
      const uint32_t idesc = tc::instr_desc_mx(256, t.n);
      const uint32_t tiles = scale_tiles(t), skip = (uint32_t)(t.n0 & 64) >> 5;
      // 64 k an instruction; the row's end cuts the last block
      const int left = p.job[t.job].K - (t.k0 + t.nk - 1) * kBlockK;
      const uint32_t tail = left >= kBlockK ? 4u : (uint32_t)((left + 63) >> 6);
      if (!acc_ready)
        ok = __all_sync(0xFFFFFFFFu, wait_bar(tm_empty + 8 * buf, ((it >> 1) & 1u) ^ 1u, limit));
      acc_ready = false;
      // the columns that it shares with the tile before, if either has so many
      if (ok && it > 0 && (buf ? before : t.n) > kApart)
        ok = __all_sync(0xFFFFFFFFu, wait_bar(tm_shared + 8 * (buf ^ 1u), ((it - 1) >> 1) & 1u, limit));
      before = t.n;
      tc::fence_after();
      const uint32_t acc_bar = tm_empty + 8 * (buf ^ 1u), acc_parity = (((it + 1) >> 1) & 1u) ^ 1u;
      Feed::Raw next_raw;
      bool have = false;                     // the next tile's record is being read
      uint32_t answer = 0;                   // to the last question: the record, or the accumulator
      for (int kb = 0; ok && kb < t.nk; ++kb) {
        if (!__all_sync(0xFFFFFFFFu, ready)) {
          ok = __all_sync(0xFFFFFFFFu, wait_bar(full + 8 * s, ph, limit));
          if (!ok) break;
        }
        if (__all_sync(0xFFFFFFFFu, answer)) {
          if (have) {
            acc_ready = true;
          } else {
            have = true;
            next_raw = feed.read();
          }
        }
        const uint32_t steps = kb == t.nk - 1 ? tail : 4u;
        tc::fence_after();
        const uint64_t at = (uint64_t)(s * (kStageBytes >> 4));
        const uint32_t stage = empty + 8 * s;
        s = s2;
        ph = ph2;
        if (++s2 == kStages) {
          s2 = 0;
          ph2 ^= 1u;
        }
        tc::load_scales(tmem, desc_sa0 + at, desc_sb0 + at, steps > 2, tiles);
        const tc::Asked r = tc::mma_stage_mx(d, desc_a0 + at, desc_b0 + at, idesc, tmem, skip, kb > 0, steps, stage,
                                             full + 8 * s2, ph2, have ? acc_bar : feed.full + 8 * feed.s,
                                             have ? acc_parity : feed.ph);
        ready = ready_next;
        ready_next = r.first;
        answer = r.second;
      }
      if (ok) tc::mma_commit_pair(tm_full + 8 * buf);
      if (ok) {
        if (have) acc_ready = acc_ready || __all_sync(0xFFFFFFFFu, answer);
        more = have ? feed.spread<kMxWords>(next_raw, t) : feed.next_uniform<kMxWords>(t, ok);
      }
      ++it;
    }
    // the other CTA's arrivals for both accumulators land before this one may exit
    for (int i = 0; ok && i < 2; ++i, ++it) {
      const uint32_t parity = ((it >> 1) & 1u) ^ 1u;
      ok = __all_sync(0xFFFFFFFFu, wait_bar(tm_empty + 8 * (it & 1u), parity, limit) &&
                                       wait_bar(tm_shared + 8 * (it & 1u), parity, limit));
    }
  } else if (live && warp == 2) {
    // ---- publishing: says that half a tile of a is written, for copies of other
    // CTAs to read, when all epilogue warps are done with it.  The fence waits for
    // their stores: in the epilogue it delayed the next tile by 0.6 us.
    while (true) {
      ok = __all_sync(0xFFFFFFFFu, wait_bar(rec_full + 8 * feed.s, feed.ph, limit));
      if (!ok) break;
      t = ring[feed.s];
      __syncwarp();
      if (!t.valid) break;
      // (Such tiles come before all others: their places' phases are the ring's.)
      if (t.job == 0 && t.split == 1) {
        ok = __all_sync(0xFFFFFFFFu, wait_bar(rec_done + 8 * feed.s, feed.ph, limit));
        if (!ok) break;
        tc::fence_async_global();
        __threadfence();
        if (lane == 0) atomicAdd(&p.groups->ready[t.epoch][group_of(p, t.e)], 1u);
      }
      feed.leave();
    }
  } else if (live && warp >= 4) {
    // ---- epilogue: tensor memory -> registers (a lane has one feature of 32
    // tokens) -> results
    uint32_t it = 0;
    const int wq = warp & 3, grp = (warp - 4) >> 2;
    const uint32_t empty0 = tc::map_rank(tm_empty, 0), shared0 = tc::map_rank(tm_shared, 0);
    float *const staged = reinterpret_cast<float *>(smem_p + kStages * kStageBytes) + grp * 32 * kStagedRow;
    while (true) {
      const int slot = feed.s;
      const bool more = feed.next(t, ok);
      const uint32_t buf = it & 1u;
      const MxJob &j = p.job[t.job];
      const bool gate = t.job == 0;
      const int rt = t.m * 2 + (int)rank;
      const int64_t row0 = (int64_t)t.e * p.cap + t.n0;
      // 32 tokens' sums of this lane's feature, from column c on -> results.  The
      // four warps of a group call it together.
      const auto emit = [&](int c, const uint32_t (&v)[32]) {
        if (gate) {
          // Through shared memory, so that a lane gets 16 features of one token: half
          // of a block, whose largest magnitude is then one exchange away, and four
          // lanes the token's 64, a whole sector of codes.  (With a lane per feature
          // and the maximum over the warp's lanes the chunk took twice as long.)
          float *const own = staged + wq * 32 + lane;
#pragma unroll
          for (int i = 0; i < 32; ++i) own[i * kStagedRow] = __uint_as_float(v[i]);
          named_sync(1 + grp, 128);
          const int at = 8 * wq + (lane & 7), f = 16 * (lane >> 3);
          const float4 *const in = reinterpret_cast<const float4 *>(staged + at * kStagedRow + f);
          float a[16];
          uint32_t most = 0;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            const float4 g4 = in[i], u4 = in[16 + i];
            const float g[4] = {g4.x, g4.y, g4.z, g4.w}, u[4] = {u4.x, u4.y, u4.z, u4.w};
#pragma unroll
            for (int k = 0; k < 4; ++k) {
              a[4 * i + k] = g[k] * sigmoid(g[k]) * u[k];
              most = max(most, __float_as_uint(a[4 * i + k]) & 0x7FFFFFFFu);
            }
          }
          named_sync(1 + grp, 128);          // all have read: the next chunk may be staged
          most = max(most, __shfl_xor_sync(0xFFFFFFFFu, most, 8));
          const uint32_t byte = mx_scale(most >> 23);
          const float inv = mx_inverse(byte);
          uint32_t code[2];
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float x[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) x[k] = byte == 255u ? 0.0f : a[8 * i + k] * inv;
            code[i] = e2m1x8(x);
          }
          const int tok = c + at, feature = rt * 64 + f;
          // features past the last have a scale of 0 in the last tile of blocks
          const uint32_t scale = feature < j.M ? byte : 0u;
          const uint32_t scales = scale | __shfl_down_sync(0xFFFFFFFFu, scale, 16) << 8;
          if (tok < t.cols) {
            if (feature < j.M)
              *reinterpret_cast<uint2 *>(j.q + ((row0 + tok) * j.M + feature) / 2) = make_uint2(code[0], code[1]);
            if (lane < 8) {
              const int r = t.n0 + tok;
              const int64_t tile = ((int64_t)t.e * j.row_tiles + (r >> 7)) * j.block_tiles + t.m;
              *reinterpret_cast<uint16_t *>(j.scale + tile * kScaleTileBytes + (r & 31) * 16 +
                                            ((r >> 5) & 3) * 4 + 2 * rank) = (uint16_t)scales;
            }
          }
        } else {
          // two tokens in a word, then two features of one: even lanes the first
          // token, odd ones the second
          const int f = rt * 128 + wq * 32;
          uint16_t *q = j.out + (row0 + c + (lane & 1)) * j.M + f + (lane & ~1);
#pragma unroll
          for (int i = 0; i < 32; i += 2) {
            const uint32_t w = pack2(__uint_as_float(v[i]), __uint_as_float(v[i + 1]));
            const uint32_t o = __shfl_xor_sync(0xFFFFFFFFu, w, 1);
            if (f < j.M && c + i + (lane & 1) < t.cols)
              *reinterpret_cast<uint32_t *>(q + (int64_t)i * j.M) =
                  (lane & 1) ? __byte_perm(o, w, 0x7632) : __byte_perm(w, o, 0x5410);
          }
        }
      };
      if (more) {
        // (the warp decides as one: it reads tensor memory next)
        ok = __all_sync(0xFFFFFFFFu, wait_bar(tm_full + 8 * buf, (it >> 1) & 1u, limit));
        tc::fence_after();
      }
      const uint32_t src = tmem + ((uint32_t)(wq * 32) << 16) + (buf ? kAcc1 : kAcc0);
      const auto arrive = [&](uint32_t bar) {     // this warp has read its part of the columns
        tc::fence_before();
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_remote(bar + 8 * buf);
      };
      // The group's chunks of 32 columns, those that the accumulators share first:
      // the first accumulator's last, the second's first.
      const int chunks = (t.n - grp * 32 + 32 * kGroups - 1) / (32 * kGroups);     // t.n >= 32
      const bool shares = buf ? grp == 0 : grp == (kApart / 32) % kGroups && t.n > kApart;
      const auto chunk = [&](int i) { return grp * 32 + 32 * kGroups * (buf ? i : chunks - 1 - i); };
      const auto read = [&](int i, uint32_t (&v)[32]) {
        tc::tmem_ld32(v, src + chunk(i));
        tc::tmem_ld_wait();
        if (i == 0 && shares) arrive(shared0);
        if (i == chunks - 1) arrive(empty0);
      };
      // The first chunk at once: the next tile may be waiting for it.
      uint32_t v[32];
      if (ok && more) {
        if (!shares) arrive(shared0);
        if (chunks > 0) read(0, v);
        else arrive(empty0);
      }
      // A group's warps agree to go on.  Both groups do where a tile is cut, which
      // they finish together; one that has given up says so at that barrier.  (Both
      // agreeing on every tile cost the batch's tiles 0.3 us each.)
      ok = named_sync_and(1 + grp, 128, ok);
      if (!ok) {
        *gave_up = 1u;
        __threadfence_block();
        named_arrive(3, 32 * kOutWarps);
        break;
      }
      if (!more) break;
      if (t.split > 1) {
        named_sync(3, 32 * kOutWarps);
        if (*gave_up) {
          ok = false;
          break;
        }
      }
      bool wrote = true;                     // this was the tile's last part
      const int64_t size = (int64_t)t.part_cols * 128;
      const float *const part = p.part + (t.slot * t.split * 2 + (int)rank) * size + wq * 32 + lane;
      if (t.split > 1) {
        // A part of a split contraction leaves its sums in the workspace
        // ([tile][part][CTA][column][128 features]); the last part to finish
        // adds all of them, in the order of the parts.
        float *own = p.part + ((t.slot * t.split + t.part) * 2 + (int)rank) * size + wq * 32 + lane;
        for (int i = 0; i < chunks; ++i) {
          if (i > 0) read(i, v);
          const int c = chunk(i);
#pragma unroll
          for (int q = 0; q < 32; ++q)
            if (c + q < t.cols) __stcg(own + (c + q) * 128, __uint_as_float(v[q]));
        }
        named_sync(3, 32 * kOutWarps);
        if (threadIdx.x == 128) {
          __threadfence();
          const uint32_t ticket = t.slot * 2 + rank, shift = 4 * (ticket & 7);
          const uint32_t was = atomicAdd(p.tickets + (ticket >> 3), 1u << shift);
          const bool last = ((was >> shift) & 15u) == (uint32_t)t.split - 1;
          if (last) atomicSub(p.tickets + (ticket >> 3), (uint32_t)t.split << shift);
          *last_in = last;
          __threadfence();
        }
        named_sync(3, 32 * kOutWarps);
        wrote = *last_in != 0;
      }
      for (int i = 0; wrote && i < chunks; ++i) {
        const int c = chunk(i);
        if (t.split > 1) {
#pragma unroll
          for (int q = 0; q < 32; ++q) v[q] = 0u;
#pragma unroll 1
          for (int s = 0; s < t.split; ++s)
#pragma unroll
            for (int q = 0; q < 32; ++q)
              if (c + q < t.cols)
                v[q] = __float_as_uint(__uint_as_float(v[q]) + __ldcg(part + s * 2 * size + (c + q) * 128));
        } else if (i > 0) {
          read(i, v);
        }
        emit(c, v);
      }
      if (gate && t.split == 1) {
        __syncwarp();
        if (lane == 0) tc::mbar_arrive_local(rec_done + 8 * slot);
      } else if (gate && wrote) {
        tc::fence_async_global();
        named_sync(3, 32 * kOutWarps);
        if (threadIdx.x == 128) {
          __threadfence();
          atomicAdd(&p.groups->ready[t.epoch][group_of(p, t.e)], 1u);
        }
      }
      ++it;
    }
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
  // Neither CTA leaves while the other may still use its shared or tensor memory
  // or its barriers: every arrival, copy and commit that comes from the other CTA
  // has been waited for above, by the warp that needed it or by its owner.
  __syncwarp();
  tc::fence_before();
  __syncthreads();
  cluster_arrive_relaxed();
  cluster_wait();
  tc::fence_after();
  if (warp == 2) tc::tmem_free_pair(tmem, kTmemCols);
}

// --- host --------------------------------------------------------------------

int64_t cdiv(int64_t a, int64_t b) { return (a + b - 1) / b; }

// Bytes [d3][d2][d1][d0] of 4-bit rows, dense: boxes of deep x rows x 128 bytes,
// 128-byte swizzle.
bool map_rows(CUtensorMap *m, const void *base, int64_t d0, int64_t d1, int64_t d2, int64_t d3, int rows,
              int deep = 1) {
  const EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {(cuuint64_t)d0, (cuuint64_t)d1, (cuuint64_t)d2, (cuuint64_t)d3};
  const cuuint64_t strides[3] = {(cuuint64_t)d0, (cuuint64_t)(d0 * d1), (cuuint64_t)(d0 * d1 * d2)};
  const cuuint32_t box[4] = {128, (cuuint32_t)rows, (cuuint32_t)deep, 1};
  const cuuint32_t step[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT8, 4, const_cast<void *>(base), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The scales' tiles [E][row tiles][block tiles][512 bytes]: boxes of `deep` x 2
// tiles, as they stand.
bool map_scales(CUtensorMap *m, const void *base, const ScaleLayout &l, int64_t E, int deep) {
  const EncodeFn fn = encode_fn();
  if (!fn) return false;
  const cuuint64_t dims[4] = {kScaleTileBytes / 4, (cuuint64_t)l.block_tiles, (cuuint64_t)l.row_tiles,
                              (cuuint64_t)E};
  const cuuint64_t s1 = kScaleTileBytes, s2 = s1 * l.block_tiles, s3 = s2 * l.row_tiles;
  const cuuint64_t strides[3] = {s1, s2, s3};
  const cuuint32_t box[4] = {kScaleTileBytes / 4, 2, (cuuint32_t)deep, 1};
  const cuuint32_t step[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_UINT32, 4, const_cast<void *>(base), dims, strides, box, step,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_NONE, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The tokens' operand: the boxes that tiles of at most cap tokens use.
bool map_tokens(MxJob &j, const void *rows, const void *scales, int64_t width, int64_t cap, int64_t E) {
  for (int i = 0; i < 4; ++i) {
    if (!map_rows(&j.b[i], rows, width / 2, cap, 1, E, 16 << i)) return false;
    if (cap <= (32 << i)) break;
  }
  const ScaleLayout l = scale_layout(cap, width);
  for (int i = 0; i < 3 && i < l.row_tiles; ++i)
    if (!map_scales(&j.b_scale[i], scales, l, E, i + 1)) return false;
  return true;
}

// Units of a product: its most tiles, each in up to kMaxSplit parts.
int64_t units(const MxJob &j, const FfnMxfp4Params &f) {
  return j.mt * f.E * cdiv(f.cap, kTileCols) * (cdiv(j.K, kBlockK) < 16 ? 1 : kMaxSplit);
}

}  // namespace

size_t ffn_mxfp4_scratch(int64_t E, int64_t cap, int64_t H, int64_t I) {
  const int64_t mt = cdiv(I, 128) > cdiv(H, 256) ? cdiv(I, 128) : cdiv(H, 256);
  const int64_t most = mt * E * cdiv(cap, kTileCols) * kMaxSplit;
  const int64_t cols = cap < kTileCols ? (cap + 31) / 32 * 32 : kTileCols;
  return (size_t)((most < kMaxPairs ? most : kMaxPairs) * cols) * 256 * sizeof(float);
}

cudaError_t launch_ffn_mxfp4(const FfnMxfp4Params &f, cudaStream_t stream) {
  MxParams p = {};
  p.counts = f.counts;
  p.hdr = f.hdr;
  p.part = f.part;
  p.tickets = f.hdr->reserved + kTicketWord;
  p.units = reinterpret_cast<UnitCounter *>(f.hdr->reserved + kUnitWord);
  p.groups = reinterpret_cast<GroupCounter *>(f.hdr->reserved + kGroupWord);
  p.E = f.E;
  p.cap = f.cap;
  MxJob &gu = p.job[0], &d = p.job[1];
  const ScaleLayout act = scale_layout(f.cap, f.I);
  if (!map_rows(&gu.a, f.w_gate_up, f.H / 2, f.I, 2, f.E, 64, 2) ||
      !map_scales(&gu.a_scale, f.w_gate_up_scale, scale_layout(2 * (int64_t)f.I, f.H), f.E, 1) ||
      !map_tokens(gu, f.x, f.x_scale, f.H, f.cap, f.E) ||
      !map_rows(&d.a, f.w_down, f.I / 2, f.H, 1, f.E, 128) ||
      !map_scales(&d.a_scale, f.w_down_scale, scale_layout(f.H, f.I), f.E, 1) ||
      !map_tokens(d, f.act, f.act_scale, f.I, f.cap, f.E))
    return cudaErrorInvalidValue;
  gu.q = f.act;
  gu.scale = f.act_scale;
  gu.row_tiles = act.row_tiles;
  gu.block_tiles = act.block_tiles;
  gu.M = f.I;
  gu.K = f.H;
  gu.mt = (int)cdiv(f.I, 128);
  d.out = f.y;
  d.M = f.H;
  d.K = f.I;
  d.mt = (int)cdiv(f.H, 256);

  static std::once_flag once[64];
  int dev = 0;
  cudaGetDevice(&dev);
  cudaError_t attr = cudaSuccess;
  std::call_once(once[dev & 63], [&] {
    attr = cudaFuncSetAttribute(ffn_mxfp4_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
  });
  if (attr != cudaSuccess) return attr;
  const int64_t tiles = units(gu, f) + units(d, f);
  int64_t most = device_sm_count() / 2;
  if (most > kMaxPairs) most = kMaxPairs;
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.gridDim = dim3((unsigned)(2 * (tiles < most ? tiles : most)));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = kSmem;
  cfg.stream = stream;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, ffn_mxfp4_kernel, p);
  return e != cudaSuccess ? e : cudaGetLastError();
}

}  // namespace moe
