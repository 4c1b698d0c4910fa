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
#include <cuda.h>
#include <cuda_bf16.h>
#include <limits.h>
#include <stddef.h>

#include <mutex>

#include "moe_ffn.cuh"
#include "moe_tc.cuh"

namespace moe {

namespace {

// What one launch computes.  kForward: a (and h), then y, whose tiles wait until
// every tile of a is written.  kRest: dx, dWgu and dWd, which need nothing of one
// another, as one list of tiles.
enum Kind { kForward = 0, kActGrad = 1, kRest = 2 };

constexpr int kPairThreads = 384;      // warps: 0 TMA, 1 MMA, 2 maps, 3 scheduling, 4-11 epilogue
constexpr int kEpiWarps = 8;           // two groups of four; each takes every other chunk of columns
constexpr int kStages = 6;
constexpr int kBlockK = 64;            // one 128-byte swizzled line of bf16
constexpr uint32_t kHalfBytes = 128 * kBlockK * 2;       // a CTA's half of one operand: 16 KB
constexpr uint32_t kStageBytes = 2 * kHalfBytes;
constexpr uint32_t kStagingBytes = 2 * 16384;            // epilogue, one buffer per group
constexpr uint32_t kBarOff = kStages * kStageBytes + kStagingBytes;
// Tiles announced ahead: kRing, and 2 where they are of kLongTile blocks or
// more, since a unit taken early is a unit that cannot go to a pair that is
// free sooner.  Measured: one token 116 us, with 4 ahead for all 122; uneven
// experts' backward (2 to 32 blocks a tile) 213 us, with 2 ahead for all 217.
constexpr int kRing = 4;
constexpr int kLongTile = 64;
constexpr uint32_t kRingOff = kBarOff + 256;
constexpr uint32_t kMapOff = kRingOff + kRing * 64;      // kActGrad: a tensor map being written
constexpr uint32_t kPairSmem = kMapOff + 128 + 1024;     // + alignment slack
static_assert(kPairSmem <= 232448, "shared memory of one CTA");
constexpr int kTileCols = 256;
constexpr uint32_t kTmemCols = 512;                      // two accumulators of 256 columns
// The tiles past the last whole round of all pairs are cut into at most
// kMaxSplit parts of their contraction: never more parts than pairs, so their
// sums take at most kMaxPairs tiles of 256 x 256.
constexpr int kMaxSplit = 8;
constexpr int kMaxPairs = 128;

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

// The launch's next unit of work (backward: past the first of every pair): the
// last pair to finish resets it.  It and the tickets are zero between launches
// and stand with the other counters in the workspace header's reserved words,
// the one place that no shape's plan uses for anything else.
struct UnitCounter {
  unsigned long long next;
  uint32_t done;           // pairs that have taken all they will
  uint32_t epoch;          // kForward: which of `ready` counts this launch's
  uint32_t ready[2];       // CTAs' halves of tiles of a that are written; the other one is 0
};
constexpr int kUnitWord = 1, kTicketWord = 8;            // in WsHeader::reserved
// A wait that runs out leaves the counters and tickets unfinished, and the
// next plan replaces the status: a split tile would then be joined one part too
// early.  kFfnBroken stays until moe_workspace_init clears the header.  It stands
// beside the status, so that one load brings both: read from a word of the
// counters' own sector it cost 0.25 us per launch.
static_assert(offsetof(WsHeader, status) % 8 == 0 &&
              offsetof(WsHeader, debug_flags) == offsetof(WsHeader, status) + 4, "read together");
struct StatusWords {
  int32_t status;
  uint32_t flags;
};
__device__ __forceinline__ StatusWords read_status_words(const WsHeader *hdr) {
  StatusWords w;
  asm volatile("ld.volatile.global.v2.u32 {%0, %1}, [%2];"
               : "=r"(w.status), "=r"(w.flags) : "l"(&hdr->status) : "memory");
  return w;
}
static_assert(kUnitWord * 4 + sizeof(UnitCounter) <= kTicketWord * 4, "the counters fit");
static_assert(offsetof(WsHeader, reserved) % 8 == 4, "the unit counter is 8-byte aligned");
static_assert(kMaxSplit < 16 && kTicketWord + kMaxPairs * 2 * 4 / 32 <= 55, "the tickets fit");

template <int KIND>
struct PairParams {
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

template <class P>
__device__ __forceinline__ int rows_of(const P &p, int e) {
  if (!p.counts) return p.cap;
  const int c = __ldg(p.counts + e);
  return c < 0 ? 0 : (c > p.cap ? p.cap : c);
}

// Tiles of `rows` tokens, and the columns of each but the last: as few tiles as
// 256 columns allow, equal, a multiple of 32 (the granularity of a matrix
// instruction's columns).  With n tiles rows > 256 (n - 1) and the columns are
// at most 256, so that the last tile is never empty.
__device__ __forceinline__ int token_tiles(int rows) { return (int)(((unsigned)rows + 255u) >> 8); }
__device__ __forceinline__ int tile_cols(int rows, int tiles) {
  return (int)((((unsigned)rows + tiles - 1) / tiles + 31) & ~31u);
}

struct alignas(16) Tile {
  int valid;               // 0: no more work
  int job, e, rows;        // product, expert, its tokens
  int m;                   // tile of 256 accumulator rows
  int n0, n;               // first column, columns of the matrix instruction
  int cols;                // row products: tokens in the tile
  int k0, nk;              // blocks of 64 of the contraction: [k0, k0 + nk); nk = 0: the result is 0
  int split, part;         // parts of the tile's contraction, and which this is
  int slot;                // split > 1: tile among those that are cut
  int part_cols;           // and columns that each part's sums have room for
  int need;                // halves of tiles of a that have to be written before the tokens are read
  int epoch;               // where they are counted
};
static_assert(sizeof(Tile) == 64, "a tile's record is 64 bytes");

// The launch's units of work in order: tiles of the row product by expert
// (each `split` times, once per part of the contraction), then the weight
// gradients' tiles.  Called by one whole warp with increasing unit.  32 experts'
// tiles are counted at a time, one expert per lane.
template <int KIND>
struct Schedule {
  const PairParams<KIND> &p;
  int64_t base;            // tiles before this batch of 32 experts
  int incl, e0, rows;      // tiles of the batch up to this lane's expert; its tokens
  int64_t whole;           // tiles that are not cut
  int split, part_cols;    // parts of the others, columns of a part's sums
  int row;                 // the row product that is being dealt out,
  int64_t first;           // its first unit,
  int need;                // and what its tiles wait for
  __device__ __forceinline__ explicit Schedule(const PairParams<KIND> &p_) : p(p_), row(0), first(0), need(0) {
    start();
  }
  __device__ __forceinline__ void start() {
    base = 0;
    e0 = 0;
    whole = INT64_MAX;
    split = 1;
    part_cols = 0;
    count();
    if (KIND != kRest && p.job[KIND == kForward ? row : 0].K >= 16 * kBlockK) choose_split();
  }
  // At most 2^46 elements of h: the batch's tiles fit an int.
  __device__ __forceinline__ void count() {
    const int lane = threadIdx.x & 31, e = e0 + lane;
    rows = e < p.E ? rows_of(p, e) : 0;
    incl = token_tiles(rows) * p.job[KIND == kForward ? row : 0].mt;
#pragma unroll
    for (int d = 1; d < 32; d <<= 1) {
      const int o = __shfl_up_sync(0xFFFFFFFFu, incl, d);
      if (lane >= d) incl += o;
    }
  }
  // The tiles that would leave pairs idle in the last round are cut, if their
  // contraction is of 1024 or more.  The estimate is in blocks of 64: a unit
  // costs its blocks and about kUnitCost more (filling the ring, the epilogue),
  // a tile that is cut kJoinCost and a block per part and 64 columns for the
  // sums.  Measured with and without: one token (two experts, H 4096, I 14336)
  // 117 and 124 us; 128 rows of one expert, H 7168, I 2048: 36 and 41; 1109
  // rows, H 4416, I 2168: 71 and 74; uneven experts' backward 206 and 205;
  // ten rows over 95 experts 28 and 26 (counting the tiles takes 1 us).
  __device__ __forceinline__ void choose_split() {
    constexpr int kUnitCost = 6, kJoinCost = 14;
    const int lane = threadIdx.x & 31;
    int64_t tiles = lane == 31 ? incl : 0;   // the first batch's sum
    int most = rows;
    for (int e = 32 + lane; e < p.E; e += 32) {
      const int r = rows_of(p, e);
      tiles += token_tiles(r) * p.job[KIND == kForward ? row : 0].mt;
      most = max(most, r);
    }
#pragma unroll
    for (int d = 16; d > 0; d >>= 1) tiles += __shfl_xor_sync(0xFFFFFFFFu, tiles, d);
    most = __reduce_max_sync(0xFFFFFFFFu, most);
    const int pairs = gridDim.x >> 1, nk = (p.job[KIND == kForward ? row : 0].K + kBlockK - 1) / kBlockK;
    const int left = (int)(tiles % pairs);
    part_cols = most >= kTileCols ? kTileCols : (most + 31) & ~31;
    // lane s - 1 prices s parts
    const int s = lane + 1;
    const bool can = s == 1 || (s <= kMaxSplit && s * left <= kMaxPairs && 4 * s <= nk);
    const int cost = can ? (s * left > pairs ? 2 : 1) * ((nk + s - 1) / s + kUnitCost) +
                               (s > 1 ? kJoinCost + s * ((part_cols + 63) >> 6) : 0)
                         : INT_MAX >> 6;
    split = left == 0 ? 1 : (__reduce_min_sync(0xFFFFFFFFu, cost * 32 + lane) & 31) + 1;
    whole = tiles - left;
  }
  __device__ __forceinline__ bool find(int64_t unit, Tile &o) {
    bool cut;
    int in;
    int64_t t;
    while (true) {
      cut = unit - first >= whole && split > 1;
      in = cut ? (int)(unit - first - whole) : 0;
      t = cut ? whole + in / split : unit - first;
      const int64_t end = base + __shfl_sync(0xFFFFFFFFu, incl, 31);
      if (t < end) break;
      base = end;
      if (e0 + 32 < p.E) {
        e0 += 32;
        count();
        continue;
      }
      incl = 0;                              // base now counts every row tile, for good
      if constexpr (KIND == kRest) return find_weight(t - base, o);
      if (KIND != kForward || row == 1) return false;
      need = (int)(uint32_t)(2 * base);      // fewer than 2^31 tiles
      first += split > 1 ? whole + (base - whole) * split : base;
      row = 1;
      start();
    }
    const int tb = (int)(t - base);
    const int l = __ffs(__ballot_sync(0xFFFFFFFFu, incl > tb)) - 1;
    const int before = __shfl_sync(0xFFFFFFFFu, incl, l > 0 ? l - 1 : 0);
    const int r = tb - (l > 0 ? before : 0);
    o.job = KIND == kForward ? row : 0;
    o.e = e0 + l;
    o.rows = __shfl_sync(0xFFFFFFFFu, rows, l);
    const int nt = token_tiles(o.rows);
    o.m = r;
    o.n0 = 0;
    o.cols = o.rows;
    if (nt > 1) {
      const int c = tile_cols(o.rows, nt);
      o.m = r / nt;
      o.n0 = (r - o.m * nt) * c;
      o.cols = min(c, o.rows - o.n0);
    }
    o.n = (o.cols + 31) & ~31;
    const int nk = (p.job[KIND == kForward ? row : 0].K + kBlockK - 1) / kBlockK;
    o.need = need;
    o.k0 = 0;
    o.nk = nk;
    o.split = cut ? split : 1;
    o.part = 0;
    o.slot = 0;
    o.part_cols = part_cols;
    if (cut) {
      o.slot = in / split;
      o.part = in - o.slot * split;
      o.k0 = nk * o.part / split;
      o.nk = nk * (o.part + 1) / split - o.k0;
    }
    return true;
  }
  __device__ __forceinline__ bool find_weight(int64_t t, Tile &o) {
    o.job = 1;
    int nt = (p.job[1].N + kTileCols - 1) / kTileCols;
    int64_t per = (int64_t)p.job[1].mt * nt;
    if (t >= per * p.E) {
      t -= per * p.E;
      o.job = 2;
      nt = (p.job[PairParams<KIND>::kJobs - 1].N + kTileCols - 1) / kTileCols;
      per = (int64_t)p.job[PairParams<KIND>::kJobs - 1].mt * nt;
      if (t >= per * p.E) return false;
    }
    const Job &j = p.job[PairParams<KIND>::kJobs == 1 ? 0 : o.job];
    o.e = (int)(t / per);
    const int r = (int)(t - o.e * per);
    o.rows = rows_of(p, o.e);
    o.m = r / nt;
    o.n0 = (r - o.m * nt) * kTileCols;
    o.n = min(kTileCols, (j.N - o.n0 + 31) & ~31);
    o.cols = o.n;
    o.k0 = 0;
    o.nk = (int)(((unsigned)o.rows + kBlockK - 1) / kBlockK);
    o.split = 1;
    o.part = o.slot = o.part_cols = o.need = 0;
    return true;
  }
};

// Wait for phase `parity` of the barrier, for `limit` ns at most and a
// bounded number of polls.
__device__ __forceinline__ bool wait_bar(uint32_t bar, uint32_t parity, uint64_t limit) {
  uint64_t t0 = 0;
  for (uint32_t it = 0; it < (1u << 26); ++it) {
    if (tc::mbar_try(bar, parity)) return true;
    if ((it & 63u) == 63u) {
      const uint64_t now = global_timer_ns();
      if (t0 == 0) t0 = now;
      else if (now - t0 > limit) return false;
    }
  }
  return false;
}

// Wait until the counter has reached `want` and what was stored before it was
// raised can be read by asynchronous copies; bounded as wait_bar.
__device__ __forceinline__ bool wait_count(const uint32_t *counter, uint32_t want, uint64_t limit) {
  uint64_t t0 = 0;
  for (uint32_t it = 0; it < (1u << 26); ++it) {
    if (ld_acquire_gpu(counter) >= want) {
      tc::fence_async_global();
      return true;
    }
    if ((it & 15u) == 15u) {
      const uint64_t now = global_timer_ns();
      if (t0 == 0) t0 = now;
      else if (now - t0 > limit) return false;
    }
  }
  return false;
}

// A warp's view of the tiles that the leader's scheduling warp announces.
struct Feed {
  const Tile *ring;
  uint32_t full, empty;    // this CTA's barriers, the leader's
  uint64_t limit;
  int s;
  uint32_t ph;
  __device__ __forceinline__ Feed(const Tile *ring_, uint32_t full_, uint32_t empty_, uint64_t limit_)
      : ring(ring_), full(full_), empty(empty_), limit(limit_), s(0), ph(0) {}
  // The next tile; false when there is none, or (ok false) when the wait ran
  // out.  Called by the whole warp.
  __device__ __forceinline__ bool next(Tile &t, bool &ok) {
    ok = __all_sync(0xFFFFFFFFu, wait_bar(full + 8 * s, ph, limit));
    if (!ok) return false;
    t = ring[s];
    __syncwarp();
    return done(t);
  }
  // The same for the words of WORDS (a bit each) alone, through shuffles, so
  // that the compiler knows the values to be the same in every lane.  In two
  // steps, for a warp that should not wait for the record: lane i < 16 reads
  // word i, spread() gives every lane all of them later.
  struct Raw {
    int word;
  };
  __device__ __forceinline__ Raw read() {
    Raw r;
    r.word = reinterpret_cast<const int *>(ring + s)[threadIdx.x & 15];
    return r;
  }
  template <uint32_t WORDS>
  __device__ __forceinline__ bool spread(const Raw &r, Tile &t) {
    int *w = reinterpret_cast<int *>(&t);
#pragma unroll
    for (int i = 0; i < 16; ++i)
      if ((WORDS >> i) & 1u) w[i] = __shfl_sync(0xFFFFFFFFu, r.word, i);
    return done(t);
  }
  template <uint32_t WORDS>
  __device__ __forceinline__ bool next_uniform(Tile &t, bool &ok) {
    ok = __all_sync(0xFFFFFFFFu, wait_bar(full + 8 * s, ph, limit));
    if (!ok) return false;
    return spread<WORDS>(read(), t);
  }

 private:
  // Every lane has read the record.  The last one's place is not used again, and
  // nobody waits for it.
  __device__ __forceinline__ bool done(const Tile &t) {
    if (t.valid == 0) return false;
    tc::mbar_arrive_warp_at(empty + 8 * s);
    if (++s == kRing) {
      s = 0;
      ph ^= 1u;
    }
    return true;
  }
};
// Words of a record: what the copies and what the matrix instructions need.
constexpr uint32_t kValid = 1u << 0, kJob = 1u << 1, kExpert = 1u << 2, kRows = 1u << 3, kM = 1u << 4,
                   kN0 = 1u << 5, kN = 1u << 6, kK0 = 1u << 8, kNk = 1u << 9, kNeed = 1u << 14, kEpoch = 1u << 15;
constexpr uint32_t kCopyWords = kValid | kJob | kExpert | kRows | kM | kN0 | kN | kK0 | kNk |
                                kNeed | kEpoch;
constexpr uint32_t kMathWords = kValid | kJob | kRows | kN | kNk;

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
  const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
  return *reinterpret_cast<const uint32_t *>(&v);
}
__device__ __forceinline__ uint2 pack4(const float (&v)[4]) {
  return make_uint2(pack2(v[0], v[1]), pack2(v[2], v[3]));
}
__device__ __forceinline__ void unpack4(const uint2 &w, float (&v)[4]) {
  v[0] = bf16_lo(w.x);
  v[1] = bf16_hi(w.x);
  v[2] = bf16_lo(w.y);
  v[3] = bf16_hi(w.y);
}
// 1 / (1 + e^-g) as 2^-20 / (2^-20 + 2^(-g log2 e - 20)): the divisor then stays
// below 2^126 down to g = -101, where the sigmoid itself is 2^-146.  (From 2^126
// on a quick quotient is 0, at g = -87.4 without the factor; SiLU(-88) is a normal
// number.)  Relative error: half a unit in the last place of the exponent
// and of log2 e, and 2^-22 of each approximate instruction, together below
// 2^-18 for |g| < 20 and 2^-16 at 100; below 2^-126 the result has a subnormal's
// bits.  Five instructions.
__device__ __forceinline__ float sigmoid(float g) {
  constexpr float kLog2E = 1.4426950408889634f, kShift = 0x1p-20f;
  float t, r;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(t) : "f"(fmaf(g, -kLog2E, -20.0f)));
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(t + kShift));
  return r * kShift;
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
    Schedule<KIND> sched(p);
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

using EncodeFn = CUresult (*)(CUtensorMap *, CUtensorMapDataType, cuuint32_t, void *,
                              const cuuint64_t *, const cuuint64_t *, const cuuint32_t *,
                              const cuuint32_t *, CUtensorMapInterleave, CUtensorMapSwizzle,
                              CUtensorMapL2promotion, CUtensorMapFloatOOBfill);

EncodeFn encode_fn() {
  static EncodeFn fn = [] {
    void *q = nullptr;
    cudaDriverEntryPointQueryResult r;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &q, 12000, cudaEnableDefault, &r) !=
            cudaSuccess || r != cudaDriverEntryPointSuccess)
      q = nullptr;
    return reinterpret_cast<EncodeFn>(q);
  }();
  return fn;
}

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
