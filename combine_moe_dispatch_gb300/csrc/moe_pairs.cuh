// moe_pairs.cuh -- what the kernels of the experts' products share: units of
// work and their order, the feed that brings them to a cluster's warps, bounded
// waits, and the tensor maps' encoder.
//
// A cluster of two CTAs (the two SMs of a pair) computes a tile of 256 rows x up
// to 256 columns at a time (tcgen05.mma.cta_group::2).  Tiles go to the pairs in
// order, as they get free.  Included by moe_ffn.cu (bf16) and moe_ffn_mxfp4.cu.
#pragma once

#include <cuda.h>
#include <cuda_bf16.h>
#include <limits.h>
#include <stddef.h>

#include "moe_tc.cuh"
#include "moe_tiles.cuh"

namespace moe {

namespace {

// What one launch computes.  kForward: a (and h), then y, whose tiles wait until
// every tile of a is written, or every one of their group of experts.  kRest: dx, dWgu and dWd, which need nothing of one
// another, as one list of tiles.
enum Kind { kForward = 0, kActGrad = 1, kRest = 2 };

constexpr int kEpiWarps = 8;           // two groups of four; each takes every other chunk of columns
// The feed's places for tiles, and how many are announced ahead in the bf16
// kernels (the 4-bit one has a figure of its own): kRing, and 2 where they are of kLongTile blocks or
// more, since a unit taken early is a unit that cannot go to a pair that is
// free sooner.  Measured: one token 116 us, with 4 ahead for all 122; uneven
// experts' backward (2 to 32 blocks a tile) 213 us, with 2 ahead for all 217.
constexpr int kRing = 4;
constexpr int kLongTile = 64;
constexpr int kTileCols = 256;
constexpr uint32_t kTmemCols = 512;                      // two accumulators of 256 columns
// The tiles past the last whole round of all pairs are cut into at most
// kMaxSplit parts of their contraction: never more parts than pairs, so their
// sums take at most kMaxPairs tiles of 256 x 256.
constexpr int kMaxSplit = 8;
constexpr int kMaxPairs = 128;

// The launch's next unit of work (backward: past the first of every pair): the
// last pair to finish resets it.  It and the tickets are zero between launches
// and stand with the other counters in the workspace header's reserved words,
// the one place that no shape's plan uses for anything else.
struct UnitCounter {
  unsigned long long next;
  uint32_t done;           // pairs that have taken all they will
  uint32_t epoch;          // kForward: which of `ready` counts this launch's
  uint32_t ready[2];       // CTAs' halves of tiles of a that are written; the other one is 0
                           // (the 4-bit kernel counts them by groups of experts, in words of its own)
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

// Where P::kExpertGroups is above 1, the experts form so many groups, in order, and
// a tile of y waits for the tiles of a of its expert's group alone.
template <class P>
__device__ __forceinline__ int group_of(const P &p, int e) { return e * P::kExpertGroups / p.E; }
template <class P>
__device__ __forceinline__ int group_start(const P &p, int g) {
  return (g * p.E + P::kExpertGroups - 1) / P::kExpertGroups;
}

template <class P>
__device__ __forceinline__ int rows_of(const P &p, int e) {
  if (!p.counts) return p.cap;
  const int c = __ldg(p.counts + e);
  return c < 0 ? 0 : (c > p.cap ? p.cap : c);
}

struct alignas(16) Tile {
  int valid;               // 0: no more work
  int job, e, rows;        // product, expert, its tokens
  int m;                   // tile of 256 accumulator rows
  int n0, n;               // first column, columns of the matrix instruction
  int cols;                // row products: tokens in the tile
  int k0, nk;              // blocks (P::kBlock) of the contraction: [k0, k0 + nk); nk = 0: the result is 0
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
template <class P>
struct Schedule {
  static constexpr int KIND = P::kKind;
  static constexpr int kBlockK = P::kBlock;  // elements of a block of the contraction
  const P &p;
  int64_t base;            // tiles before this batch of 32 experts
  int incl, e0, rows;      // tiles of the batch up to this lane's expert; its tokens
  int64_t whole;           // tiles that are not cut
  int split, part_cols;    // parts of the others, columns of a part's sums
  int row;                 // the row product that is being dealt out,
  int64_t first;           // its first unit,
  int need;                // and what its tiles wait for (one group: all of a)
  int group, group_need;   // several: the group counted last
  __device__ __forceinline__ explicit Schedule(const P &p_) : p(p_), row(0), first(0), need(0), group(-1), group_need(0) {
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
  // contraction is of 16 blocks or more (1024 elements of bf16, 4096 of 4 bits).  The
  // estimate is in blocks: a unit costs its blocks and about kUnitCost more (filling
  // the ring, the epilogue), a tile that is cut kJoinCost and a block per part and 64
  // columns for the sums.  The costs and the 16 are those of bf16's blocks; with 4
  // bits' they were not measured apart.  In bf16, with and without: one token (two experts, H 4096, I 14336)
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
      o.m = r / nt;
      const int i = r - o.m * nt;
      const TokenTile tokens = token_tile<P::kTileStep>(o.rows, nt, i);
      o.n0 = tokens.first;
      o.cols = tokens.count;
    }
    o.n = (o.cols + 31) & ~31;
    const int nk = (p.job[KIND == kForward ? row : 0].K + kBlockK - 1) / kBlockK;
    o.need = need;
    if constexpr (P::kExpertGroups > 1)
      if (row == 1) o.need = count_group(group_of(p, o.e));
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
  // Halves of tiles of a of a group's experts.
  __device__ __forceinline__ int count_group(int g) {
    if (g != group) {
      group = g;
      const int end = group_start(p, group + 1);
      int tiles = 0;
      for (int x = group_start(p, group) + (threadIdx.x & 31); x < end; x += 32) tiles += token_tiles(rows_of(p, x));
#pragma unroll
      for (int d = 16; d > 0; d >>= 1) tiles += __shfl_xor_sync(0xFFFFFFFFu, tiles, d);
      group_need = (int)(2u * (unsigned)tiles * (unsigned)p.job[0].mt);
    }
    return group_need;
  }
  __device__ __forceinline__ bool find_weight(int64_t t, Tile &o) {
    o.job = 1;
    int nt = (p.job[1].N + kTileCols - 1) / kTileCols;
    int64_t per = (int64_t)p.job[1].mt * nt;
    if (t >= per * p.E) {
      t -= per * p.E;
      o.job = 2;
      nt = (p.job[P::kJobs - 1].N + kTileCols - 1) / kTileCols;
      per = (int64_t)p.job[P::kJobs - 1].mt * nt;
      if (t >= per * p.E) return false;
    }
    const auto &j = p.job[P::kJobs == 1 ? 0 : o.job];
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

// Arrive at barrier `id` of `n` threads without waiting.
__device__ __forceinline__ void named_arrive(uint32_t id, uint32_t n) {
  asm volatile("bar.arrive %0, %1;" ::"r"(id), "r"(n) : "memory");
}

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

  // Every lane is done with the record: its place is free, on to the next.
  __device__ __forceinline__ void leave() {
    tc::mbar_arrive_warp_at(empty + 8 * s);
    if (++s == kRing) {
      s = 0;
      ph ^= 1u;
    }
  }

 private:
  // Every lane has read the record.  The last one's place is not used again, and
  // nobody waits for it.
  __device__ __forceinline__ bool done(const Tile &t) {
    if (t.valid == 0) return false;
    leave();
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

}  // namespace

}  // namespace moe
