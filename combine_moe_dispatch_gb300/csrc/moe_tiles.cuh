// moe_tiles.cuh -- how an expert's tokens are dealt out to the columns of the
// matrix products' tiles.  Plain integer arithmetic, which a host compiler takes too.
#pragma once

#ifdef __CUDACC__
#define MOE_HOST_DEVICE __host__ __device__ __forceinline__
#else
#define MOE_HOST_DEVICE inline
#endif

namespace moe {

// Tiles of `rows` tokens, and the columns of each but the last: as few tiles as
// 256 columns allow, equal, a multiple of 32 (the granularity of a matrix
// instruction's columns).  With n tiles rows > 256 (n - 1) and the columns are
// at most 256, so that the last tile is never empty.  Where tiles start on
// multiples of STEP > 32, the steps are dealt out evenly: some tiles have one
// more than the others.  Rows go up to 2^31 - 1: rounded up, they are unsigned.
MOE_HOST_DEVICE int token_tiles(int rows) { return (int)(((unsigned)rows + 255u) >> 8); }
MOE_HOST_DEVICE int tile_cols(int rows, int tiles) {
  return (int)((((unsigned)rows + (unsigned)tiles - 1u) / (unsigned)tiles + 31u) & ~31u);
}

// Tile i of `tiles`: its first token, and how many it has.
struct TokenTile {
  int first, count;
};
template <int STEP>
MOE_HOST_DEVICE TokenTile token_tile(int rows, int tiles, int i) {
  TokenTile t;
  int most;
  if (STEP == 32) {
    most = tile_cols(rows, tiles);
    t.first = i * most;
  } else {
    const int steps = (int)(((unsigned)rows + (unsigned)STEP - 1u) / (unsigned)STEP);
    const int each = steps / tiles, more = steps - each * tiles;
    t.first = STEP * (i * each + (i < more ? i : more));
    most = STEP * (each + (i < more ? 1 : 0));
  }
  t.count = rows - t.first < most ? rows - t.first : most;
  return t;
}

}  // namespace moe
