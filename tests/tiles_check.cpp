// tiles_check.cpp -- the tiles of an expert's tokens (csrc/moe_tiles.cuh) for
// many row counts, up to the largest: they follow one another from token 0 to the
// last, none is empty or wider than 256, and each starts on a multiple of STEP.
//
// Usage: tiles_check 32|64
// Prints "rows R tiles N bad B" and exits 0.
#include <stdint.h>
#include <stdio.h>
#include <stdlib.h>

#include "moe_tiles.cuh"

template <int STEP>
static int64_t check(int rows, int64_t &tiles) {
  const int n = moe::token_tiles(rows);
  int64_t bad = 0, next = 0;
  if (n < 1 || (int64_t)n * 256 < rows || (int64_t)(n - 1) * 256 >= rows) return 1;
  // all tiles of few, the first and last ones of many
  for (int i = 0; i < n; ++i) {
    if (n > 4096 && i == 1024) {
      i = n - 1024;
      next = moe::token_tile<STEP>(rows, n, i).first;
    }
    const moe::TokenTile t = moe::token_tile<STEP>(rows, n, i);
    bad += t.first != next || t.count < 1 || t.count > 256 || t.first % STEP != 0 ||
           (int64_t)t.first + t.count > rows;
    next = (int64_t)t.first + t.count;
    ++tiles;
  }
  return bad + (next != rows);
}

int main(int argc, char **argv) {
  const int step = argc > 1 ? atoi(argv[1]) : 0;
  int64_t rows = 0, tiles = 0, bad = 0;
  const auto one = [&](int64_t r) {
    if (r < 1 || r > INT32_MAX) return;
    ++rows;
    bad += step == 64 ? check<64>((int)r, tiles) : check<32>((int)r, tiles);
  };
  for (int64_t r = 1; r <= 5000; ++r) one(r);
  for (int b = 13; b <= 31; ++b)
    for (int64_t d = -300; d <= 300; ++d) one(((int64_t)1 << b) + d);
  for (int64_t r = 1; r < INT32_MAX; r += 104729LL * 257) one(r);
  printf("rows %lld tiles %lld bad %lld\n", (long long)rows, (long long)tiles, (long long)bad);
  return step == 32 || step == 64 ? 0 : 2;
}
