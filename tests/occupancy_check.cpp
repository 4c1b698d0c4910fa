// occupancy_check.cpp -- the table of kernels' resident blocks (csrc/moe_occupancy.cuh):
// how often it asks, and whether each answer is the one asked for.
//
// Usage: occupancy_check KERNELS DEVICES
// Prints "first A again B wrong W" and exits 0: questions in the first round over all
// kernels and devices, in three further rounds, and answers that were another's.
#include <stdio.h>
#include <stdlib.h>

#include "moe_occupancy.cuh"

int main(int argc, char **argv) {
  const int kernels = argc > 1 ? atoi(argv[1]) : 0, devices = argc > 2 ? atoi(argv[2]) : 0;
  static moe::OccupancyTable table;
  long asked = 0, first = 0, wrong = 0;
  for (int round = 0; round < 4; ++round) {
    for (int d = 0; d < devices; ++d)
      for (int k = 0; k < kernels; ++k)
        for (int form = 0; form < 2; ++form) {           // two block sizes of the same kernel
          const int want = 1 + (k * 7 + d * 3 + form) % 32;
          const auto ask = [&] {
            ++asked;
            return want;
          };
          // functions of a program: some hundred bytes apart
          const void *kern = (const void *)(0x400000ull + 0x180ull * k);
          wrong += table.get(kern, d, form ? 512 : 256, 1024u * form, ask) != want;
        }
    if (round == 0) first = asked;
  }
  printf("first %ld again %ld wrong %ld\n", first, asked - first, wrong);
  return 0;
}
