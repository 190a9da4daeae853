// Launch grids of any number of blocks.
#pragma once

#include <stdint.h>

namespace moe {

struct Grid {
  unsigned x, y;
};

// A grid dimension holds fewer than 2^32 threads; a launch of more runs their
// number modulo 2^32, without an error. Blocks past half of that go on in
// further lines of nearly equal length, a multiple of `unit`, and some (fewer
// than y * unit) may lie behind the last of `blocks`, but none with one line.
inline Grid fold_grid(int64_t blocks, int threads, int unit = 1) {
  const int64_t most = (INT64_C(1) << 31) / threads / unit * unit;
  const int64_t y = (blocks + most - 1) / most;
  const int64_t x = y > 1 ? ((blocks + y - 1) / y + unit - 1) / unit * unit : blocks;
  return {(unsigned)x, (unsigned)y};
}

}  // namespace moe
