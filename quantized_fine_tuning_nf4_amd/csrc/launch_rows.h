// How many rows one launch takes (host arithmetic alone).
#pragma once
#include <stdint.h>

namespace qn {

// Rows of `chunks` workgroups of `threads` threads each that fit a launch: its
// work items are counted in 32 bits, its workgroups in 31.  At least one.
inline int64_t rows_per_launch(int64_t chunks, int64_t threads) {
  const int64_t items = (((int64_t)1 << 32) - 1) / threads, groups = ((int64_t)1 << 31) - 1;
  const int64_t rows = (items < groups ? items : groups) / chunks;
  return rows > 0 ? rows : 1;
}

}  // namespace qn
