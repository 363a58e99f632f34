// The rows of an expert, clamped to the buffer (internal; plain code that the
// host compiles as well).
#pragma once

#include <stdint.h>

#if defined(__HIPCC__)
#define EP_ROWS_FN __host__ __device__ __forceinline__
#else
#define EP_ROWS_FN inline
#endif

namespace ep {

// Rows first .. first + count - 1 of a buffer of num_rows, from any two
// offsets: 0 <= first, 0 <= count, first + count <= num_rows.  (The end is
// clamped to first before the difference is taken: the difference of two wild
// offsets need not fit an int.)
EP_ROWS_FN void span_rows(int32_t begin, int32_t end, int32_t num_rows, int32_t& first, int32_t& count) {
  first = begin < 0 ? 0 : (begin < num_rows ? begin : num_rows);
  const int32_t last = end < first ? first : (end < num_rows ? end : num_rows);
  count = last - first;
}

// A number of row tiles.  Wild offsets may span the whole buffer for every
// other expert: 512 times 2^27 rows in tiles of 16 are 2^32.
typedef int64_t RowTiles;

// The expert whose row tiles start[e] .. start[e + 1] - 1 hold tile q <
// start[E] (start: of E + 1, not falling, from 0 on).
EP_ROWS_FN int expert_of_tile(const RowTiles* start, int E, RowTiles q) {
  int lo = 0, hi = E;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start[mid] <= q) lo = mid; else hi = mid;
  }
  return lo;
}

}  // namespace ep
