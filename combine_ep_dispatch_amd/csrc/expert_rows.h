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

// Stages of 64 elements of a sum of n (as many as 2^31 - 1 rows: n + 63 need not
// fit an int).
EP_ROWS_FN int32_t stages_of_sum(int32_t n) { return static_cast<int32_t>((static_cast<uint32_t>(n) + 63) / 64); }

// Tiles of a launch: its row tiles by nt tiles of channels, or none where they
// reach 2^30.  Rows that lie apart stay far below; offsets that run back may let
// experts share rows so often that 32 bits would not hold the sum, and then nothing
// is computed rather than a part.  row_tiles is a sum of at most 64 addends modulo
// 2^32, high the same sum of the addends' upper halves: below 2^14 of those the
// sum is below 2^30 + 2^22 and has not wrapped.
EP_ROWS_FN uint32_t tiles_or_none(uint32_t row_tiles, uint32_t high, uint32_t nt) {
  const uint64_t tiles = static_cast<uint64_t>(row_tiles) * nt;
  return high >= 1u << 14 || tiles >= 1u << 30 ? 0 : static_cast<uint32_t>(tiles);
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
