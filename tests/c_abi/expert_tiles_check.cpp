// Row tiles of any offsets, against plain 64-bit counting (host build of
// combine_ep_dispatch_amd/csrc/expert_rows.h).
#include <cstdio>
#include <vector>

#include "../../combine_ep_dispatch_amd/csrc/expert_rows.h"

int main() {
  const int E = 1024, BM = 16;
  const int32_t rows = (1 << 27) - 1;  // the most that 128 channels allow
  for (int pattern = 0; pattern < 3; ++pattern) {
    std::vector<int32_t> offset(E + 1);
    for (int e = 0; e <= E; ++e)
      offset[e] = pattern == 0 ? (e % 2 ? rows : 0) : (pattern == 1 ? (e % 2 ? INT32_MAX : INT32_MIN) : e * 3 % 50);
    std::vector<ep::RowTiles> start(E + 1);
    std::vector<int32_t> count(E);
    unsigned long long total = 0;
    for (int e = 0; e < E; ++e) {
      int32_t first;
      ep::span_rows(offset[e], offset[e + 1], rows, first, count[e]);
      start[e] = static_cast<ep::RowTiles>(total);
      total += (count[e] + BM - 1) / BM;
    }
    start[E] = static_cast<ep::RowTiles>(total);
    if (static_cast<unsigned long long>(start[E]) != total || (pattern < 2 && total != 1ull << 32)) return std::printf("total\n"), 1;
    for (unsigned long long i = 0; i <= 4096; ++i) {
      const unsigned long long q = i * (total - 1) / 4096;
      const int e = ep::expert_of_tile(start.data(), E, static_cast<ep::RowTiles>(q));
      const unsigned long long local = q - static_cast<unsigned long long>(start[e]);
      // (its rows are there: what the kernel reads stays in the buffer)
      if (q < static_cast<unsigned long long>(start[e]) || q >= static_cast<unsigned long long>(start[e + 1]) ||
          local * BM >= static_cast<unsigned long long>(count[e]))
        return std::printf("tile %llu expert %d\n", q, e), 1;
    }
  }
  std::puts("ok");
}
