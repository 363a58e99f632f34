// Tiles of a launch from any offsets, counted in 32 bits as the wavefronts count
// them (64 lanes, E / 64 experts each), against 64-bit counting (host build of
// combine_ep_dispatch_amd/csrc/expert_rows.h).
#include <cstdio>
#include <vector>

#include "../../combine_ep_dispatch_amd/csrc/expert_rows.h"

int main() {
  int none = 0, some = 0;
  for (const int E : {1, 2, 65, 256, 1024})
    for (const int BM : {64, 128, 192, 256})
      for (const uint32_t nt : {1u, 2u, 7u, 512u, 1024u})
        for (const long long rows : {1ll, 1000ll, 1ll << 18, (1ll << 22) - 1, 1ll << 22, (1ll << 26) + 5, 1ll << 29, (1ll << 31) - 1})
          for (int pattern = 0; pattern < 4; ++pattern) {
            std::vector<int32_t> offset(E + 1);
            for (int e = 0; e <= E; ++e) {
              const long long in_order = rows * e / E;
              offset[e] = pattern == 0   ? static_cast<int32_t>(in_order)
                          : pattern == 1 ? (e % 2 ? static_cast<int32_t>(rows) : 0)
                          : pattern == 2 ? (e % 2 ? INT32_MAX : INT32_MIN)
                                         : (e % 7 == 3 ? static_cast<int32_t>(rows) : static_cast<int32_t>(in_order / 2));
            }
            uint32_t total = 0, high = 0;
            unsigned long long all = 0;
            const int per = (E + 63) / 64;
            for (int lane = 0; lane < 64; ++lane) {
              uint32_t mine = 0;
              for (int e = lane * per; e < lane * per + per && e < E; ++e) {
                int32_t first, count;
                ep::span_rows(offset[e], offset[e + 1], static_cast<int32_t>(rows), first, count);
                mine += (static_cast<uint32_t>(count) + BM - 1) / BM;
                all += (static_cast<unsigned long long>(count) + BM - 1) / BM;
              }
              total += mine;
              high += mine >> 16;
            }
            const uint32_t got = ep::tiles_or_none(total, high, nt);
            const unsigned long long want = all * nt >= 1ull << 30 ? 0 : all * nt;
            if (got != want)
              return std::printf("E %d BM %d nt %u rows %lld pattern %d: %u, not %llu\n", E, BM, nt, rows, pattern, got, want), 1;
            (got == 0 && all ? none : some)++;
            // offsets in order, of rows as wide as the contract allows: rows * channels < 2^34, a tile of 32 channels or more
            if (pattern == 0 && rows * 32 * nt <= 1ll << 34 && (got == 0 || got >= 1u << 27)) return std::printf("in order\n"), 1;
          }
  std::puts(none && some ? "ok" : "one side only");
}
