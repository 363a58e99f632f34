// Stages of a sum of any length, against 64-bit counting (host build of
// combine_ep_dispatch_amd/csrc/expert_rows.h).
#include <cstdio>

#include "../../combine_ep_dispatch_amd/csrc/expert_rows.h"

int main() {
  const long long lengths[] = {0, 1, 63, 64, 65, 127, 128, 129, 65536, (1ll << 31) - 129, (1ll << 31) - 128, (1ll << 31) - 65,
                               (1ll << 31) - 64, (1ll << 31) - 63, (1ll << 31) - 2, (1ll << 31) - 1};
  for (const long long n : lengths)
    if (ep::stages_of_sum(static_cast<int32_t>(n)) != (n + 63) / 64)
      return std::printf("%lld: %d\n", n, static_cast<int>(ep::stages_of_sum(static_cast<int32_t>(n)))), 1;
  std::puts("ok");
}
