// Prints span_rows (combine_ep_dispatch_amd/csrc/expert_rows.h) for the
// triples "begin end num_rows" given on the command line, one line "first
// count" each.
#include <cstdio>
#include <cstdlib>

#include "../../combine_ep_dispatch_amd/csrc/expert_rows.h"

int main(int argc, char** argv) {
  for (int i = 1; i + 2 < argc; i += 3) {
    int32_t first, count;
    ep::span_rows(static_cast<int32_t>(atoll(argv[i])), static_cast<int32_t>(atoll(argv[i + 1])),
                  static_cast<int32_t>(atoll(argv[i + 2])), first, count);
    printf("%d %d\n", first, count);
  }
  return 0;
}
