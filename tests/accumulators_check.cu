// Host-side check of how the matrix products' sums are divided into
// accumulators (tc_group_end), compiled and run by
// tests/test_accumulators_cpu.py without a GPU: every division covers all
// steps, no accumulator takes more than kTcLead of them -- an epilogue waits
// for one accumulator at a time, and its wait is limited --, and those of the
// leading term take no more than the group asked for.
#include <cstdio>
#include <cstdlib>

#include "tc.cuh"

using namespace rlca;

template <int GROUP>
void check() {
  const int lengths[] = {1, 2, 7, 8, 9, 63, 64, 65, 127, 128, 129, 1000, 4097, 262144};
  for (int terms : {1, 2, 6})
    for (int stages : lengths) {
      const int all = stages * terms, lead = all - stages;
      int at = 0;
      while (at < all) {
        const int end = tc_group_end<GROUP>(at, stages, terms);
        const bool ok = end > at && end <= all && end - at <= kTcLead && (at < lead ? end <= lead : end - at <= GROUP);
        if (!ok) {
          std::printf("FAIL group %d terms %d stages %d: steps %d to %d\n", GROUP, terms, stages, at, end);
          std::exit(1);
        }
        at = end;
      }
    }
}

int main() {
  check<2>();
  check<8>();
  check<16>();
  check<64>();
  std::printf("accumulators ok\n");
}
