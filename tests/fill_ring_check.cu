// Host-side check of the ring that feeds the layer norm's gradient
// (FillRing), compiled and run by tests/test_fill_ring_cpu.py without a GPU:
// for every number of rows and every row whose wait gives up, the parity that
// is waited for at the end is that of each stage's last fill, if that fill has
// not been waited for already.
#include <cstdio>
#include <cstdlib>

#include "tma.cuh"

using namespace rlca;

template <int STAGES>
void check() {
  for (int rows = 1; rows < 50; ++rows)
    for (int gives_up = 0; gives_up < rows; ++gives_up) {
      int fills[STAGES] = {}, waited[STAGES] = {};
      for (int i = 0; i < STAGES - 1 && i < rows; ++i) ++fills[i];
      FillRing<STAGES> ring;
      for (int row = 0; row < rows; ++row) {
        if (ring.ok && row + STAGES - 1 < rows) ++fills[ring.fill_stage()];
        if (ring.ok) {
          // a wait is for the fill that follows those already waited for
          if (ring.phase != (uint32_t)(waited[ring.stage] & 1)) std::printf("FAIL phase\n"), std::exit(1);
          if (row == gives_up) ring.ok = false;
          else ++waited[ring.stage];
        }
        ring.next();
      }
      for (int i = 0; i < STAGES; ++i)
        if (fills[i] > waited[i] && (fills[i] != waited[i] + 1 || ring.last_fill(i) != (uint32_t)((fills[i] - 1) & 1))) {
          std::printf("FAIL %d stages, %d rows, given up at %d: stage %d, %d fills\n", STAGES, rows, gives_up, i, fills[i]);
          std::exit(1);
        }
    }
}

int main() {
  check<3>();
  check<4>();
  std::printf("ring ok\n");
}
