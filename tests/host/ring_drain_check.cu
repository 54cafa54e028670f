// Host-side check of drain_ring (window_tc.cuh): a ring of `stages` loads into
// which `issued` items went, with the loader's and its consumer's phases kept
// here; after the drain no item may be in flight.
#include <cstdio>
#include <vector>

#include "window_tc.cuh"

int main() {
  int fails = 0, cases = 0;
  for (int stages = 1; stages <= 8; ++stages)
    for (int issued = 0; issued <= 5 * stages + 1; ++issued, ++cases) {
      std::vector<bool> flying(issued, false);
      for (int n = 0; n < issued; ++n) {
        if (n >= stages) flying[n - stages] = false;  // its stage was released, so it had landed
        flying[n] = true;
      }
      int asked = 0;
      longnet::wt::drain_ring(issued, stages, [&](int stage, uint32_t parity) {
        ++asked;
        for (int n = 0; n < issued; ++n)
          if (flying[n] && n % stages == stage && (uint32_t)(n / stages % 2) == parity) flying[n] = false;
        return true;
      });
      for (int n = 0; n < issued; ++n)
        if (flying[n]) ++fails, printf("FAIL stages=%d issued=%d item %d in flight\n", stages, issued, n);
      if (asked != (issued < stages ? issued : stages)) ++fails, printf("FAIL stages=%d issued=%d asked %d\n", stages, issued, asked);
      asked = 0;  // a wait that runs out ends it
      longnet::wt::drain_ring(issued, stages, [&](int, uint32_t) { return ++asked < 2; });
      if (asked > 2) ++fails, printf("FAIL stages=%d issued=%d went on\n", stages, issued);
    }
  printf("cases=%d fails=%d\n", cases, fails);
  return fails != 0;
}
