// Host-only check of the places that a fork's plan gives to fresh pages, built by
// tests/test_launch_plans_pages.py with nvcc (no GPU needed): the running sums of
// sv_pages.cuh, for what sequences may want within the interface's limits, against
// sums in 64 bits.
#include <algorithm>
#include <cstdio>

#include "sv_pages.cuh"

namespace {

int bad = 0;
long long places = 0;

// want(j): fresh pages of sequence j, at most W
template <typename F>
void check(int B2, int W, int nfree, F want) {
  int nfresh = 0;       // as the plan holds it
  long long exact = 0;
  for (int j0 = 0; j0 < B2; j0 += sv::kPgThreads) {
    long long sum = 0;  // of this turn: its own prefix sums have to fit too
    for (int j = j0; j < std::min(B2, j0 + sv::kPgThreads); ++j) {
      const int w = want(j);
      for (int i : {0, w - 1}) {
        if (i < 0) continue;
        const long long r = nfresh + sum + i, true_r = exact + sum + i;
        ++places;
        if (r > 0x7FFFFFFFll || (r < nfree) != (true_r < nfree) || (r < nfree && r != true_r)) {
          if (bad++ < 10)
            std::printf("sequence %d of %d, page %d of %d: place %lld, in 64 bits %lld of %d\n", j, B2, i, w, r,
                        true_r, nfree);
        }
      }
      sum += w;
    }
    exact += sum;
    nfresh = sv::pg_many(nfresh, (int)sum);
    if (sum > 0x7FFFFFFFll) ++bad;
  }
  if (std::min((long long)nfresh, (long long)nfree) != std::min(exact, (long long)nfree)) ++bad;
}

}  // namespace

int main() {
  for (int B2 : {1, 1023, 1024, 1025, 2049, 5000, SPEC_KV_MAX_TABLE})
    for (int W : {1, 3, 4096, SPEC_KV_MAX_TABLE})
      for (int nfree : {0, 1, 40, SPEC_KV_MAX_PAGES - 1, SPEC_KV_MAX_PAGES}) {
        check(B2, W, nfree, [&](int) { return W; });
        check(B2, W, nfree, [&](int j) { return j % 3 == 0 ? W : j % 3 == 1 ? 0 : 1; });
        check(B2, W, nfree, [&](int j) { return (int)((j * 2654435761ll) % (W + 1)); });
      }
  std::printf("%lld places checked\n", places);
  return bad != 0;
}
