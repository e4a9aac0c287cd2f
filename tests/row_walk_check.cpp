// Host check of the walk over a group's rows: for each (r0, r1, threads) prints one
// line "r0 r1 threads visited in_range", the rows visited by all threads together
// (at most 8 of a thread are followed, so that a wrong walk ends) and 1 where each
// lay in [r0, r1).
#include <cstdio>
#include <cstdlib>

#include "../precision_rl_amd/csrc/row_walk.h"

namespace {
struct Stop {};
}  // namespace

int main(int argc, char** argv) {
  for (int a = 1; a + 2 < argc; a += 3) {
    const int64_t r0 = std::atoll(argv[a]), r1 = std::atoll(argv[a + 1]);
    const int threads = std::atoi(argv[a + 2]);
    int64_t visited = 0;
    bool inside = true;
    for (int t = 0; t < threads; ++t) {
      int followed = 0;
      try {
        w4a4::walk_rows(r0, r1, t, threads, [&](int64_t r) {
          if (++followed > 8) throw Stop{};
          ++visited;
          inside = inside && r >= r0 && r < r1;
        });
      } catch (const Stop&) {
        inside = false;
      }
    }
    std::printf("%lld %lld %d %lld %d\n", static_cast<long long>(r0), static_cast<long long>(r1), threads,
                static_cast<long long>(visited), inside);
  }
  return 0;
}
