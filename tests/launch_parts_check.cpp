// Host check of the grid splitting: prints one line per case,
// "threads workgroups launches covered most_threads", `covered` being 1 where the parts
// follow each other from 0 to the end.
#include <cstdio>
#include <cstdlib>

#include "../precision_rl_amd/csrc/launch_parts.h"

int main(int argc, char** argv) {
  for (int a = 1; a + 1 < argc; a += 2) {
    const int threads = std::atoi(argv[a]);
    const int64_t total = std::atoll(argv[a + 1]);
    int64_t at = 0, launches = 0, most = 0;
    bool covered = true;
    w4a4::launch_parts(total, threads, [&](int64_t first, int64_t count) {
      covered = covered && first == at && count > 0;
      at = first + count;
      ++launches;
      const int64_t grid = (count + 7) / 8 * 8;   // as xcd_grid rounds it
      most = std::max(most, grid * threads);
    });
    std::printf("%d %lld %lld %d %lld\n", threads, static_cast<long long>(total), static_cast<long long>(launches),
                covered && at == total, static_cast<long long>(most));
  }
  return 0;
}
