// Host check: prints, per device number of the command line, whether the call
// succeeded and how often the setter has run for it; a device number below zero
// stands for that device (its absolute value) with a setter that fails.
#include <cstdio>
#include <cstdlib>
#include <map>

#include "../precision_rl_amd/csrc/once_per_device.h"

int main(int argc, char** argv) {
  w4a4::OncePerDevice once;
  std::map<int, int> runs;
  for (int a = 1; a < argc; ++a) {
    const int n = std::atoi(argv[a]), device = std::abs(n);
    const bool ok = once(device, [&] { ++runs[device]; return n >= 0; });
    std::printf("%d %d\n", ok ? 1 : 0, runs[device]);
  }
  return 0;
}
