// Splitting a grid over launches (host only, no HIP).
#pragma once

#include <stdint.h>

#include <algorithm>

namespace w4a4 {

// Workgroups of `threads` that one launch takes at most: fewer than 2^32
// threads, in whole rounds over the 8 XCDs.
constexpr int64_t max_workgroups(int threads) { return ((int64_t{1} << 32) - 1) / threads / 8 * 8; }

// Calls launch(first, count) over [0, workgroups) in parts of at most
// max_workgroups(threads).
template <class F>
void launch_parts(int64_t workgroups, int threads, F launch) {
  const int64_t most = max_workgroups(threads);
  for (int64_t first = 0; first < workgroups; first += most) launch(first, std::min(most, workgroups - first));
}

}  // namespace w4a4
