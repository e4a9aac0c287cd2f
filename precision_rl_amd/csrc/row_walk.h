// Rows of a group shared out among threads (host and device, no HIP).
#pragma once

#include <stdint.h>

namespace w4a4 {

// Calls f(r) for r = r0 + first, r0 + first + step, ... below r1.  Row indices go
// up to 2^31 - 1, and a thread's first row may lie behind the group's end: in 32
// bits it would be negative there, below r1, and written in front of the buffer.
template <class F>
constexpr void walk_rows(int64_t r0, int64_t r1, int first, int step, F f) {
  for (int64_t r = r0 + first; r < r1; r += step) f(r);
}

}  // namespace w4a4
