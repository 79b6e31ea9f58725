// Which rows of the queries a sequence of the attention has.  Plain arithmetic, without HIP, so that host code can check
// it against the buffers' sizes.
#pragma once

#include <stdint.h>

namespace qg {

struct Queries {
  int64_t first;
  int count;
};

// Rows begin .. end - 1 of the `tokens` that there are, max_q of them at most.  Offsets are data of the device: whatever they
// hold, the rows lie inside (none where they descend, by more than 2^31, too).
constexpr Queries sequence_queries(int32_t begin, int32_t end, int64_t tokens, int max_q) {
  const int64_t first = begin < 0 ? 0 : begin, last = end < tokens ? end : tokens, n = last - first;
  return Queries{first, n <= 0 ? 0 : n < max_q ? (int)n : max_q};
}

}  // namespace qg
