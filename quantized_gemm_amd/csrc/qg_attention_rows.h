// Which rows of the queries a sequence of the attention has.  Plain arithmetic, without HIP, so that host code can check
// it against the buffers' sizes.
#pragma once

#include <stdint.h>

namespace qg {

struct Queries {
  int32_t first, count;
};

// Rows begin .. end - 1 of the `tokens` that there are, max_q of them at most.  Offsets are data of the device: whatever they
// hold, the rows lie inside (none where they descend).  Both ends are brought to zero and above before they are
// subtracted, so that 32 bits hold the difference (comparisons of 64 go through the vector unit: 4% of a small call).
constexpr Queries sequence_queries(int32_t begin, int32_t end, int32_t tokens, int32_t max_q) {
  const int32_t first = begin > 0 ? begin : 0, below = end < tokens ? end : tokens, last = below > 0 ? below : 0;
  const int32_t n = last - first, some = n > 0 ? n : 0;
  return Queries{first, some < max_q ? some : max_q};
}

}  // namespace qg
