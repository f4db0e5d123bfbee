// The workspace of a split decode: merge counters at its start, one int per
// unit of work, then the chunks' results.  It is zero-filled once and may serve
// calls of any shape in turn, but where one plan has results another has
// counters.  So the first kCounterSpan bytes are zero between calls: the CTA
// that joins a unit's chunks resets the unit's counter and clears those of its
// chunks' results that lie in the span (16 KB in all, whatever the plan).  A
// plan with more counters than the span holds has them cleared before it.
#pragma once

#include <cstddef>

namespace sa {

constexpr size_t kCounterSpan = 16384;

// End of the span of a workspace that starts with `counters`.
__device__ __forceinline__ const float *counter_span_end(const int *counters) {
  return reinterpret_cast<const float *>(counters + kCounterSpan / sizeof(int));
}

}  // namespace sa
