// Layout of the decode workspace.
#pragma once

#include "fa_internal.cuh"

namespace far {

// The status block and the split counters of the calls that have no more
// (slice, KV head) pairs than fit here; the partials of every call begin behind
// it.  Counters are zero between calls and partials are not, so where the one
// ends must not depend on a call's shape: calls of any shapes may use one
// workspace in turn.  A call with more pairs has its counters behind this block
// and clears them itself.
constexpr size_t kFixedBytes = 16384;
constexpr size_t kFixedUnits = (kFixedBytes - kStatusBytes) / sizeof(unsigned int);

}  // namespace far
