// Where a group's rows begin and end, from bounds that only the device has seen.
#pragma once

#include <cstdint>

namespace deto {

// Bound g, brought into [0, limit]. Bounds of an array that goes down somewhere
// (`down`) count as the largest up to them, so that no row has two groups and
// the groups' tiles and blocks are never more than in order they could be.
__device__ __forceinline__ int group_bound(const int32_t *offsets, int limit, int g, bool down)
{
    int v = min(max(offsets[g], 0), limit);
    if (down)
        for (int i = 0; i < g; ++i) v = max(v, min(offsets[i], limit));
    return v;
}

}  // namespace deto
