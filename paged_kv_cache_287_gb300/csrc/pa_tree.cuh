// pa_tree.cuh - draft trees: what the pa_tree_* kernels share.
#pragma once

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {

// Sequence s's tree: rows [row0, row0 + n) of the node arrays.  n = -1 where the
// offsets are not those of a tree of at most max_tree nodes within the arrays.
struct TreeSpan {
    int row0, n;
};

__device__ __forceinline__ TreeSpan tree_span(const TreeGeom &t, int s) {
    const int lo = t.cu[s], hi = t.cu[s + 1];
    if (lo < 0 || hi < lo || hi > t.total_nodes || hi - lo > t.max_tree) return {0, -1};
    return {lo, hi - lo};
}

}  // namespace pa
