// pa_tree.cuh - draft trees: what the pa_tree_* kernels share.
#pragma once

#include <atomic>

#include "pa_common.cuh"
#include "pa_internal.h"

namespace pa {

// Read a translation unit's device error word, and clear it where it is set; nothing to
// read before this process's first launch of its kernels.  (A copy takes the host some 7 us:
// with a read and a clearing of all six words pa_error_check took 84 us.)
template <typename Word>
cudaError_t take_error_word(const std::atomic<bool> &launched, Word &word, unsigned *bits) {
    *bits = 0;
    if (!launched.load()) return cudaSuccess;
    const unsigned zero = 0;
    const cudaError_t e = cudaMemcpyFromSymbol(bits, word, sizeof(unsigned));
    return e == cudaSuccess && *bits ? cudaMemcpyToSymbol(word, &zero, sizeof(unsigned)) : e;
}

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

// The top of every kernel launched by launch_pdl: the next launch may begin, and what
// came before has completed.
__device__ __forceinline__ void pdl_begin() {
    asm volatile("griddepcontrol.launch_dependents;" :::);
    asm volatile("griddepcontrol.wait;" ::: "memory");
}

// Launch as a programmatic dependent of whatever comes before on the stream (its launch
// and set-up overlap that kernel's end): every kernel here waits (griddepcontrol.wait)
// before it reads or writes memory.  cluster: CTAs per cluster.
template <typename... P>
cudaError_t launch_pdl(void (*kern)(P...), dim3 grid, int threads, size_t smem, int cluster,
                       cudaStream_t stream, P... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3((unsigned)threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = (unsigned)cluster;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = cluster > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, kern, args...);
}

}  // namespace pa
