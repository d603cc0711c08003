// pa_tree_accept.cu - keep the accepted nodes of draft trees in the KV cache.
//
// A tree's nodes were written behind their context, node j at position base + j
// (base = seq_len - T).  The accepted path p_0 < p_1 < ... moves to base, base + 1,
// ...: row base + i := row base + p_i, for K and V of every KV head, in place.
//
// Since p is strictly increasing, p_i >= i: when the rows move in ascending i, a
// destination i lies at or below its own source and strictly below every later
// source p_k (k > i), so no move overwrites a row that is still to be read.  The
// columns of a row are independent.  A thread therefore owns one 16-byte column
// (side, head, chunk) of its sequence and moves it row by row, up to kBatch rows
// loaded before the first is stored, with no barrier and no staging: a pure copy
// of (accepted - 1) * 2 * Hkv * D * element bytes each way.
//
// Bound: a chain of dependent reads (lengths, path, block table, rows), not the bytes: 256
// paths of 1 to 9 nodes, 8 heads of 128, read and write 8 MB in some 6 us on the device,
// in a call whose arguments' checks take the host longer.  Eight rows in flight per thread
// cover the rows' latency (paths of more than nine nodes take it twice).
#include <algorithm>

#include "pa_tree.cuh"

namespace pa {
namespace {

__device__ unsigned g_err_tree_accept;
std::atomic<bool> g_launched{false};  // in this process, on any device

constexpr int kBatch = 8;

struct AcceptArgs {
    uint4 *kv;
    const int32_t *accepted, *num_accepted, *block_tables, *seq_lens;
    int32_t *new_seq_lens;
    TreeGeom t;
    int num_blocks, block_size, num_kv_heads, max_blocks;
    int vecs;  // 16-byte vectors in one head's row
};

__global__ void __launch_bounds__(256) tree_accept_kernel(const AcceptArgs a) {
    // Pool row (side K, head 0) of each move's source and destination; -1: no move.
    __shared__ int s_src[64], s_dst[64];
    pdl_begin();
    const int s = blockIdx.x, i0 = threadIdx.x;
    // The list's entries are read with the sequence's data, before its count is known.
    int p = 0, p_before = -1;
    if (i0 < a.t.max_tree) {
        const int32_t *path = a.accepted + (size_t)s * a.t.max_tree;
        p = path[i0];
        if (i0 > 0) p_before = path[i0 - 1];
    }
    const TreeSpan span = tree_span(a.t, s);
    const int len = a.seq_lens[s], n = a.num_accepted[s];
    bool bad = span.n < 0 || len < span.n || len > (long long)a.max_blocks * a.block_size ||
               n < 0 || n > span.n;
    // The whole list is checked before a row moves.
    const bool mine = !bad && i0 < n;
    if (mine) bad = p < 0 || p >= span.n || p <= p_before;
    if (mine && !bad) {
        const int base = len - span.n;
        const int32_t *bt = a.block_tables + (size_t)s * a.max_blocks;
        const int b0 = bt[(base + p) / a.block_size], b1 = bt[(base + i0) / a.block_size];
        const bool out = b0 < 0 || b0 >= a.num_blocks || b1 < 0 || b1 >= a.num_blocks;
        if (out && p != i0) atomicOr(&g_err_tree_accept, kErrOob);
        const int rows = 2 * a.num_kv_heads * a.block_size;  // of a block
        s_src[i0] = out || p == i0 ? -1 : b0 * rows + (base + p) % a.block_size;
        s_dst[i0] = out || p == i0 ? -1 : b1 * rows + (base + i0) % a.block_size;
    }
    bad = __syncthreads_or(bad);
    if (blockIdx.y == 0 && i0 == 0) {
        if (bad) atomicOr(&g_err_tree_accept, kErrOob);
        if (a.new_seq_lens) a.new_seq_lens[s] = bad ? len : len - span.n + n;
    }
    if (bad) return;
    const int col = blockIdx.y * blockDim.x + i0;  // (side, head, vector)
    if (col >= 2 * a.num_kv_heads * a.vecs) return;
    const int row = col / a.vecs, c = col - row * a.vecs;  // row = side * Hkv + head
    auto at = [&](int r) { return ((int64_t)r + row * a.block_size) * a.vecs + c; };
    for (int i = 0; i < n; i += kBatch) {
        uint4 x[kBatch];
        int dst[kBatch];
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            dst[k] = i + k < n ? s_dst[i + k] : -1;
            if (dst[k] >= 0) x[k] = a.kv[at(s_src[i + k])];
        }
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (dst[k] >= 0) a.kv[at(dst[k])] = x[k];
    }
}

}  // namespace

cudaError_t take_error_tree_accept(unsigned *bits) {
    return take_error_word(g_launched, g_err_tree_accept, bits);
}

cudaError_t launch_tree_accept(void *kv_cache, const KvGeom &g, int elem_bytes,
                               const int32_t *accepted, const int32_t *num_accepted,
                               const TreeGeom &t, const int32_t *block_tables,
                               int max_blocks_per_seq, const int32_t *seq_lens,
                               int32_t *new_seq_lens, cudaStream_t stream) {
    AcceptArgs a;
    a.kv = static_cast<uint4 *>(kv_cache);
    a.accepted = accepted;
    a.num_accepted = num_accepted;
    a.block_tables = block_tables;
    a.seq_lens = seq_lens;
    a.new_seq_lens = new_seq_lens;
    a.t = t;
    a.num_blocks = g.num_blocks;
    a.block_size = g.block_size;
    a.num_kv_heads = g.num_kv_heads;
    a.max_blocks = max_blocks_per_seq;
    a.vecs = g.head_size * elem_bytes / 16;
    const int cols = 2 * g.num_kv_heads * a.vecs;
    // At least the 64 threads that check a path.
    const int threads = std::min(256, std::max(64, (cols + 31) / 32 * 32));
    const dim3 grid((unsigned)t.num_seqs, (unsigned)((cols + threads - 1) / threads));
    g_launched.store(true);
    return launch_pdl(tree_accept_kernel, grid, threads, 0, 1, stream, a);
}

}  // namespace pa
