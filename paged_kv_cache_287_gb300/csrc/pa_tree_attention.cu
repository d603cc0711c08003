// pa_tree_attention.cu - attention of draft trees over a paged KV cache.
//
// Node i of a sequence's tree (T nodes behind a context of seq_len - T tokens)
// attends to the context, to its ancestors and to itself:
//   out = sum_t softmax_t(scale q.K_t) V_t.
// One warp per (node, query head): the lanes share the head's dims, the keys are
// taken one at a time with a running maximum and sum.
#include <algorithm>

#include "pa_tree.cuh"

namespace pa {
namespace {

__device__ unsigned g_err_tree_attention;

struct TreeAttnArgs {
    __nv_bfloat16 *out;
    const __nv_bfloat16 *q;
    const uint8_t *kv;
    const int32_t *block_tables, *seq_lens;
    TreeGeom t;
    int num_heads, num_kv_heads, group;
    int block_size, max_blocks, num_blocks;
    float scale, k_scale, v_scale;
};

template <int D, bool KV8>
__global__ void __launch_bounds__(128) tree_attention_kernel(const TreeAttnArgs a) {
    constexpr int kPer = D / 32;  // dims a lane holds
    const int s = blockIdx.y, lane = threadIdx.x & 31;
    const TreeSpan span = tree_span(a.t, s);
    const int len = a.seq_lens[s];
    if (span.n < 0 || len < span.n || len > (long long)a.max_blocks * a.block_size) {
        if (threadIdx.x == 0) atomicOr(&g_err_tree_attention, kErrOob);
        return;
    }
    const int w = blockIdx.x * 4 + (threadIdx.x >> 5);
    const int node = w / a.num_heads, hq = w - node * a.num_heads;
    if (node >= span.n) return;
    const int h = hq / a.group;
    const size_t row = ((size_t)(span.row0 + node) * a.num_heads + hq) * D + lane * kPer;
    float q[kPer], acc[kPer], m = -INFINITY, l = 0.f;
#pragma unroll
    for (int i = 0; i < kPer; ++i) {
        q[i] = __bfloat162float(a.q[row + i]);
        acc[i] = 0.f;
    }
    const int32_t *bt = a.block_tables + (size_t)s * a.max_blocks;
    auto key = [&](int pos) {
        const int blk = bt[pos / a.block_size];
        float k[kPer] = {}, v[kPer] = {};
        if (blk < 0 || blk >= a.num_blocks) {
            if (lane == 0) atomicOr(&g_err_tree_attention, kErrOob);
        } else {
            const size_t kr = (((size_t)blk * 2 * a.num_kv_heads + h) * a.block_size +
                               pos % a.block_size) * D + lane * kPer;
            const size_t vr = kr + (size_t)a.num_kv_heads * a.block_size * D;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                if constexpr (KV8) {
                    uint32_t x, y, z;
                    e4m3x4_to_f16x4((uint32_t)a.kv[kr + i] | (uint32_t)a.kv[vr + i] << 8, x, y);
                    z = x;
                    k[i] = f16_lo(z) * a.k_scale;
                    v[i] = f16_hi(z) * a.v_scale;
                } else {
                    const __nv_bfloat16 *kv = reinterpret_cast<const __nv_bfloat16 *>(a.kv);
                    k[i] = __bfloat162float(kv[kr + i]);
                    v[i] = __bfloat162float(kv[vr + i]);
                }
            }
        }
        float x = 0.f;
#pragma unroll
        for (int i = 0; i < kPer; ++i) x += q[i] * k[i];
        for (int o = 16; o > 0; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
        x *= a.scale;
        const float mn = fmaxf(m, x);
        const float c = __expf(m - mn), p = __expf(x - mn);
        m = mn;
        l = l * c + p;
#pragma unroll
        for (int i = 0; i < kPer; ++i) acc[i] = acc[i] * c + p * v[i];
    };
    const int ctx = len - span.n;
    for (int pos = 0; pos < ctx; ++pos) key(pos);
    for (int j = node; j >= 0;) {
        key(ctx + j);
        const int up = a.t.parents[span.row0 + j];
        if (up < -1 || up >= j) {
            if (lane == 0) atomicOr(&g_err_tree_attention, kErrOob);
            break;
        }
        j = up;
    }
#pragma unroll
    for (int i = 0; i < kPer; ++i) a.out[row + i] = __float2bfloat16_rn(acc[i] / l);
}

}  // namespace

cudaError_t take_error_tree_attention(unsigned *bits) {
    unsigned zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(bits, g_err_tree_attention, sizeof(unsigned));
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_err_tree_attention, &zero, sizeof(unsigned));
    return e;
}

size_t tree_attention_workspace_bytes(int num_seqs, int max_tree, int group, int head_size,
                                      int sm_count) {
    return 256;
}

cudaError_t launch_tree_attention(void *out, const void *q, const TreeGeom &t,
                                  const void *kv_cache, const KvGeom &g, int num_heads,
                                  const int32_t *block_tables, int max_blocks_per_seq,
                                  const int32_t *seq_lens, int max_seq_len, float scale, bool kv8,
                                  float k_scale, float v_scale, void *workspace,
                                  cudaStream_t stream) {
    TreeAttnArgs a;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.kv = static_cast<const uint8_t *>(kv_cache);
    a.block_tables = block_tables;
    a.seq_lens = seq_lens;
    a.t = t;
    a.num_heads = num_heads;
    a.num_kv_heads = g.num_kv_heads;
    a.group = num_heads / g.num_kv_heads;
    a.block_size = g.block_size;
    a.max_blocks = max_blocks_per_seq;
    a.num_blocks = g.num_blocks;
    a.scale = scale;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    const dim3 grid((unsigned)((t.max_tree * num_heads + 3) / 4), (unsigned)t.num_seqs);
    if (t.num_seqs > 65535) return cudaErrorInvalidValue;
    if (kv8)
        tree_attention_kernel<128, true><<<grid, 128, 0, stream>>>(a);
    else if (g.head_size == 128)
        tree_attention_kernel<128, false><<<grid, 128, 0, stream>>>(a);
    else
        tree_attention_kernel<64, false><<<grid, 128, 0, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace pa
