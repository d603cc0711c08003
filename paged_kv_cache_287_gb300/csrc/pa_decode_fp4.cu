// pa_decode_fp4.cu - decode attention over a 4-bit pool: one query token per sequence.
#include <algorithm>
#include <atomic>

#include "pa_fp4.cuh"
#include "pa_tree.cuh"

namespace pa {
namespace {

__device__ unsigned g_err_decode_fp4;
std::atomic<bool> g_launched{false};

struct Args {
    __nv_bfloat16 *out;
    const __nv_bfloat16 *q;
    const uint8_t *kv;
    const int32_t *block_tables, *seq_lens;
    int num_heads, num_kv_heads, group, block_size, max_blocks, num_blocks, max_seq_len;
    float scale_log2, k_scale, v_scale;
};

// A CTA per (sequence, KV head), eight warps that take every eighth token.
template <int D>
__global__ void __launch_bounds__(256) decode_fp4_kernel(const Args a) {
    pdl_begin();
    constexpr int E = D / 32;  // elements per lane
    __shared__ float s_acc[8][8][D];
    __shared__ float s_m[8][8], s_l[8][8];
    const int s = blockIdx.x / a.num_kv_heads, h = blockIdx.x % a.num_kv_heads;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, G = a.group;
    const int cap = min(a.max_seq_len, a.max_blocks * a.block_size);
    int len = a.seq_lens[s];
    if (len < 0 || len > cap) {
        atomicOr(&g_err_decode_fp4, kErrOob);
        len = len < 0 ? 0 : cap;
    }
    const __nv_bfloat16 *q = a.q + ((size_t)s * a.num_heads + (size_t)h * G) * D;
    float acc[8][E], qv[8][E], m[8], l[8];
#pragma unroll
    for (int g = 0; g < 8; ++g) {
        m[g] = -3.4028235e38f;
        l[g] = 0.f;
#pragma unroll
        for (int e = 0; e < E; ++e) {
            acc[g][e] = 0.f;
            qv[g][e] = g < G ? __bfloat162float(q[g * D + lane * E + e]) : 0.f;
        }
    }
    auto element = [&](const Fp4Row &row, int e) {
        const int d = lane * E + e;
        const uint32_t byte = a.kv[row.codes + d / 2];
        uint32_t f[4];
        e2m1x8_to_f16x8(byte, f);
        const float c = d & 1 ? f16_hi(f[0]) : f16_lo(f[0]);
        return c * f16_lo(e4m3x2_to_f16x2(a.kv[row.scale + d / kFp4Group]));
    };
    for (int t = warp; t < len; t += 8) {
        const int blk = a.block_tables[(size_t)s * a.max_blocks + t / a.block_size];
        const bool oob = blk < 0 || blk >= a.num_blocks;
        if (oob) atomicOr(&g_err_decode_fp4, kErrOob);
        const Fp4Row kr =
            fp4_row<D>(oob ? 0 : blk, t % a.block_size, h, 0, a.num_kv_heads, a.block_size);
        const Fp4Row vr =
            fp4_row<D>(oob ? 0 : blk, t % a.block_size, h, 1, a.num_kv_heads, a.block_size);
        float k[E], v[E];
#pragma unroll
        for (int e = 0; e < E; ++e) {
            k[e] = oob ? 0.f : element(kr, e);
            v[e] = oob ? 0.f : element(vr, e);
        }
#pragma unroll
        for (int g = 0; g < 8; ++g) {
            if (g >= G) break;
            float x = 0.f;
#pragma unroll
            for (int e = 0; e < E; ++e) x += qv[g][e] * k[e];
#pragma unroll
            for (int o = 16; o; o >>= 1) x += __shfl_xor_sync(0xffffffffu, x, o);
            x *= a.scale_log2 * a.k_scale;
            const float mn = fmaxf(m[g], x), c = fast_exp2(m[g] - mn), p = fast_exp2(x - mn);
            m[g] = mn;
            l[g] = l[g] * c + p;
#pragma unroll
            for (int e = 0; e < E; ++e) acc[g][e] = acc[g][e] * c + p * v[e];
        }
    }
#pragma unroll
    for (int g = 0; g < 8; ++g) {
        if (lane == 0) {
            s_m[warp][g] = m[g];
            s_l[warp][g] = l[g];
        }
#pragma unroll
        for (int e = 0; e < E; ++e) s_acc[warp][g][lane * E + e] = acc[g][e];
    }
    __syncthreads();
    for (int i = threadIdx.x; i < G * D; i += 256) {
        const int g = i / D, d = i % D;
        float M = s_m[0][g], num = 0.f, den = 0.f;
        for (int w = 1; w < 8; ++w) M = fmaxf(M, s_m[w][g]);
        for (int w = 0; w < 8; ++w) {
            const float c = fast_exp2(s_m[w][g] - M);
            num += c * s_acc[w][g][d];
            den += c * s_l[w][g];
        }
        a.out[((size_t)s * a.num_heads + (size_t)h * G + g) * D + d] =
            __float2bfloat16_rn(len == 0 ? 0.f : num / den * a.v_scale);
    }
}

}  // namespace

cudaError_t take_error_decode_fp4(unsigned *bits) {
    return take_error_word(g_launched, g_err_decode_fp4, bits);
}

size_t decode_fp4_workspace_bytes(int head_size, int sm_count) {
    return (size_t)sm_count * 2 * 8 * (head_size + 2) * 4 + 256;
}

cudaError_t launch_decode_fp4(void *out, const void *q, const void *kv_cache, const KvGeom &g,
                              int num_heads, const int32_t *block_tables, int max_blocks_per_seq,
                              const int32_t *seq_lens, int num_seqs, int max_seq_len, float scale,
                              float k_scale, float v_scale, void *workspace,
                              cudaStream_t stream) {
    Args a;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.kv = static_cast<const uint8_t *>(kv_cache);
    a.block_tables = block_tables;
    a.seq_lens = seq_lens;
    a.num_heads = num_heads;
    a.num_kv_heads = g.num_kv_heads;
    a.group = num_heads / g.num_kv_heads;
    a.block_size = g.block_size;
    a.max_blocks = max_blocks_per_seq;
    a.num_blocks = g.num_blocks;
    a.max_seq_len = max_seq_len;
    a.scale_log2 = scale * 1.4426950408889634f;
    a.k_scale = k_scale;
    a.v_scale = v_scale;
    g_launched.store(true);
    const dim3 grid((unsigned)num_seqs * (unsigned)g.num_kv_heads);
    if (g.head_size == 128)
        return launch_pdl(decode_fp4_kernel<128>, grid, 256, 0, 1, stream, a);
    return launch_pdl(decode_fp4_kernel<64>, grid, 256, 0, 1, stream, a);
}

}  // namespace pa
