// pa_cache_fp4.cu - rows of K and V into a 4-bit pool (quantised) and back (bf16).
//
// A thread per 16 elements, the group that shares a scale: 32 bytes of bf16 on one side, 8 bytes
// of codes and one of scale on the other: 2.56 bytes an element, each moved once.  What bounds the
// write is its quantising, during which a thread has no loads in flight, and the starts and ends of
// its passes (3.2 TB/s at 4344 tokens, 4.6 at 32768); the read-back waits for memory (ncu: 10 of 14
// cycles between a warp's instructions; 83 % of the copy rate).  A block's threads lie over the groups of one token's K and V rows
// (several tokens where those are few), so that a thread keeps its column and finds only the
// token's slot anew; it takes two or four tokens at once to have as many loads in flight.
//
// 4344 tokens of 2 x 8 heads of 128, in a graph: written in 7.2 us (7.5 at a scale of 1, whose
// ties are common; 10.9 when each tie was divided, 12 with a division per element), read back in
// 5.9 (6.0 and 4.7 where three pools in turn stay in L2); 32768 tokens 37 and 30.9, 4.6 and 5.6
// TB/s.  Stores with other cache policies (evict first, streaming, write through) change nothing in
// the read-back.
#include <algorithm>
#include <atomic>

#include "pa_fp4.cuh"
#include "pa_tree.cuh"

namespace pa {
namespace {

__device__ unsigned g_err_cache_fp4;
std::atomic<bool> g_launched{false};

constexpr int kThreads = 256;
// Tokens of a thread in flight, and blocks per SM (quantising takes the registers).
template <bool kWrite>
constexpr int kTokens = kWrite ? 2 : 4;
template <bool kWrite>
constexpr int kPerSm = kWrite ? 3 : 4;

struct RowsArgs {
    uint8_t *kv;
    uint8_t *k, *v;  // rows of the caller's, row_bytes apart
    const int32_t *slots;
    int64_t row_bytes, num_slots;
    int num_tokens, block_shift, num_kv_heads;
    int wide;  // rows lie on 32-byte boundaries
    Fp4Scale ks, vs;
};

template <int D, bool kWrite>
__global__ void __launch_bounds__(kThreads, kPerSm<kWrite>) rows_kernel(const RowsArgs a) {
    pdl_begin();
    constexpr int kGroups = D / kFp4Group;  // of a head's row
    constexpr int kTok = kTokens<kWrite>;
    const int per_side = a.num_kv_heads * kGroups, cols = 2 * per_side;
    const int width = min(cols, kThreads), at_once = kThreads / width;  // tokens of a block's pass
    const int first = threadIdx.x / width;
    if (first >= at_once) return;
    const int bs = 1 << a.block_shift;
    const unsigned step = gridDim.x * at_once, tokens = a.num_tokens;  // (sums pass 2^31)
    for (int col = threadIdx.x - first * width; col < cols; col += width) {
        const int side = col >= per_side, c = col - side * per_side;
        const int head = c / kGroups, grp = c % kGroups;
        const Fp4Scale scale_of = side ? a.vs : a.ks;
        const float g = scale_of.g;
        uint8_t *rows = (side ? a.v : a.k) + c * 32;
        for (unsigned tok = blockIdx.x * at_once + first; tok < tokens; tok += kTok * step) {
            uint32_t x[kTok][8];
            uint2 codes[kTok];
            uint32_t scale[kTok];
            int slot[kTok];
            Fp4Row row[kTok];
#pragma unroll
            for (int k = 0; k < kTok; ++k) {
                const unsigned t = tok + k * step;
                slot[k] = t < tokens ? a.slots[t] : -1;
                if (kWrite && t < tokens) {  // a skipped row's is there as well
                    const uint8_t *p = rows + (int64_t)t * a.row_bytes;
                    if (a.wide) {
                        ld_32(x[k], p);
                    } else {
                        const uint4 y = reinterpret_cast<const uint4 *>(p)[0];
                        const uint4 z = reinterpret_cast<const uint4 *>(p)[1];
                        x[k][0] = y.x, x[k][1] = y.y, x[k][2] = y.z, x[k][3] = y.w;
                        x[k][4] = z.x, x[k][5] = z.y, x[k][6] = z.z, x[k][7] = z.w;
                    }
                }
            }
#pragma unroll
            for (int k = 0; k < kTok; ++k) {
                if (slot[k] >= a.num_slots) {
                    atomicOr(&g_err_cache_fp4, kErrOob);
                    slot[k] = -1;
                }
                if (slot[k] < 0) continue;
                row[k] = fp4_row<D>(slot[k] >> a.block_shift, slot[k] & (bs - 1), head, side,
                                    a.num_kv_heads, bs);
                if constexpr (!kWrite) {
                    codes[k] = reinterpret_cast<const uint2 *>(a.kv + row[k].codes)[grp];
                    scale[k] = a.kv[row[k].scale + grp];
                }
            }
#pragma unroll
            for (int k = 0; k < kTok; ++k) {
                if (slot[k] < 0) continue;
                if constexpr (kWrite) {
                    uint2 q;
                    const uint32_t s = fp4_quantise(x[k], scale_of, q);
                    reinterpret_cast<uint2 *>(a.kv + row[k].codes)[grp] = q;
                    a.kv[row[k].scale + grp] = (uint8_t)s;
                } else {
                    const uint32_t sc = e4m3x2_to_f16x2(scale[k] | scale[k] << 8);
                    uint32_t o[8];
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        uint32_t f[4];
                        e2m1x8_to_f16x8(w ? codes[k].y : codes[k].x, f);
#pragma unroll
                        for (int j = 0; j < 4; ++j) {
                            const uint32_t p = hmul2_u32(f[j], sc);  // exact
                            float lo = f16_lo(p), hi = f16_hi(p);
                            mul2(lo, hi, g, g);
                            o[4 * w + j] = pack_bf16(lo, hi);
                        }
                    }
                    uint8_t *p = rows + (int64_t)(tok + k * step) * a.row_bytes;
                    if (a.wide) {
                        st_32(p, o);
                    } else {
                        reinterpret_cast<uint4 *>(p)[0] = make_uint4(o[0], o[1], o[2], o[3]);
                        reinterpret_cast<uint4 *>(p)[1] = make_uint4(o[4], o[5], o[6], o[7]);
                    }
                }
            }
        }
    }
}

}  // namespace

cudaError_t take_error_cache_fp4(unsigned *bits) {
    return take_error_word(g_launched, g_err_cache_fp4, bits);
}

cudaError_t launch_cache_fp4(bool write, void *kv_cache, const KvGeom &g, void *k_rows,
                             void *v_rows, int64_t row_stride, const int32_t *slots,
                             int num_tokens, float k_scale, float v_scale, cudaStream_t stream) {
    RowsArgs a;
    a.kv = static_cast<uint8_t *>(kv_cache);
    a.k = static_cast<uint8_t *>(k_rows);
    a.v = static_cast<uint8_t *>(v_rows);
    a.slots = slots;
    a.row_bytes = row_stride * 2;
    a.num_slots = (int64_t)g.num_blocks * g.block_size;
    a.num_tokens = num_tokens;
    a.block_shift = g.block_size == 8 ? 3 : (g.block_size == 16 ? 4 : 5);
    a.num_kv_heads = g.num_kv_heads;
    a.wide = (reinterpret_cast<uintptr_t>(k_rows) | reinterpret_cast<uintptr_t>(v_rows) |
              (uintptr_t)a.row_bytes) % 32 == 0;
    a.ks = fp4_scale(k_scale);
    a.vs = fp4_scale(v_scale);
    const int cols = 2 * g.num_kv_heads * (g.head_size / kFp4Group);
    const int at_once = kThreads / std::min(cols, kThreads);
    // Blocks that fill the GPU once, or a token per thread where that takes fewer.
    const long long passes = ((long long)num_tokens + at_once - 1) / at_once;
    const int blocks = (int)std::min<long long>(passes, (long long)device_sm_count() *
                                                               (write ? kPerSm<true> : kPerSm<false>));
    g_launched.store(true);
    auto kern = g.head_size == 128 ? (write ? rows_kernel<128, true> : rows_kernel<128, false>)
                                   : (write ? rows_kernel<64, true> : rows_kernel<64, false>);
    return launch_pdl(kern, dim3((unsigned)blocks), kThreads, 0, 1, stream, a);
}

}  // namespace pa
