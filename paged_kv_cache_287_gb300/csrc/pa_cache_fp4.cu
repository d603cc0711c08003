// pa_cache_fp4.cu - rows of K and V into a 4-bit pool (quantised) and back (bf16).
//
// A thread per 16 elements, the group that shares a scale: 32 bytes of bf16 on one side, 8 bytes
// of codes and one of scale on the other.  Both directions are bound by HBM: 2.56 bytes an
// element, each moved once.
#include <algorithm>
#include <atomic>

#include "pa_fp4.cuh"
#include "pa_tree.cuh"

namespace pa {
namespace {

__device__ unsigned g_err_cache_fp4;
std::atomic<bool> g_launched{false};

struct RowsArgs {
    uint8_t *kv;
    uint4 *k, *v;  // rows of the caller's, row_vecs 16-byte vectors apart
    const int32_t *slots;
    int64_t row_vecs, num_slots;
    int num_tokens, block_size, num_kv_heads;
    float gk, gv, hk, hv;  // k_scale, v_scale, and six times those
};

// The slot of token tok, or -1 for none.
__device__ __forceinline__ int slot_of(const RowsArgs &a, int tok) {
    const int slot = a.slots[tok];
    if (slot >= 0 && slot >= a.num_slots) {
        atomicOr(&g_err_cache_fp4, kErrOob);
        return -1;
    }
    return slot;
}

template <int D, bool kWrite>
__global__ void __launch_bounds__(256) rows_kernel(const RowsArgs a) {
    pdl_begin();
    constexpr int kGroups = D / kFp4Group;  // of a head's row
    const int per_side = a.num_kv_heads * kGroups;
    const int64_t total = (int64_t)a.num_tokens * 2 * per_side;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total;
         i += (int64_t)gridDim.x * 256) {
        const int tok = (int)(i / (2 * per_side));
        const int r = (int)(i - (int64_t)tok * 2 * per_side);
        const int side = r >= per_side;
        const int col = r - side * per_side, head = col / kGroups, grp = col % kGroups;
        const int slot = slot_of(a, tok);
        if (slot < 0) continue;
        const int blk = slot / a.block_size;
        const Fp4Row row =
            fp4_row<D>(blk, slot - blk * a.block_size, head, side, a.num_kv_heads, a.block_size);
        uint4 *rows = (side ? a.v : a.k) + (int64_t)tok * a.row_vecs + 2 * col;
        uint2 *codes = reinterpret_cast<uint2 *>(a.kv + row.codes) + grp;
        const float g = side ? a.gv : a.gk;
        if constexpr (kWrite) {
            const uint4 x0 = rows[0], x1 = rows[1];
            const uint32_t x[8] = {x0.x, x0.y, x0.z, x0.w, x1.x, x1.y, x1.z, x1.w};
            uint2 c;
            const uint32_t s = fp4_quantise(x, g, side ? a.hv : a.hk, c);
            *codes = c;
            a.kv[row.scale + grp] = (uint8_t)s;
        } else {
            const uint2 c = *codes;
            const uint32_t s = a.kv[row.scale + grp];
            const uint32_t sc = e4m3x2_to_f16x2(s | s << 8);
            uint32_t o[8];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                uint32_t f[4];
                e2m1x8_to_f16x8(k ? c.y : c.x, f);
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    const uint32_t p = hmul2_u32(f[j], sc);  // exact
                    o[4 * k + j] = pack_bf16(__fmul_rn(f16_lo(p), g), __fmul_rn(f16_hi(p), g));
                }
            }
            rows[0] = make_uint4(o[0], o[1], o[2], o[3]);
            rows[1] = make_uint4(o[4], o[5], o[6], o[7]);
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
    a.k = static_cast<uint4 *>(k_rows);
    a.v = static_cast<uint4 *>(v_rows);
    a.slots = slots;
    a.row_vecs = row_stride / 8;
    a.num_slots = (int64_t)g.num_blocks * g.block_size;
    a.num_tokens = num_tokens;
    a.block_size = g.block_size;
    a.num_kv_heads = g.num_kv_heads;
    a.gk = k_scale;
    a.gv = v_scale;
    a.hk = 6.f * k_scale;
    a.hv = 6.f * v_scale;
    const long long work =
        (long long)num_tokens * 2 * g.num_kv_heads * (g.head_size / kFp4Group);
    const int blocks =
        (int)std::min<long long>((work + 255) / 256, (long long)device_sm_count() * 8);
    g_launched.store(true);
    auto kern = g.head_size == 128 ? (write ? rows_kernel<128, true> : rows_kernel<128, false>)
                                   : (write ? rows_kernel<64, true> : rows_kernel<64, false>);
    return launch_pdl(kern, dim3((unsigned)blocks), 256, 0, 1, stream, a);
}

}  // namespace pa
