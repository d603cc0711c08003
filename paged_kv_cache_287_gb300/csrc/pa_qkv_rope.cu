// pa_qkv_rope.cu - a projection's q, k, v rows on their way to the attention, in one pass:
// norms of q and k per head, rotary positions, q out, K and V into the pool.
//
//   norm       y = x / sqrt(mean(x^2) + eps) * w, over a head's elements
//   rotation   pair (a, b) by the angle of its position: (a c - b s, b c + a s).  Pair i of
//              rot_dim / 2 is (i, i + rot_dim / 2), or (2i, 2i + 1) when interleaved; its
//              position is that of axis pair_axis[i]
// All of it in fp32 from the bf16 input to one rounding: q and K to bf16, from which an FP8 or
// 4-bit pool quantises K as pa_cache_write_fp8 / pa_cache_write_fp4 would.  Products and sums of
// the rotation are rounded apart (no fused multiply-add), so that a rotation without a norm
// gives the same bits as the formula's steps in fp32.
//
// Bound by HBM: every element read once and written once.  A thread holds the two 8-element
// vectors that a rotation pairs (t and t + rot_dim / 16 vectors further; or 2t and 2t + 1), so
// rotating needs no exchange; head_size / 16 threads make a head, a warp 4 or 8 heads.  The
// cosines and sines of a token stay in registers for all heads that a warp takes of it.
#include <algorithm>
#include <atomic>

#include "pa_fp4.cuh"
#include "pa_tree.cuh"

namespace pa {
namespace {

__device__ unsigned g_err_qkv_rope;
std::atomic<bool> g_launched{false};

// One 8-element bf16 vector as 8 floats, and back.
__device__ __forceinline__ void unpack8(const uint4 &v, float (&x)[8]) {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        x[2 * i] = bf16_lo(w[i]);
        x[2 * i + 1] = bf16_hi(w[i]);
    }
}
__device__ __forceinline__ uint4 pack8(const float (&x)[8]) {
    return make_uint4(pack_bf16(x[0], x[1]), pack_bf16(x[2], x[3]), pack_bf16(x[4], x[5]),
                      pack_bf16(x[6], x[7]));
}

__device__ __forceinline__ uint2 fp8_codes(const uint4 &v, float scale) {
    float x[8];
    unpack8(v, x);
    uint32_t c[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        c[i] = pack_e4m3x2(__fdiv_rn(x[2 * i], scale), __fdiv_rn(x[2 * i + 1], scale));
    return make_uint2(c[0] | c[1] << 16, c[2] | c[3] << 16);
}

template <int D, int kBits>
__global__ void __launch_bounds__(256) qkv_rope_kernel(const QkvRopeArgs a) {
    pdl_begin();
    constexpr int kLanes = D / 16;            // threads of a head
    constexpr int kHeads = 32 / kLanes;       // heads of a warp
    const int lane = threadIdx.x & 31, t = lane % kLanes;
    const int warp = blockIdx.x * 8 + (threadIdx.x >> 5);
    const int heads = a.num_heads + 2 * a.num_kv_heads;
    const int groups = (heads + kHeads - 1) / kHeads;
    const int tok = warp / a.chunks, chunk = warp - tok * a.chunks;
    if (tok >= a.num_tokens) return;

    // This thread's vectors of a rotated head, and its pairs' cosines and sines.
    const bool turns = t < a.rot_dim / 16;
    const bool split = turns && !a.interleaved;
    const int v0 = split ? t : 2 * t, v1 = split ? t + a.rot_dim / 16 : 2 * t + 1;
    float c[8], s[8];
    bool bad = false;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        c[i] = 1.f;
        s[i] = 0.f;
        if (turns) {
            int axis = a.pair_axis ? a.pair_axis[8 * t + i] : 0;
            if (axis < 0 || axis >= a.num_axes) {
                atomicOr(&g_err_qkv_rope, kErrOob);
                axis = 0;
            }
            const int pos = a.positions[(int64_t)axis * a.num_tokens + tok];
            if (pos < 0 || pos >= a.max_position) {
                bad = true;
            } else {
                const float *row = a.cos_sin + (int64_t)pos * a.rot_dim + 8 * t + i;
                c[i] = row[0];
                s[i] = row[a.rot_dim / 2];
            }
        }
    }
    if (__any_sync(0xffffffffu, bad)) {  // nothing of this token is written
        if (lane == 0) atomicOr(&g_err_qkv_rope, kErrOob);
        return;
    }
    int slot = a.slots[tok];
    if (slot >= 0 && slot >= (int64_t)a.num_blocks * a.block_size) {
        if (lane == 0) atomicOr(&g_err_qkv_rope, kErrOob);
        slot = -1;
    }
    const int blk = slot < 0 ? 0 : slot / a.block_size, off = slot - blk * a.block_size;

    for (int grp = chunk; grp < groups; grp += a.chunks) {
        const int hd = grp * kHeads + lane / kLanes;
        const bool live = hd < heads;
        const bool is_q = hd < a.num_heads, is_v = hd >= a.num_heads + a.num_kv_heads;
        const int side = is_v ? 1 : 0, kvh = hd - a.num_heads - side * a.num_kv_heads;
        const int i0 = is_v ? 2 * t : v0, i1 = is_v ? 2 * t + 1 : v1;
        uint4 y0 = make_uint4(0, 0, 0, 0), y1 = y0;
        if (live) {
            const uint4 *row = reinterpret_cast<const uint4 *>(a.qkv + (int64_t)tok * a.row_stride +
                                                               (int64_t)hd * D);
            y0 = row[i0];
            y1 = row[i1];
        }
        if (!is_v || !live) {
            float x0[8], x1[8];
            unpack8(y0, x0);
            unpack8(y1, x1);
            float r = 1.f;
            const uint4 *w = static_cast<const uint4 *>(is_q ? a.q_weight : a.k_weight);
            if (w) {
                float q = 0.f;
#pragma unroll
                for (int i = 0; i < 8; ++i) q += x0[i] * x0[i] + x1[i] * x1[i];
                // The lanes of this head: those of V's heads are not here.
                const uint32_t mask = ((1u << kLanes) - 1u) << (lane - t);
#pragma unroll
                for (int o = 1; o < kLanes; o <<= 1) q += __shfl_xor_sync(mask, q, o);
                r = 1.f / sqrtf(q * (1.f / D) + a.eps);
                float w0[8], w1[8];
                unpack8(w[i0], w0);
                unpack8(w[i1], w1);
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    x0[i] = x0[i] * r * w0[i];
                    x1[i] = x1[i] * r * w1[i];
                }
            }
            if (turns) {
#pragma unroll
                for (int i = 0; i < 8; ++i) {
                    // pair i of this thread: (x0[i], x1[i]), or two neighbours
                    float &p = split ? x0[i] : (i < 4 ? x0[2 * (i & 3)] : x1[2 * (i & 3)]);
                    float &q = split ? x1[i] : (i < 4 ? x0[2 * (i & 3) + 1] : x1[2 * (i & 3) + 1]);
                    const float pc = __fmul_rn(p, c[i]), qs = __fmul_rn(q, s[i]);
                    const float qc = __fmul_rn(q, c[i]), ps = __fmul_rn(p, s[i]);
                    p = __fsub_rn(pc, qs);
                    q = __fadd_rn(qc, ps);
                }
            }
            y0 = pack8(x0);
            y1 = pack8(x1);
        }
        __syncwarp();
        if (live && is_q) {
            uint4 *o = reinterpret_cast<uint4 *>(a.q_out) +
                       ((int64_t)tok * a.num_heads + hd) * (D / 8);
            o[i0] = y0;
            o[i1] = y1;
        }
        if constexpr (kBits == 4) {
            // A scale's 16 elements are vectors 2t and 2t + 1: fetch them from where they are.
            const int half = a.rot_dim / 16;
            uint32_t x[8];
#pragma unroll
            for (int k = 0; k < 2; ++k) {
                const int v = 2 * t + k;
                int from = t, second = k;  // lane of the head, and which of its two vectors
                if (!is_v && !a.interleaved && v < 2 * half) {
                    from = v < half ? v : v - half;
                    second = v < half ? 0 : 1;
                }
                const int src = lane - t + from;
                const uint32_t w0[4] = {y0.x, y0.y, y0.z, y0.w};
                const uint32_t w1[4] = {y1.x, y1.y, y1.z, y1.w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    const uint32_t p = __shfl_sync(0xffffffffu, w0[i], src);
                    const uint32_t q = __shfl_sync(0xffffffffu, w1[i], src);
                    x[4 * k + i] = second ? q : p;
                }
            }
            if (live && !is_q && slot >= 0) {
                const Fp4Row row = fp4_row<D>(blk, off, kvh, side, a.num_kv_heads, a.block_size);
                const float g = side ? a.v_scale : a.k_scale;
                uint2 codes;
                uint8_t *kv = static_cast<uint8_t *>(a.kv);
                kv[row.scale + t] = (uint8_t)fp4_quantise(x, g, 6.f * g, codes);
                reinterpret_cast<uint2 *>(kv + row.codes)[t] = codes;
            }
        } else if (live && !is_q && slot >= 0) {
            const int64_t row =
                ((((int64_t)blk * 2 + side) * a.num_kv_heads + kvh) * a.block_size + off) * (D / 8);
            if constexpr (kBits == 16) {
                uint4 *kv = static_cast<uint4 *>(a.kv) + row;
                kv[i0] = y0;
                kv[i1] = y1;
            } else {
                uint2 *kv = static_cast<uint2 *>(a.kv) + row;
                const float g = side ? a.v_scale : a.k_scale;
                kv[i0] = fp8_codes(y0, g);
                kv[i1] = fp8_codes(y1, g);
            }
        }
    }
}

}  // namespace

cudaError_t take_error_qkv_rope(unsigned *bits) {
    return take_error_word(g_launched, g_err_qkv_rope, bits);
}

cudaError_t launch_qkv_rope(QkvRopeArgs a, int head_size, int kv_bits, cudaStream_t stream) {
    const int per_warp = 32 / (head_size / 16);
    const int groups = (a.num_heads + 2 * a.num_kv_heads + per_warp - 1) / per_warp;
    // A warp takes a token's heads, or a share of them while that leaves warps idle.
    const long long want = (long long)device_sm_count() * 32;
    a.chunks = (int)std::min<long long>(groups, (want + a.num_tokens - 1) / a.num_tokens);
    const long long warps = (long long)a.num_tokens * a.chunks;
    const dim3 grid((unsigned)((warps + 7) / 8));
    g_launched.store(true);
    auto pick = [&](auto k128, auto k64) {
        return launch_pdl(head_size == 128 ? k128 : k64, grid, 256, 0, 1, stream, a);
    };
    if (kv_bits == 16) return pick(qkv_rope_kernel<128, 16>, qkv_rope_kernel<64, 16>);
    if (kv_bits == 8) return pick(qkv_rope_kernel<128, 8>, qkv_rope_kernel<64, 8>);
    return pick(qkv_rope_kernel<128, 4>, qkv_rope_kernel<64, 4>);
}

}  // namespace pa
