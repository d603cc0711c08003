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
// vectors that a rotation pairs (t and t + rot_dim / 16 vectors further; or two with pairs of
// their own), so rotating needs no exchange; head_size / 16 threads make a head, a warp a group of 4 or 8 heads
// (1 KB).  A warp takes a token, whose cosines and sines stay in registers for all its heads,
// and copies its next groups into shared memory ahead (each thread its own vectors, so nothing
// is synchronised); 151 instructions a group of query heads with a norm, 96 without.
//
// 4344 tokens of 32 + 2 x 8 heads of 128, bf16 pool, in a graph over three states: 18.9 us with
// one axis (5.7 TB/s moved, 85 % of the copy rate; norms make no difference), 20.1 with three
// (a lane holds an axis' position, asked for before the axes are known: 20.7 without);
// FP8 pool 18.5, 4-bit 21.1 (64 bytes of codes and 8 of scales a head scatter more).  When the
// ring came (three axes): 21.7; with the rows loaded to registers two groups at a time 28.8,
// rings of 4, 5, 8 groups 22.1, 22.3, 27.8 (fewer blocks fit), a token shared by two warps 25.3,
// blocks of 128 and 64 threads 22.2, 22.8.
#include <algorithm>
#include <atomic>

#include "pa_fp4.cuh"
#include "pa_tree.cuh"

namespace pa {
namespace {

__device__ unsigned g_err_qkv_rope;
std::atomic<bool> g_launched{false};

// The 16 elements of a thread as 8 pairs (p[i], q[i]): the elements of its two vectors, or
// neighbours; and back.
template <bool kNeighbours>
__device__ __forceinline__ void unpack(const uint4 &y0, const uint4 &y1, float (&p)[8],
                                       float (&q)[8]) {
    const uint32_t w[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if constexpr (kNeighbours) {
            p[i] = bf16_lo(w[i]);
            q[i] = bf16_hi(w[i]);
        } else {
            float(&x)[8] = i < 4 ? p : q;
            x[2 * i % 8] = bf16_lo(w[i]);
            x[2 * i % 8 + 1] = bf16_hi(w[i]);
        }
    }
}
template <bool kNeighbours>
__device__ __forceinline__ void pack(const float (&p)[8], const float (&q)[8], uint4 &y0,
                                     uint4 &y1) {
    uint32_t w[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float(&x)[8] = i < 4 ? p : q;
        w[i] = kNeighbours ? pack_bf16(p[i], q[i]) : pack_bf16(x[2 * i % 8], x[2 * i % 8 + 1]);
    }
    y0 = make_uint4(w[0], w[1], w[2], w[3]);
    y1 = make_uint4(w[4], w[5], w[6], w[7]);
}

constexpr int kThreads = 256;
constexpr int kRing = 3;        // groups of heads (1 KB each) in flight per warp
constexpr int kPerSm = 4;       // blocks; 32 warps of 64 registers
constexpr int kWarpsPerSm = 24; // a token's heads are shared out while there are fewer warps

// What divides K and V: by the scales (FP8), by six times those (4 bits).
struct Divisors {
    Around k, v;
};

// kNeighbours: pairs are neighbours (interleaved).
template <int D, int kBits, bool kNeighbours>
__global__ void __launch_bounds__(kThreads, kPerSm) qkv_rope_kernel(const QkvRopeArgs a,
                                                                  const Divisors by) {
    constexpr int kLanes = D / 16;       // threads of a head
    constexpr int kHeads = 32 / kLanes;  // heads of a warp
    __shared__ uint4 ring[kThreads / 32][kRing][2][32];
    __shared__ __align__(16) float weights[2][D];  // of q's and K's norms
    pdl_begin();
    const int lane = threadIdx.x & 31, t = lane % kLanes;
    const int warp = blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5);
    const int heads = a.num_heads + 2 * a.num_kv_heads, rot_heads = a.num_heads + a.num_kv_heads;
    const int groups = (heads + kHeads - 1) / kHeads;
    const int tok = warp / a.chunks, chunk = warp - tok * a.chunks;
    const bool idle = tok >= a.num_tokens;

    // This thread's two vectors of a rotated head: those that a pair joins, or kLanes apart where
    // pairs are neighbours (a warp's 16-byte accesses then lie side by side: with 2t and 2t + 1
    // the 4344 tokens took 29 us instead of 20); of V's, too, but for a 4-bit pool's, where
    // vectors 2t and 2t + 1 share a scale.
    const bool split = !kNeighbours && t < a.rot_dim / 16;
    const int v0 = split || kNeighbours ? t : 2 * t;
    const int v1 = split ? t + a.rot_dim / 16 : (kNeighbours ? t + kLanes : 2 * t + 1);
    const int u0 = kBits == 4 ? 2 * t : t, u1 = kBits == 4 ? 2 * t + 1 : t + kLanes;
    // Its pairs, four and four: whether they turn, and the first.
    const bool turns[2] = {kNeighbours ? 8 * v0 < a.rot_dim : split,
                           kNeighbours ? 8 * v1 < a.rot_dim : split};
    const int pair[2] = {kNeighbours ? 4 * v0 : 8 * t, kNeighbours ? 4 * v1 : 8 * t + 4};
    const int first = lane / kLanes * (D / 8);  // its head's first vector in a group's 64

    // The first rows are asked for before what the rest hangs on.
    const uint4 *row = reinterpret_cast<const uint4 *>(a.qkv + (int64_t)tok * a.row_stride);
    uint4(*mine)[2][32] = ring[threadIdx.x >> 5];
    auto fetch = [&](int grp, int at) {
        const int hd = grp * kHeads + lane / kLanes;
        if (hd < heads) {
            const uint4 *head = row + 64 * grp + first;
            copy16(&mine[at][0][lane], head + (hd < rot_heads ? v0 : u0));
            copy16(&mine[at][1][lane], head + (hd < rot_heads ? v1 : u1));
        }
        copies_commit();
    };
    int slot = -1, pos[8], axis[8], own = 0;  // own: the position of axis `lane`
    if (!idle) {
#pragma unroll
        for (int k = 0; k < kRing; ++k) fetch(min(chunk + k * a.chunks, groups), k);
        slot = a.slots[tok];
        if (a.pair_axis) {
#pragma unroll
            for (int i = 0; i < 8; ++i)
                axis[i] = turns[i / 4] ? a.pair_axis[pair[i / 4] + i % 4] : 0;
            if (lane < a.num_axes) own = a.positions[(int64_t)lane * a.num_tokens + tok];
        } else {
            pos[0] = a.positions[tok];
        }
    }
    if (a.q_weight || a.k_weight) {
        // (neighbours: of each vector the first ones of its pairs, then the second ones)
        for (int i = threadIdx.x; i < 2 * D; i += kThreads) {
            const void *w = i < D ? a.q_weight : a.k_weight;
            const int from = kNeighbours ? (i & ~7) | (2 * i & 6) | (i >> 2 & 1) : i;
            if (w)
                (&weights[0][0])[i] =
                    __bfloat162float(static_cast<const __nv_bfloat16 *>(w)[from % D]);
        }
        __syncthreads();
    }
    if (idle) return;

    // Their positions, cosines and sines.
    float c[8], s[8];
    bool bad = false, one[2] = {true, true};  // one: a single position for the four
    if (a.pair_axis) {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            if (axis[i] < 0 || axis[i] >= a.num_axes) {
                atomicOr(&g_err_qkv_rope, kErrOob);
                axis[i] = 0;
            }
            one[i / 4] = one[i / 4] && axis[i] == axis[i & 4];
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            pos[i] = __shfl_sync(0xffffffffu, own, axis[i]);
            bad = bad || (turns[i / 4] && (pos[i] < 0 || pos[i] >= a.max_position));
        }
    } else {
        pos[4] = pos[0];
        bad = (turns[0] || turns[1]) && (pos[0] < 0 || pos[0] >= a.max_position);
    }
    if (__any_sync(0xffffffffu, bad)) {  // nothing of this token is written
        if (lane == 0) atomicOr(&g_err_qkv_rope, kErrOob);
        copies_wait<0>();
        return;
    }
#pragma unroll
    for (int h = 0; h < 2; ++h) {
#pragma unroll
        for (int i = 4 * h; i < 4 * h + 4; ++i) {
            c[i] = 1.f;
            s[i] = 0.f;
        }
        if (!turns[h]) continue;
        if (one[h]) {
            const float *cs = a.cos_sin + (int64_t)pos[4 * h] * a.rot_dim + pair[h];
            const float4 u = *reinterpret_cast<const float4 *>(cs);
            const float4 v = *reinterpret_cast<const float4 *>(cs + a.rot_dim / 2);
            c[4 * h] = u.x, c[4 * h + 1] = u.y, c[4 * h + 2] = u.z, c[4 * h + 3] = u.w;
            s[4 * h] = v.x, s[4 * h + 1] = v.y, s[4 * h + 2] = v.z, s[4 * h + 3] = v.w;
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const float *cs = a.cos_sin + (int64_t)pos[4 * h + i] * a.rot_dim + pair[h] + i;
                c[4 * h + i] = cs[0];
                s[4 * h + i] = cs[a.rot_dim / 2];
            }
        }
    }
    if (slot >= 0 && slot >= (int64_t)a.num_blocks * a.block_size) {
        if (lane == 0) atomicOr(&g_err_qkv_rope, kErrOob);
        slot = -1;
    }
    const int blk = slot < 0 ? 0 : slot / a.block_size, off = slot - blk * a.block_size;
    uint4 *q_out = static_cast<uint4 *>(a.q_out) + (int64_t)tok * a.num_heads * (D / 8);

    // Norm and rotation of this thread's 16 elements of a head.
    const bool whole = a.rot_dim == D;
    auto transform = [&](uint4 &y0, uint4 &y1, bool norm, const float *w) {
        float p[8], q[8];
        unpack<kNeighbours>(y0, y1, p, q);
        if (norm) {
            float sum0 = 0.f, sum1 = 0.f;
#pragma unroll
            for (int i = 0; i < 8; i += 2) {
                fma2(sum0, sum1, p[i], p[i + 1], p[i], p[i + 1], sum0, sum1);
                fma2(sum0, sum1, q[i], q[i + 1], q[i], q[i + 1], sum0, sum1);
            }
            float sum = sum0 + sum1;
            // The lanes of this head: in a group with V's heads not all are here.
            const uint32_t mask = ((1u << kLanes) - 1u) << (lane - t);
#pragma unroll
            for (int o = 1; o < kLanes; o <<= 1) sum += __shfl_xor_sync(mask, sum, o);
            const float r = rsqrtf(sum * (1.f / D) + a.eps);
            // Of the pairs' first and second elements: a vector's each, or half of both.
            const float4 *w0 = reinterpret_cast<const float4 *>(w + 8 * v0);
            const float4 *w1 = reinterpret_cast<const float4 *>(w + 8 * v1);
#pragma unroll
            for (int i = 0; i < 8; i += 4) {
                const float4 u = kNeighbours ? (i ? w1[0] : w0[0]) : w0[i / 4];
                const float4 v = kNeighbours ? (i ? w1[1] : w0[1]) : w1[i / 4];
                mul2(p[i], p[i + 1], r, r);
                mul2(p[i + 2], p[i + 3], r, r);
                mul2(q[i], q[i + 1], r, r);
                mul2(q[i + 2], q[i + 3], r, r);
                mul2(p[i], p[i + 1], u.x, u.y);
                mul2(p[i + 2], p[i + 3], u.z, u.w);
                mul2(q[i], q[i + 1], v.x, v.y);
                mul2(q[i + 2], q[i + 3], v.z, v.w);
            }
        }
        auto turn = [&](int i) {  // pairs i and i + 1
            float pc0 = p[i], pc1 = p[i + 1], ps0 = p[i], ps1 = p[i + 1];
            float qc0 = q[i], qc1 = q[i + 1], qs0 = q[i], qs1 = q[i + 1];
            mul2(pc0, pc1, c[i], c[i + 1]);
            mul2(ps0, ps1, s[i], s[i + 1]);
            mul2(qc0, qc1, c[i], c[i + 1]);
            mul2(qs0, qs1, s[i], s[i + 1]);
            fma2(p[i], p[i + 1], qs0, qs1, -1.f, -1.f, pc0, pc1);  // pc - qs, rounded once
            add2(qc0, qc1, ps0, ps1);
            q[i] = qc0;
            q[i + 1] = qc1;
        };
        if (whole) {  // no lane but turns
#pragma unroll
            for (int i = 0; i < 8; i += 2) turn(i);
        } else {
#pragma unroll
            for (int i = 0; i < 8; i += 2)
                if (turns[i / 4]) turn(i);
        }
        pack<kNeighbours>(p, q, y0, y1);
    };

    // Groups of q's heads alone, then the others.
    int at = 0, grp = chunk;
    for (; (grp + 1) * kHeads <= a.num_heads; grp += a.chunks) {
        copies_wait<kRing - 1>();
        uint4 y0 = mine[at][0][lane], y1 = mine[at][1][lane];
        transform(y0, y1, a.q_weight != nullptr, weights[0]);
        fetch(min(grp + kRing * a.chunks, groups), at);
        at = at + 1 == kRing ? 0 : at + 1;
        uint4 *o = q_out + 64 * grp + first;
        o[v0] = y0;
        o[v1] = y1;
    }
    // K's and V's heads lie one after the other in the pool's block, too (not in a 4-bit one).
    const int64_t at_slot =
        ((int64_t)blk * 2 * a.num_kv_heads * a.block_size + off) * (D / 8);
    for (; grp < groups; grp += a.chunks) {
        const int hd = grp * kHeads + lane / kLanes, kvh2 = hd - a.num_heads;
        const bool live = hd < heads, is_q = kvh2 < 0, is_v = hd >= rot_heads;
        const int i0 = is_v ? u0 : v0, i1 = is_v ? u1 : v1;
        copies_wait<kRing - 1>();
        uint4 y0 = mine[at][0][lane], y1 = mine[at][1][lane];
        if (!is_v)
            transform(y0, y1, (is_q ? a.q_weight : a.k_weight) != nullptr, weights[is_q ? 0 : 1]);
        fetch(min(grp + kRing * a.chunks, groups), at);
        at = at + 1 == kRing ? 0 : at + 1;
        __syncwarp();
        if (is_q) {
            uint4 *o = q_out + 64 * grp + first;
            o[i0] = y0;
            o[i1] = y1;
        }
        if (slot < 0) continue;
        const int side = is_v ? 1 : 0;
        if constexpr (kBits == 4) {
            // A scale's 16 elements are vectors 2t and 2t + 1: of K they are fetched from where
            // they are.
            uint32_t x[8] = {y0.x, y0.y, y0.z, y0.w, y1.x, y1.y, y1.z, y1.w};
            if (__any_sync(0xffffffffu, live && !is_q && !is_v)) {
                const int half = kNeighbours ? kLanes : a.rot_dim / 16;
                const uint32_t w0[4] = {y0.x, y0.y, y0.z, y0.w};
                const uint32_t w1[4] = {y1.x, y1.y, y1.z, y1.w};
#pragma unroll
                for (int e = 0; e < 2; ++e) {
                    const int v = 2 * t + e;
                    const bool moved = !is_v && v < 2 * half;
                    const int src = lane - t + (!moved ? t : (v < half ? v : v - half));
                    const bool second = moved ? v >= half : e != 0;
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const uint32_t p = __shfl_sync(0xffffffffu, w0[i], src);
                        const uint32_t q = __shfl_sync(0xffffffffu, w1[i], src);
                        x[4 * e + i] = second ? q : p;
                    }
                }
            }
            if (live && !is_q) {
                const Fp4Row to = fp4_row<D>(blk, off, kvh2 - side * a.num_kv_heads, side,
                                             a.num_kv_heads, a.block_size);
                uint2 codes;
                uint8_t *kv = static_cast<uint8_t *>(a.kv);
                kv[to.scale + t] = (uint8_t)fp4_quantise(
                    x, side ? Fp4Scale{a.v_scale, 6.f * a.v_scale, by.v}
                            : Fp4Scale{a.k_scale, 6.f * a.k_scale, by.k},
                    codes);
                reinterpret_cast<uint2 *>(kv + to.codes)[t] = codes;
            }
        } else if (live && !is_q) {
            const int64_t to = at_slot + kvh2 * a.block_size * (D / 8);
            if constexpr (kBits == 16) {
                uint4 *kv = static_cast<uint4 *>(a.kv) + to;
                kv[i0] = y0;
                kv[i1] = y1;
            } else {
                uint2 *kv = static_cast<uint2 *>(a.kv) + to;
                const float g = side ? a.v_scale : a.k_scale;
                const Around r = side ? by.v : by.k;
                kv[i0] = e4m3_of_quotients(y0, g, r);
                kv[i1] = e4m3_of_quotients(y1, g, r);
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
    const long long want = (long long)device_sm_count() * kWarpsPerSm;
    a.chunks = (int)std::min<long long>(groups, (want + a.num_tokens - 1) / a.num_tokens);
    const long long warps = (long long)a.num_tokens * a.chunks;
    const dim3 grid((unsigned)((warps + kThreads / 32 - 1) / (kThreads / 32)));
    const float times = kv_bits == 4 ? 6.f : 1.f;
    const Divisors by{around(times * a.k_scale), around(times * a.v_scale)};
    g_launched.store(true);
    auto pick = [&](auto k128, auto k64, auto n128, auto n64) {
        return launch_pdl(a.interleaved ? (head_size == 128 ? n128 : n64)
                                        : (head_size == 128 ? k128 : k64),
                          grid, kThreads, 0, 1, stream, a, by);
    };
    if (kv_bits == 16)
        return pick(qkv_rope_kernel<128, 16, false>, qkv_rope_kernel<64, 16, false>,
                    qkv_rope_kernel<128, 16, true>, qkv_rope_kernel<64, 16, true>);
    if (kv_bits == 8)
        return pick(qkv_rope_kernel<128, 8, false>, qkv_rope_kernel<64, 8, false>,
                    qkv_rope_kernel<128, 8, true>, qkv_rope_kernel<64, 8, true>);
    return pick(qkv_rope_kernel<128, 4, false>, qkv_rope_kernel<64, 4, false>,
                qkv_rope_kernel<128, 4, true>, qkv_rope_kernel<64, 4, true>);
}

}  // namespace pa
