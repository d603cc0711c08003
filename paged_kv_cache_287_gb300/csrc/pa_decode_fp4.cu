// pa_decode_fp4.cu - decode attention over a 4-bit pool: one query token per sequence.
//
//   out[s][h] = v_scale sum_t P[t] (code s)_V[t] / sum_t P[t],
//   P[t] = 2^(scale log2(e) k_scale (x[t] - m)), x[t] = q.(code s)_K[t], m a running reference
//   that gives the largest 2^11 to 2^15
//
// Bound by HBM: 9/16 of a byte per element, read once.  At that rate an SM meets some 43
// elements a clock, so the work per element must stay below three instructions, and the layout
// is chosen for that:
//   * Tiles of 32 tokens of one (sequence, KV head): K and V, codes and scales, of a block are
//     one run of memory, which the lanes of a warp copy 16 bytes each (asynchronously, nine
//     copies a tile).  Every warp has a ring of tiles of its own and no warp waits for another
//     in the loop; a stage is filled anew as soon as its V is in registers.
//   * S^T = K.Q^T by m16n8k16 (16 tokens x 8 query heads): a lane reads 32 dims (16 bytes) of
//     its token at once; which of the MMA's k-slots a dim takes is free, so the query's
//     fragments are laid out to match (32 consecutive dims a lane).  A byte of codes becomes an
//     f16x2 by one conversion, times its scale by one multiplication, both exact.
//   * O^T += V^T.P^T: MMA row g stands for dims 16 g .. 16 g + 15 over the m-tiles, so a lane's
//     dims share one scale per token; two tokens' nibbles are interleaved (two shifts and two
//     selects per 16 codes), and the conversion then gives pairs of tokens.  A lane ends with 16
//     consecutive dims of two heads and stores them as they are.
//   * Row r of a tile's 8 tokens is token r ^ ((r >> 1) & 1): without it the four tokens that a
//     load of V takes would lie in the same banks.
// The tiles of all (sequence, KV head) segments are one list, cut into equal ranges, one per
// CTA and within it one per warp.  Pieces of a segment in one CTA are merged in shared memory,
// those in several CTAs by a second kernel (a record per CTA and end of its range); few or short
// segments go to CTAs whole (rules at launch_decode_fp4).
//
// Measured (32 + 8 heads of 128, in a graph): 256 sequences of 512 - 4096 tokens 111.7 us,
// 92 % of the copy rate, 32 of up to 131072 tokens 154 us, 95 % (heads of 64: 256 sequences 74.5 us,
// 69 %, by its instructions, with a rolled loop of four stages); in the steady state 0.66 ns a
// tile of the whole GPU, 7.0 TB/s, so what is left are the ends (of 256 sequences: 2.1 us to the
// first copy, 2 from the median CTA's last tile to the last CTA's, 2 of merges, 1.1 of hand-over,
// 1.3 the second kernel).  Of 524 warp instructions a tile 302 are the products with their
// conversions, 39 the softmax, 95 loads, scales and interleaving, the rest copies, waits and
// bookkeeping.  Each of these brought its part: the tiles' blocks found 16 tiles at a time by all
// lanes and kept in a table (120, 163 without), the loop unrolled by its stages, so that their
// addresses are constants (118, 161 without).  Tried and slower: 12, 14 or 15 warps (117, 125,
// 119; the registers allow 16), 12 with three stages each (122); before those steps a bulk copy
// per block by one lane, completing on an mbarrier (by 2 %; the copies' uniform operands cost as
// many instructions, and the loads a fence before the next copy), 8 warps with four stages each
// (by a quarter), the last of the CTAs to come merging a segment in place of the second kernel
// (by 4 %).
#include <algorithm>
#include <atomic>
#include <cmath>
#include <type_traits>

#include "pa_fp4.cuh"
#include "pa_tree.cuh"

namespace pa {
namespace {

__device__ unsigned g_err_decode_fp4;
std::atomic<bool> g_launched{false};

constexpr int kTokens = 32;  // of a tile
constexpr int kWarps = 16;   // one CTA per SM
constexpr int kHeads = 8;    // query heads per KV head, padded to the MMA's N
// m lies kLift powers of two below a running maximum, and is only raised when a score exceeds that
// by more than kSlack: P reaches 2^15 (f16 ends at 2^16), and the weights of a tail keep f16's 11
// bits down to 2^-25 of the largest and are lost below 2^-36.  (With m at the maximum itself a tail
// of 2^-25 was in l, which is summed in fp32, but not in the product.)  m is kept in the scores' own
// units, so that the difference is taken before any scaling.
constexpr float kLift = 11.f, kSlack = 4.f;
constexpr float kLowest = -3.4028235e38f;  // m before the first score
// A record's m is in log2 units times this: a score is below 2^21 units of its own and their factor
// below 2^128, so that their product may be beyond binary32 and the differences that count not.
// That factor is at least kLeast, with which every weight is the same.
constexpr float kRecUnit = 0x1p-40f, kPerRecUnit = 0x1p40f, kLeast = 0x1p-80f;

template <int D>
constexpr int kStageBytes = kTokens *D * 9 / 8;
template <int D>
constexpr int kRecFloats = kHeads * (D + 2);  // acc [8][D], then (m, l) [8]
// Tiles in flight per warp: 147 KB in flight per SM; one where the batch's tables need the room.
template <int D>
constexpr int kMaxStages = 256 / D;

struct Args {
    __nv_bfloat16 *out;
    const __nv_bfloat16 *q;
    const uint8_t *kv;
    const int32_t *block_tables, *seq_lens;
    float *recs;  // [CTAs][2][kRecFloats]: a segment's piece at the range's start, at its end
    int4 *meta;   // [CTAs]: piece at the start, it ends here, piece at the end, its segment
    int num_seqs, num_heads, num_kv_heads, group, max_blocks, num_blocks, max_seq_len;
    int aligned;  // CTA c is segment c
    int whole;    // every CTA takes whole segments: no piece leaves it
    float factor, v_scale;  // factor * 2^factor_exp: scale * log2(e) * k_scale
    int factor_exp;
};

// What a warp leaves for the merge in its CTA: a piece of a segment that began before its range
// (a) and whether the segment ended there; one that began in its range and goes on (b).
struct WarpPieces {
    int a, a_ends, b, b_seg;
};

__device__ __forceinline__ int clamped(const Args &a, int len) {
    return len < 0 ? 0 : (len > a.max_seq_len ? a.max_seq_len : len);
}

// The sequence of tile x of the list: the last that begins at or before it.
__device__ __forceinline__ int sequence_of(const int *pre, int num_seqs, int num_kv_heads, int x) {
    int lo = 0, hi = num_seqs - 1;
    while (lo < hi) {
        const int mid = (lo + hi + 1) >> 1;
        if (num_kv_heads * pre[mid] <= x) lo = mid; else hi = mid - 1;
    }
    return lo;
}

// The score above which the reference -nm is raised, of a factor cs to log2 units.  It is rounded
// down and the reference up, so that no P passes 2^15 where scores are so large that their own steps
// come to several powers of two.  (The quotients may be off by their last bits; a cs above 2^126
// makes them 0, less than a step of any score.)
__device__ __forceinline__ float raised_above(float nm, float cs) {
    return __fsub_rd(__fdividef(kLift + kSlack, cs), nm);
}

// Flags of a tile beside its tokens: the last, the first of its segment.
constexpr int kLast = 64, kFirst = 128;
// Ints of a tile's entry: segment, flags, blocks; a multiple of two.
template <int BS>
constexpr int kEntryInts = BS == 8 ? 6 : 4;

// 16 (D 128) or 8 consecutive dims of one head: acc[mt][e] and acc[mt][e + 2] are dims 2 mt and
// 2 mt + 1 of them.  V's scale after the division by l: their quotient may be no normal number.
template <int D>
__device__ __forceinline__ void store_rows(__nv_bfloat16 *dst, const float (&acc)[D / 16][4],
                                           int e, float l, float v_scale) {
    const float inv = 1.f / l;
    uint32_t w[D / 16];
#pragma unroll
    for (int mt = 0; mt < D / 16; ++mt)
        w[mt] = pack_bf16(acc[mt][e] * inv * v_scale, acc[mt][e + 2] * inv * v_scale);
#pragma unroll
    for (int i = 0; i < D / 64; ++i)
        reinterpret_cast<uint4 *>(dst)[i] =
            make_uint4(w[4 * i], w[4 * i + 1], w[4 * i + 2], w[4 * i + 3]);
}

template <int D>
__device__ __forceinline__ void store_rec(float *rec, const float (&acc)[D / 16][4], int lane,
                                          float m0, float l0, float m1, float l1) {
    const int g = lane >> 2, c = lane & 3;
#pragma unroll
    for (int e = 0; e < 2; ++e) {
        float4 *dst = reinterpret_cast<float4 *>(rec + (2 * c + e) * D + g * (D / 8));
#pragma unroll
        for (int i = 0; i < D / 32; ++i)
            dst[i] = make_float4(acc[2 * i][e], acc[2 * i][e + 2], acc[2 * i + 1][e],
                                 acc[2 * i + 1][e + 2]);
    }
    if (g == 0)
        *reinterpret_cast<float4 *>(rec + kHeads * D + 4 * c) = make_float4(m0, l0, m1, l1);
}

template <int D, int BS, int S>
__global__ void __launch_bounds__(kWarps * 32, 1) decode_fp4_kernel(const Args a) {
    constexpr int kStage = kStageBytes<D>, kRec = kRecFloats<D>;
    constexpr int kTile = BS * D * 9 / 16;      // K's (or V's) bytes of a (block, head)
    constexpr int kNB = kTokens / BS;           // blocks of a tile
    constexpr int kRow = D / 2, kScRow = D / 16;
    extern __shared__ __align__(128) uint8_t smem[];
    constexpr int kEntry = kEntryInts<BS>;
    uint8_t *ring = smem;
    float *recs = reinterpret_cast<float *>(ring + kWarps * S * kStage);
    int *entries = reinterpret_cast<int *>(recs + kWarps * kRec) + (threadIdx.x >> 5) * 32 * kEntry;
    WarpPieces *pieces =
        reinterpret_cast<WarpPieces *>(recs + kWarps * (kRec + 32 * kEntry));
    int *sums = reinterpret_cast<int *>(pieces + kWarps);
    const int B = a.num_seqs, Hkv = a.num_kv_heads, G = a.group;
    int *lens = sums + kWarps;  // [num_seqs], and their tiles' prefix sums [num_seqs + 1];
    int *pre = lens + B;        // not in aligned mode

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int g = lane >> 2, c = lane & 3;
    uint8_t *stages = ring + warp * S * kStage;
    if (lane == 0) pieces[warp] = {0, 0, 0, 0};
    pdl_begin();

    // This warp's tiles [t0, t1) of the list (aligned mode: of its CTA's segment).
    int t0, t1, active;  // active: warps of this CTA with tiles
    int own_len = 0;     // aligned mode: the segment's tokens
    {
        int r0, r1;
        if (a.aligned) {
            const int len = a.seq_lens[blockIdx.x / Hkv];
            if (tid == 0 && (len < 0 || len > a.max_seq_len))
                atomicOr(&g_err_decode_fp4, kErrOob);
            own_len = clamped(a, len);
            r0 = 0;
            r1 = (own_len + kTokens - 1) / kTokens;
        } else {
            const int per = (B + kWarps * 32 - 1) / (kWarps * 32);
            for (int s = tid; s < B; s += kWarps * 32) {
                const int len = a.seq_lens[s];
                if (len < 0 || len > a.max_seq_len) atomicOr(&g_err_decode_fp4, kErrOob);
                lens[s] = clamped(a, len);
                pre[s] = (clamped(a, len) + kTokens - 1) / kTokens;
            }
            __syncthreads();
            int sum = 0;
            for (int i = tid * per; i < min(B, (tid + 1) * per); ++i) sum += pre[i];
            int v = sum;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int u = __shfl_up_sync(0xffffffffu, v, o);
                if (lane >= o) v += u;
            }
            if (lane == 31) sums[warp] = v;
            __syncthreads();
            // The sums of the warps before this one, lane w holding warp w's.
            int run = __reduce_add_sync(0xffffffffu, lane < warp ? sums[lane] : 0) + v - sum;
            for (int i = tid * per; i < min(B, (tid + 1) * per); ++i) {
                const int n = pre[i];
                pre[i] = run;
                run += n;
            }
            if (tid == kWarps * 32 - 1) pre[B] = run;
            __syncthreads();
            const int T = pre[B] * Hkv;  // below 2^31
            // With fewer tiles than CTAs the first T take one each: no range before another's
            // is empty, so a segment's pieces are those of consecutive CTAs.
            const int ctas = max(1, min(T, (int)gridDim.x));
            const int cta = blockIdx.x, each = T / ctas, rest = T - each * ctas;
            r0 = cta < ctas ? cta * each + min(cta, rest) : 0;
            r1 = cta < ctas ? r0 + each + (cta < rest) : 0;
            if (a.whole) {  // the nearest ends of segments
                auto end_near = [&](int x) {
                    if (x >= T) return T;
                    const int s = sequence_of(pre, B, Hkv, x), nt = pre[s + 1] - pre[s];
                    const int j = (x - Hkv * pre[s]) % nt;
                    return 2 * j < nt ? x - j : x - j + nt;
                };
                r0 = end_near(r0);
                r1 = end_near(r1);
            }
        }
        const int n = r1 - r0;
        active = min(n, kWarps);
        const int each = n / kWarps, rest = n % kWarps;
        t0 = r0 + warp * each + min(warp, rest);
        t1 = t0 + each + (warp < rest);
    }

    // Tile i of this warp has entry i % 32 of a table: its segment (sequence << 8 | head), its
    // tokens | kLast | kFirst, and its blocks as numbers of a (block, head) (-1: none, or outside
    // the pool).  `count` entries from tile `from` on, a lane each.
    const int n = t1 - t0;
    auto describe = [&](int from, int count) {
        const int i = from + lane, x = t0 + i;
        if (lane < count && i < n) {
            int s, h, j;
            if (a.aligned) {
                s = blockIdx.x / Hkv;
                h = blockIdx.x - s * Hkv;
                j = x;
            } else {
                s = sequence_of(pre, B, Hkv, x);
                const int nt = pre[s + 1] - pre[s], r = x - Hkv * pre[s];
                h = r / nt;
                j = r - h * nt;
            }
            const int left = (a.aligned ? own_len : lens[s]) - j * kTokens;
            const int32_t *bt = a.block_tables + (size_t)s * a.max_blocks + j * kNB;
            int *e = entries + i % 32 * kEntry;
            *reinterpret_cast<int2 *>(e) =
                make_int2(s << 8 | h, min(left, kTokens) | (left <= kTokens ? kLast : 0) |
                                          (j == 0 ? kFirst : 0));
#pragma unroll
            for (int b = 0; b < kNB; ++b) {
                int unit = -1;
                if (b * BS < left) {
                    const int id = bt[b];
                    if (id >= 0 && id < a.num_blocks)
                        unit = id * Hkv + h;
                    else
                        atomicOr(&g_err_decode_fp4, kErrOob);
                }
                e[2 + b] = unit;
            }
        }
        __syncwarp();
    };
    describe(0, 32);
    const uint64_t policy = policy_evict_first();

    // Called by the whole warp, for i in order: a group of copies, empty past the last tile.  A
    // lane copies every 32nd chunk of 16 bytes; a block that is not there becomes zeros.
    constexpr int kChunks = 2 * kTile / 16;  // of a block
    const uint32_t stages_at = smem_u32(stages) + lane * 16;
    const uint8_t *kv = a.kv + lane * 16;
    int refill = 24;  // the tile before whose copy the table's older half is written anew
    auto issue = [&](int i, int st) {
        if (i < n) {
            // (the table's older half has been used: S is at most 8)
            if (i == refill) {
                describe(i + 8, 16);
                refill += 16;
            }
            const int *units = entries + i % 32 * kEntry + 2;
            // Chunk `lane` of a tile that began with block b.
            int unit = units[0];
            auto base = [&](int b) {
                return kv + (int64_t)max(unit, 0) * (2 * kTile) - b * 2 * kTile;
            };
            const uint8_t *src = base(0);
            bool live = unit >= 0;
            const uint32_t dst = stages_at + st * kStage;
#pragma unroll
            for (int k = 0; k < (kNB * kChunks + 31) / 32; ++k) {
                // A block ends inside these 32 chunks, or none does (no block begins with them).
                const int b1 = (32 * k + 31) / kChunks;
                if (b1 > 32 * k / kChunks && b1 < kNB) {
                    const uint8_t *before = src;
                    const bool live_before = live, up = lane >= b1 * kChunks - 32 * k;
                    unit = units[b1];
                    src = base(b1);
                    live = unit >= 0;
                    copy16_hint(dst + 512 * k, (up ? src : before) + 512 * k,
                                up ? live : live_before, policy);
                } else if (32 * k + 32 <= kNB * kChunks || lane < kNB * kChunks - 32 * k) {
                    copy16_hint(dst + 512 * k, src + 512 * k, live, policy);
                }
            }
        }
        copies_commit();
    };
#pragma unroll
    for (int i = 0; i < S; ++i) issue(i, i);

    // Rows of sequences without tokens (while the first tiles are on their way).
    for (int s = a.aligned ? blockIdx.x / Hkv : blockIdx.x; s < B;
         s += a.aligned ? B : gridDim.x) {
        if (a.aligned ? active > 0 : pre[s + 1] != pre[s]) continue;
        const int rows = a.aligned ? G : a.num_heads;
        uint4 *dst = reinterpret_cast<uint4 *>(
            a.out + ((size_t)s * a.num_heads + (a.aligned ? blockIdx.x % Hkv * G : 0)) * D);
        for (int i = tid; i < rows * (D / 8); i += kWarps * 32) dst[i] = make_uint4(0, 0, 0, 0);
    }

    float acc[D / 16][4];
    uint32_t qf[D / 16][2];
    // Of heads 2c and 2c + 1: what brings a score to log2 units; in the score's own units minus
    // the reference, and the score above which it is raised; the sum of P.
    float cs0 = 0.f, cs1 = 0.f, nm0 = 0.f, nm1 = 0.f, bar0 = 0.f, bar1 = 0.f;
    float l0 = 0.f, l1 = 0.f;
    int seg = -1;
    bool inside = false;  // whether this piece begins inside its segment
    // Offsets of 8-token group j's first row, and of this lane's rows: K's row g is token rk of
    // the group, V's k-slots 2c and 2c + 1 are tokens rv and rv ^ 1.
    auto codes_at = [](int j) { return 8 * j / BS * 2 * kTile + 8 * j % BS * kRow; };
    auto scales_at = [](int j) { return 8 * j / BS * 2 * kTile + BS * kRow + 8 * j % BS * kScRow; };
    const int rk = g ^ ((g >> 1) & 1), rv = 2 * c + (c & 1);
    const int tok_v0 = rv, tok_v1 = rv ^ 1;

    auto step = [&](int i, int st) __attribute__((always_inline)) {
        // Of the S groups in flight the oldest is this tile.
        copies_wait<S - 1>();
        __syncwarp();
        const uint8_t *buf = stages + st * kStage;
        const int2 d = *reinterpret_cast<const int2 *>(entries + i % 32 * kEntry);
        const int valid = d.y & 63;
        if (d.x != seg) {
            // A new segment: its query heads, scaled by powers of two into [1, 2) at their
            // largest element.
            seg = d.x;
            inside = !(d.y & kFirst);
            float qv[D / 4];
            float mx = 0.f;
            const uint4 *src = reinterpret_cast<const uint4 *>(
                a.q + ((size_t)(seg >> 8) * a.num_heads + (seg & 255) * G + g) * D + c * (D / 4));
#pragma unroll
            for (int k = 0; k < D / 32; ++k) {
                const uint4 w = g < G ? src[k] : make_uint4(0, 0, 0, 0);
                const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    qv[8 * k + 2 * e] = bf16_lo(u[e]);
                    qv[8 * k + 2 * e + 1] = bf16_hi(u[e]);
                    mx = fmax3(mx, fabsf(bf16_lo(u[e])), fabsf(bf16_hi(u[e])));
                }
            }
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
            mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
            int ex = mx > 0.f ? (int)(__float_as_uint(mx) >> 23) - 127 : 0;
            ex = max(-126, min(126, ex));
            float down = __uint_as_float((uint32_t)(127 - ex) << 23);
            if (a.factor < 0.f) down = -down;
#pragma unroll
            for (int k = 0; k < D / 16; ++k) {
                qf[k][0] = pack_f16(qv[4 * k] * down, qv[4 * k + 1] * down);
                qf[k][1] = pack_f16(qv[4 * k + 2] * down, qv[4 * k + 3] * down);
            }
            const int e0 = __shfl_sync(0xffffffffu, ex, 8 * c);
            const int e1 = __shfl_sync(0xffffffffu, ex, 8 * c + 4);
            // The factor's exponent meets the query's before anything is rounded.  Positive and
            // finite, so that -inf stays -inf.
            const int f0 = max(-126, min(127, a.factor_exp + e0));
            const int f1 = max(-126, min(127, a.factor_exp + e1));
            cs0 = fabsf(a.factor) * __uint_as_float((uint32_t)(127 + f0) << 23);
            cs1 = fabsf(a.factor) * __uint_as_float((uint32_t)(127 + f1) << 23);
            cs0 = fminf(fmaxf(cs0, kLeast), -kLowest);
            cs1 = fminf(fmaxf(cs1, kLeast), -kLowest);
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt)
#pragma unroll
                for (int e = 0; e < 4; ++e) acc[mt][e] = 0.f;
            nm0 = nm1 = -kLowest;
            bar0 = raised_above(nm0, cs0);
            bar1 = raised_above(nm1, cs1);
            l0 = l1 = 0.f;
        }

        // Scores of two halves of 16 tokens: [0], [1] are heads 2c, 2c + 1 of row g, [2], [3] of
        // row g + 8.
        float x[2][4] = {{0.f, 0.f, 0.f, 0.f}, {0.f, 0.f, 0.f, 0.f}};
        {
            constexpr int kWords = D / 32;  // words of codes per lane and token
            uint32_t w[4][kWords], sl[4], sh[4];
#pragma unroll
            for (int r = 0; r < 4; ++r) {
                const uint8_t *row = buf + codes_at(r) + rk * kRow + c * (D / 8);
                const uint8_t *scl = buf + scales_at(r) + rk * kScRow + c * (D / 64);
                if constexpr (D == 128) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(row);
                    w[r][0] = v.x;
                    w[r][1] = v.y;
                    w[r][2] = v.z;
                    w[r][3] = v.w;
                    const uint32_t s2 =
                        e4m3x2_to_f16x2(*reinterpret_cast<const uint16_t *>(scl));
                    sl[r] = prmt(s2, 0u, 0x1010u);
                    sh[r] = prmt(s2, 0u, 0x3232u);
                } else {
                    const uint2 v = *reinterpret_cast<const uint2 *>(row);
                    w[r][0] = v.x;
                    w[r][1] = v.y;
                    const uint32_t b = *scl;
                    sl[r] = sh[r] = e4m3x2_to_f16x2(b | b << 8);
                }
            }
#pragma unroll
            for (int k = 0; k < kWords; ++k) {
#pragma unroll
                for (int m = 0; m < 2; ++m) {
                    uint32_t f0[4], f1[4];
                    e2m1x8_to_f16x8(w[2 * m][k], f0);
                    e2m1x8_to_f16x8(w[2 * m + 1][k], f1);
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        f0[e] = hmul2_u32(f0[e], 2 * k < kWords ? sl[2 * m] : sh[2 * m]);
                        f1[e] = hmul2_u32(f1[e], 2 * k < kWords ? sl[2 * m + 1] : sh[2 * m + 1]);
                    }
                    const uint32_t p[4] = {f0[0], f1[0], f0[1], f1[1]};
                    const uint32_t q[4] = {f0[2], f1[2], f0[3], f1[3]};
                    mma_f16(x[m], p, qf[2 * k][0], qf[2 * k][1]);
                    mma_f16(x[m], q, qf[2 * k + 1][0], qf[2 * k + 1][1]);
                }
            }
        }
        if (valid < kTokens) {
            // What lies behind the sequence may be anything: its scores are -inf, V's scales zero.
#pragma unroll
            for (int m = 0; m < 2; ++m) {
                if (16 * m + rk >= valid) x[m][0] = x[m][1] = -INFINITY;
                if (16 * m + 8 + rk >= valid) x[m][2] = x[m][3] = -INFINITY;
            }
            if (lane >= valid) {
                const int j = lane / 8, o = lane % 8;
                uint8_t *scl = stages + st * kStage + kTile + 8 * j / BS * 2 * kTile + BS * kRow +
                               (8 * j % BS + o) * kScRow;
                if constexpr (D == 128)
                    *reinterpret_cast<uint2 *>(scl) = make_uint2(0u, 0u);
                else
                    *reinterpret_cast<uint32_t *>(scl) = 0u;
            }
            __syncwarp();
        }
        float t0x = fmaxf(fmax3(x[0][0], x[0][2], x[1][0]), x[1][2]);
        float t1x = fmaxf(fmax3(x[0][1], x[0][3], x[1][1]), x[1][3]);
        if (__any_sync(0xffffffffu, t0x > bar0 || t1x > bar1)) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                t0x = fmaxf(t0x, __shfl_xor_sync(0xffffffffu, t0x, o));
                t1x = fmaxf(t1x, __shfl_xor_sync(0xffffffffu, t1x, o));
            }
            const float n0 = fminf(nm0, __fsub_rd(__fdividef(kLift, cs0), t0x));
            const float n1 = fminf(nm1, __fsub_rd(__fdividef(kLift, cs1), t1x));
            const float r0 = fast_exp2((n0 - nm0) * cs0), r1 = fast_exp2((n1 - nm1) * cs1);
            nm0 = n0;
            nm1 = n1;
            bar0 = raised_above(nm0, cs0);
            bar1 = raised_above(nm1, cs1);
            l0 *= r0;
            l1 *= r1;
#pragma unroll
            for (int mt = 0; mt < D / 16; ++mt) {
                acc[mt][0] *= r0;
                acc[mt][1] *= r1;
                acc[mt][2] *= r0;
                acc[mt][3] *= r1;
            }
        }
        // P, summed in fp32 before its rounding to f16; transposed to the MMA's B operand.
        uint32_t pb[2][2];
#pragma unroll
        for (int m = 0; m < 2; ++m) {
            float p[4] = {x[m][0], x[m][1], x[m][2], x[m][3]};
#pragma unroll
            for (int e = 0; e < 4; e += 2) {
                add2(p[e], p[e + 1], nm0, nm1);
                mul2(p[e], p[e + 1], cs0, cs1);
                p[e] = fast_exp2(p[e]);
                p[e + 1] = fast_exp2(p[e + 1]);
                add2(l0, l1, p[e], p[e + 1]);
            }
            pb[m][0] = movmatrix_t(pack_f16(p[0], p[1]));
            pb[m][1] = movmatrix_t(pack_f16(p[2], p[3]));
        }

        // V: all of it into registers, tokens interleaved, and the stage is free for its next
        // tile while they are multiplied.
        constexpr int kWords = D / 64;  // words of codes per lane and token
        uint32_t ws[4];                 // scales of the tokens of slots 2c, 2c + 1 of 8-token groups
        uint32_t ev[4][kWords], od[4][kWords];
#pragma unroll
        for (int r = 0; r < 4; ++r) {
            const uint8_t *row = buf + kTile + codes_at(r) + g * (D / 16);
            const uint8_t *scl = buf + kTile + scales_at(r) + (D == 128 ? g : g >> 1);
            const uint32_t s0 = scl[tok_v0 * kScRow], s1 = scl[tok_v1 * kScRow];
            ws[r] = e4m3x2_to_f16x2(prmt(s0, s1, 0x0040u));
            uint32_t u[kWords], v[kWords];
            if constexpr (D == 128) {
                const uint2 y = *reinterpret_cast<const uint2 *>(row + tok_v0 * kRow);
                const uint2 z = *reinterpret_cast<const uint2 *>(row + tok_v1 * kRow);
                u[0] = y.x;
                u[1] = y.y;
                v[0] = z.x;
                v[1] = z.y;
            } else {
                u[0] = *reinterpret_cast<const uint32_t *>(row + tok_v0 * kRow);
                v[0] = *reinterpret_cast<const uint32_t *>(row + tok_v1 * kRow);
            }
#pragma unroll
            for (int k = 0; k < kWords; ++k) {
                ev[r][k] = (u[k] & 0x0f0f0f0fu) | ((v[k] << 4) & 0xf0f0f0f0u);
                od[r][k] = ((u[k] >> 4) & 0x0f0f0f0fu) | (v[k] & 0xf0f0f0f0u);
            }
        }
        __syncwarp();
        issue(i + S, st);
#pragma unroll
        for (int m = 0; m < 2; ++m) {
#pragma unroll
            for (int k = 0; k < kWords; ++k) {
                uint32_t f[4][4];
                e2m1x8_to_f16x8(ev[2 * m][k], f[0]);
                e2m1x8_to_f16x8(od[2 * m][k], f[1]);
                e2m1x8_to_f16x8(ev[2 * m + 1][k], f[2]);
                e2m1x8_to_f16x8(od[2 * m + 1][k], f[3]);
#pragma unroll
                for (int e = 0; e < 4; ++e) {
                    const uint32_t p[4] = {hmul2_u32(f[0][e], ws[2 * m]),
                                           hmul2_u32(f[1][e], ws[2 * m]),
                                           hmul2_u32(f[2][e], ws[2 * m + 1]),
                                           hmul2_u32(f[3][e], ws[2 * m + 1])};
                    mma_f16(acc[4 * k + e], p, pb[m][0], pb[m][1]);
                }
            }
        }

        const bool last = d.y & kLast;
        if (last || i == n - 1) {
#pragma unroll
            for (int o = 4; o < 32; o <<= 1) {
                l0 += __shfl_xor_sync(0xffffffffu, l0, o);
                l1 += __shfl_xor_sync(0xffffffffu, l1, o);
            }
            if (!inside && last) {
                __nv_bfloat16 *row =
                    a.out + ((size_t)(seg >> 8) * a.num_heads + (seg & 255) * G + 2 * c) * D +
                    g * (D / 8);
                if (2 * c < G) store_rows<D>(row, acc, 0, l0, a.v_scale);
                if (2 * c + 1 < G) store_rows<D>(row + D, acc, 1, l1, a.v_scale);
            } else if (inside) {
                store_rec<D>(recs + warp * kRec, acc, lane, -nm0 * (cs0 * kRecUnit), l0,
                             -nm1 * (cs1 * kRecUnit), l1);
                if (lane == 0) {
                    pieces[warp].a = 1;
                    pieces[warp].a_ends = last;
                }
            } else {  // the range's last tile: the ring is empty
                store_rec<D>(reinterpret_cast<float *>(stages), acc, lane, -nm0 * (cs0 * kRecUnit),
                             l0, -nm1 * (cs1 * kRecUnit), l1);
                if (lane == 0) {
                    pieces[warp].b = 1;
                    pieces[warp].b_seg = seg;
                }
            }
            seg = -1;
        }
    };
    if constexpr (S == 2) {  // (a stage's addresses are constants then)
        for (int i = 0; i < n; i += 2) {
            step(i, 0);
            if (i + 1 < n) step(i + 1, 1);
        }
    } else {
        for (int i = 0, st = 0; i < n; ++i, st = st + 1 == S ? 0 : st + 1) step(i, st);
    }

    // The pieces of segments that span warps, a group of them per warp in which such a segment
    // began and one for the segment that began before the CTA's range: a warp per group and
    // two heads.  (Mostly the latency of few instructions, fetched for the first time: 2.2 us at
    // 16 groups of 4 heads one by one, 1.7 so; four heads at once 0.5 faster there, as much slower
    // for the one segment of a short context.)
    __syncthreads();
    const WarpPieces lp = lane < kWarps ? pieces[lane] : WarpPieces{0, 0, 0, 0};
    const uint32_t through = __ballot_sync(0xffffffffu, lp.a && !lp.a_ends);  // a whole range
    const uint32_t ending = __ballot_sync(0xffffffffu, lp.a_ends);
    const uint32_t begun = __ballot_sync(0xffffffffu, lp.b);
    // The last warp of the pieces that follow warp e - 1's, and whether the segment ends there.
    auto follow = [&](int e, bool &ends) {
        while (through >> e & 1) ++e;
        ends = ending >> e & 1;
        return ends ? e : e - 1;
    };
    constexpr int kTogether = 2;
    const int groups = __popc(begun) + pieces[0].a, parts = (G + kTogether - 1) / kTogether;
    for (int item = warp; item < groups * parts; item += kWarps) {
        // Of an odd group's last part the second head is the first again.
        const int hd = item % parts * kTogether, next = hd + kTogether <= G ? 1 : 0;
        int nth = item / parts;
        const bool head = nth == __popc(begun);
        uint32_t left = begun;
        for (; nth > 0 && left; --nth) left &= left - 1;
        const int w = head ? 0 : __ffs(left) - 1;  // the first piece's warp
        bool ends;
        const int e = follow(head ? 0 : w + 1, ends), np = e - w + 1;
        auto rec_of = [&](int k) {  // piece k
            return k == 0 && !head ? reinterpret_cast<const float *>(ring + w * S * kStage)
                                   : recs + (w + k) * kRec;
        };
        float M[kTogether], den[kTogether];
        constexpr int E = D / 32;  // consecutive dims of a lane
        using Dims = std::conditional_t<D == 128, float4, float2>;
        float num[kTogether][E];
#pragma unroll
        for (int u = 0; u < kTogether; ++u) {
            M[u] = kLowest;
            den[u] = 0.f;
#pragma unroll
            for (int j = 0; j < E; ++j) num[u][j] = 0.f;
        }
#pragma unroll 2
        for (int k = 0; k < np; ++k) {
            const float *r = rec_of(k) + kHeads * D;
#pragma unroll
            for (int u = 0; u < kTogether; ++u) M[u] = fmaxf(M[u], r[2 * (hd + u * next)]);
        }
#pragma unroll 2
        for (int k = 0; k < np; ++k) {
            const float *r = rec_of(k);
#pragma unroll
            for (int u = 0; u < kTogether; ++u) {
                const int at = hd + u * next;
                const float2 ml = *reinterpret_cast<const float2 *>(r + kHeads * D + 2 * at);
                const Dims v = *reinterpret_cast<const Dims *>(r + at * D + lane * E);
                const float f = fast_exp2((ml.x - M[u]) * kPerRecUnit);
                den[u] += f * ml.y;
#pragma unroll
                for (int j = 0; j < E; ++j) num[u][j] += f * reinterpret_cast<const float *>(&v)[j];
            }
        }
        const int sg = pieces[w].b_seg;
#pragma unroll
        for (int u = 0; u < kTogether; ++u) {
            const int at = hd + u * next;
            if (!head && ends) {
                const float inv = 1.f / den[u];
                uint32_t *row = reinterpret_cast<uint32_t *>(
                    a.out + ((size_t)(sg >> 8) * a.num_heads + (sg & 255) * G + at) * D +
                    lane * E);
#pragma unroll
                for (int j = 0; j < E; j += 2)
                    row[j / 2] = pack_bf16(num[u][j] * inv * a.v_scale,
                                           num[u][j + 1] * inv * a.v_scale);
            } else {
                float *r = a.recs + ((size_t)blockIdx.x * 2 + (head ? 0 : 1)) * kRec;
                Dims v;
#pragma unroll
                for (int j = 0; j < E; ++j) reinterpret_cast<float *>(&v)[j] = num[u][j];
                *reinterpret_cast<Dims *>(r + at * D + lane * E) = v;
                if (lane == 0)
                    *reinterpret_cast<float2 *>(r + kHeads * D + 2 * at) =
                        make_float2(M[u], den[u]);
            }
        }
    }
    if (!a.whole && tid == 0) {
        bool head_ends = false, tail_ends = true;
        follow(0, head_ends);
        const int w = 31 - __clz(begun);  // the one piece that may leave the CTA begins here
        if (begun) follow(w + 1, tail_ends);
        a.meta[blockIdx.x] = make_int4(lp.a, head_ends, !tail_ends,
                                       begun ? pieces[w].b_seg : 0);
    }
}

// Block i merges the segment that begins in CTA i and goes on: CTA i's record at its end, then
// the next CTAs' at their starts, up to the one in which it ends.  A thread per head and four
// dims.  The first two pieces are requested before it is known whether there are any (0.5 us),
// more of them eight at once.
template <int D>
__global__ void __launch_bounds__(kHeads * D / 4) decode_fp4_merge_kernel(const Args a, int ctas) {
    pdl_begin();
    constexpr int kRec = kRecFloats<D>, kThreads = kHeads * D / 4, kBatch = 8;
    __shared__ int s_last;
    const int i = blockIdx.x, tid = threadIdx.x, G = a.group;
    const int hd = tid * 4 / D, dim = tid * 4 % D;
    auto rec_of = [&](int p) {
        return a.recs + (p == 0 ? (size_t)i * 2 + 1 : (size_t)(i + p) * 2) * kRec;
    };
    if (tid == 0) s_last = ctas - 1;
    const int4 mine = a.meta[i];
    float2 ml[kBatch];
    float4 v[kBatch];
    auto request = [&](int k, int p) {
        ml[k] = *reinterpret_cast<const float2 *>(rec_of(p) + kHeads * D + 2 * hd);
        v[k] = *reinterpret_cast<const float4 *>(rec_of(p) + hd * D + dim);
    };
    request(0, 0);
    request(1, i + 1 < ctas ? 1 : 0);
    int stop = ctas - 1;  // of the CTAs that this thread looks at, the first to end the segment
    for (int k = i + 1 + tid; k < ctas; k += kThreads) {
        const int2 m = *reinterpret_cast<const int2 *>(a.meta + k);
        if (!m.x || m.y) stop = min(stop, m.x ? k : k - 1);
    }
    __syncthreads();
    if (!mine.z) return;
    if (stop < ctas - 1) atomicMin(&s_last, stop);
    __syncthreads();
    const int np = s_last - i + 1;
    if (hd >= G) return;
    float M = kLowest, den = 0.f;
    float4 num = make_float4(0.f, 0.f, 0.f, 0.f);
    auto add = [&](int count) {
        float m = M;
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (k < count) m = fmaxf(m, ml[k].x);
        const float back = fast_exp2((M - m) * kPerRecUnit);
        M = m;
        den *= back;
        num.x *= back;
        num.y *= back;
        num.z *= back;
        num.w *= back;
#pragma unroll
        for (int k = 0; k < kBatch; ++k) {
            if (k >= count) continue;
            const float f = fast_exp2((ml[k].x - m) * kPerRecUnit);
            den += f * ml[k].y;
            num.x += f * v[k].x;
            num.y += f * v[k].y;
            num.z += f * v[k].z;
            num.w += f * v[k].w;
        }
    };
    add(min(np, 2));
    for (int p0 = 2; p0 < np; p0 += kBatch) {
#pragma unroll
        for (int k = 0; k < kBatch; ++k)
            if (p0 + k < np) request(k, p0 + k);
        add(np - p0);
    }
    const float f = 1.f / den;
    *reinterpret_cast<uint2 *>(
        a.out + ((size_t)(mine.w >> 8) * a.num_heads + (mine.w & 255) * G + hd) * D + dim) =
        make_uint2(pack_bf16(num.x * f * a.v_scale, num.y * f * a.v_scale),
                   pack_bf16(num.z * f * a.v_scale, num.w * f * a.v_scale));
}

template <int D, int BS>
size_t smem_bytes(int stages, int num_seqs) {
    return (size_t)kWarps * (stages * kStageBytes<D> + kRecFloats<D> * 4 + 32 * kEntryInts<BS> * 4 +
                             sizeof(WarpPieces) + 4) +
           ((size_t)num_seqs * 2 + 1) * 4;
}

constexpr size_t kSmemMax = 232448;

template <int D>
int max_seqs(int block_size) {
    const size_t rest = block_size == 8 ? smem_bytes<D, 8>(1, 0) : smem_bytes<D, 16>(1, 0);
    return (int)((kSmemMax - rest) / 8);
}

template <int D, int BS, int S>
cudaError_t launch_stages(const Args &a, int grid, cudaStream_t stream) {
    const size_t smem = smem_bytes<D, BS>(S, a.aligned ? 0 : a.num_seqs);
    const cudaError_t e = ensure_smem<decode_fp4_kernel<D, BS, S>>(smem);
    if (e != cudaSuccess) return e;
    return launch_pdl(decode_fp4_kernel<D, BS, S>, dim3((unsigned)grid), kWarps * 32, smem, 1,
                      stream, a);
}

template <int D, int BS>
cudaError_t launch(const Args &a, int grid, cudaStream_t stream) {
    g_launched.store(true);
    const bool room =
        smem_bytes<D, BS>(kMaxStages<D>, a.aligned ? 0 : a.num_seqs) <= kSmemMax;
    const cudaError_t e = room ? launch_stages<D, BS, kMaxStages<D>>(a, grid, stream)
                               : launch_stages<D, BS, 1>(a, grid, stream);
    if (e != cudaSuccess || a.whole) return e;
    return launch_pdl(decode_fp4_merge_kernel<D>, dim3((unsigned)grid), kHeads * D / 4, 0, 1,
                      stream, a, grid);
}

}  // namespace

cudaError_t take_error_decode_fp4(unsigned *bits) {
    return take_error_word(g_launched, g_err_decode_fp4, bits);
}

size_t decode_fp4_workspace_bytes(int head_size, int sm_count) {
    return (size_t)sm_count * (2 * kHeads * (head_size + 2) * 4 + sizeof(int4));
}

int decode_fp4_max_seqs(int head_size, int block_size) {
    return head_size == 128 ? max_seqs<128>(block_size) : max_seqs<64>(block_size);
}

// Whether every segment (of up to `tiles` tiles) gets a CTA of its own: no scan of the lengths, no
// second kernel, but a segment has one SM's rate, 0.1 us a tile (0.06 at head size 64), where the
// split has a share of all SMs, costs some 2 us and grows with the tiles of all segments.  Equal where
// tiles * (5/8 SMs - segments) = slope * SMs; up to 8 segments later, as the second kernel is slow
// over many pieces.  Nowhere above 4096 tokens: one long sequence among short ones would have the one
// SM.  Measured (us, CTA per segment / split, by segments and tokens; the border lies between):
//   head size 128:  2: 1280 9.3/9.1, 1536 10.2/10.1   4: 1280 9.3/9.8, 1792 10.9/10.9
//     8: 1024 8.7/9.1, 1152 9.1/8.6   16: 768 8.0/8.1, 896 8.3/7.9   32: 768 8.0/8.1, 896 8.4/8.3
//     48: 1024 9.0/9.0, 1152 9.5/9.4   72: 2048 12.5/13.8, 4096 19.1/17.4   144: 4096 20.7/23.4
//   head size 64:  1: 2560 9.6/11.9, 4096 12.6/15.2   4: 2048 8.5/9.7, 2560 9.5/8.9
//     8: 1536 7.6/7.9, 1792 8.1/7.6   16: 1152 7.1/7.0, 1280 7.3/6.9   32: 1280 7.3/7.6, 1536 7.8/7.8
//     48: 2048 8.9/9.2, 2560 9.9/9.4   72: 2560 9.9/10.4, 4096 13.5/13.2   144: 4096 14.9/17.7
static bool cta_per_segment(long long segs, long long tiles, int sms, int head_size) {
    const bool wide = head_size == 128;
    if (segs > sms || tiles > 128) return false;
    if (segs <= 4) return tiles <= (wide ? 44 : 144 - 18 * segs);
    if (segs <= 8) return tiles <= (wide ? 33 : 50);
    return tiles <= 24 || tiles * (5 * sms - 8 * segs) <= 8LL * (wide ? 11 : 19) * sms;
}

cudaError_t launch_decode_fp4(void *out, const void *q, const void *kv_cache, const KvGeom &g,
                              int num_heads, const int32_t *block_tables, int max_blocks_per_seq,
                              const int32_t *seq_lens, int num_seqs, int max_seq_len, float scale,
                              float k_scale, float v_scale, void *workspace,
                              cudaStream_t stream) {
    const int sms = device_sm_count();
    Args a;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.kv = static_cast<const uint8_t *>(kv_cache);
    a.block_tables = block_tables;
    a.seq_lens = seq_lens;
    a.recs = static_cast<float *>(workspace);
    a.meta = reinterpret_cast<int4 *>(a.recs + (size_t)sms * 2 * kHeads * (g.head_size + 2));
    a.num_seqs = num_seqs;
    a.num_heads = num_heads;
    a.num_kv_heads = g.num_kv_heads;
    a.group = num_heads / g.num_kv_heads;
    a.max_blocks = max_blocks_per_seq;
    a.num_blocks = g.num_blocks;
    a.max_seq_len = max_seq_len;
    a.factor = (float)std::frexp((double)scale * 1.4426950408889634 * k_scale, &a.factor_exp);
    a.v_scale = v_scale;
    const long long segs = (long long)num_seqs * g.num_kv_heads;
    const long long tiles = (max_seq_len + (long long)kTokens - 1) / kTokens;
    a.aligned = cta_per_segment(segs, tiles, sms, g.head_size);
    // More segments than SMs: whole segments to a CTA, by the prefix sums, spare the second kernel
    // and cost up to half a segment of imbalance.  160 segments of one length, whole / split:
    // 9.9 / 11.3 us at 512 tokens, 11.7 / 11.6 at 768, 12.6 / 12.0 at 896 (head size 64: 7.7 / 9.1,
    // 8.8 / 9.2, 9.4 / 9.4); 376 of any length up to 512, 768, 1024: 10.3 / 11.4, 12.1 / 12.3, 15.0 /
    // 14.7 (8.2 / 9.2, 9.1 / 9.6, 10.4 / 10.4); 2048 of up to 768, 1024: 33.6 / 34.5, 38.4 / 38.7
    // (25.1 / 25.9, 28.1 / 28.3).
    a.whole = a.aligned || tiles <= 24;
    const int grid = (int)(a.aligned ? segs : std::min<long long>(sms, std::max(1LL, segs * tiles)));
    if (g.head_size == 128) {
        if (g.block_size == 8) return launch<128, 8>(a, grid, stream);
        if (g.block_size == 16) return launch<128, 16>(a, grid, stream);
        return launch<128, 32>(a, grid, stream);
    }
    if (g.block_size == 8) return launch<64, 8>(a, grid, stream);
    if (g.block_size == 16) return launch<64, 16>(a, grid, stream);
    return launch<64, 32>(a, grid, stream);
}

}  // namespace pa
