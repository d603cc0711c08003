// pa_tree_attention.cu - attention of draft trees over a paged KV cache.
//
// Node i of a sequence's tree (n nodes behind a context of len - n tokens) attends
// to the context, to its ancestors and to itself:
//   out = sum_t softmax_t(scale q.K_t) V_t,
// computed in one pass over the keys with a running maximum m and sum l.
//
// Bound: every K and V row once per KV head, 4 Hkv D bytes a token from a bf16 pool; up to
// some 60 rows per KV head HBM binds, with more the tensor pipe.
//
// Design (tcgen05)
//   * A query tile is up to 128 rows: floor(128 / G) nodes times the G query heads
//     of one KV head, so a K/V tile of 64 keys is fetched once for all of them.
//     Trees of more rows have several row groups, whose CTAs (a team) walk the same keys
//     side by side (all but the first fetch of a tile hit L2).
//   * Work = the list of tiles over (sequence, KV head), a list per number of row groups,
//     each cut into equal contiguous ranges, one per team (Walk).  Two CTAs share an
//     SM (each with half of its shared memory and tensor memory), so that one CTA's
//     loads and products run under the other's softmax.  A segment (sequence, KV
//     head) that falls across ranges leaves its pieces' (m, l, O) in the workspace,
//     merged by log-sum-exp in a second, dependent kernel; a segment that lies in one
//     range is written at once.
//   * Warp 0 finds the range, publishes its segments to the other warps and streams K (and
//     V, or another warp does: kVWarp) through the block table, a block's rows of one head
//     per copy (its 8-row groups and 64-dim panels in one 4-D box: with a 2-D copy per
//     panel of 16 rows the copies' issue bounded the kernel at some 100 cycles each);
//     the table entries are read a tile ahead.  The segment's queries come by TMA as well,
//     those of up to 64 rows a segment ahead.
//   * Single threads issue the products: S = Q.K^T into two buffers by turns, up to two tiles
//     ahead, and O += P.V with P from tensor memory over its own scores.  A product takes
//     46 cycles (64 keys) to 64 (128 dims), a commit some 200 of its thread.
//   * The softmax warps (two for up to 64 rows, else four) hold one query row per thread:
//     softmax, P, the O rescale (rare: only when a row's maximum rises by more than 2^8), the
//     epilogue.  A warp whose 32 rows hold no query skips all that.
//   * From an FP8 pool K is multiplied as codes, the query being the sum of two e4m3
//     rows (split_q); only V is converted, to f16, by two more warps.  (Converting both
//     left the converting warps the bound: 64 sequences' chains 118 us, now 78.)
//   * Masks: a row's ancestors are a 64-bit word (pointer doubling over the parents,
//     six shuffle rounds); only tiles that reach past the context look at it.  What
//     a row does not see gets the score -inf, and V rows of tree nodes are cleared of
//     NaN and infinities before the product (0 * NaN would reach every row); the rows
//     that do see one get it added back in the epilogue.
//   * Rounding: scores, statistics and O in fp32; P to bf16 (f16 from an FP8 pool) as the
//     product's operand, the row sum from the fp32 values; the output once to bf16.
//
// Measured (GB300, HBM copy 6689 GB/s, whole call): 32 sequences of 512-4096 tokens with
// 12-16 nodes, 32 query and 8 KV heads of 128: 60 us, 5.2 TB/s; 8 sequences of 1024-131072
// tokens with 7-23 nodes: 142 us, 6.1 TB/s; 16 sequences of 1024-8192 tokens, 33-64 nodes,
// 64 and 8 heads: 130-136 us by machine, 880-910 TFLOP/s (visible pairs); the first batch's kind
// from an FP8 pool, 64 sequences, chains of 3-8: 78 us, 3.9 TB/s.  Per call some 5 us until the
// first products, 4 to 8 us for the merge.  The wide case keeps the tensor pipe 51 % busy, the
// FP8 one 41 % with DRAM at 3.9 TB/s: the chain of a tile, scores, softmax, output, scores over
// the same buffer, takes 1400 to 1800 cycles per tile and CTA, and the two CTAs of an SM do not
// fill each other's gaps entirely.  (That is some 80 us of the wide kernel's 112; beside the
// start, what the rest goes to has not been located.)  All figures here are of head size 128,
// and of an FP8 pool for up to 64 rows: the rules drawn from them hold for the others too,
// which are tested and not timed.
#include <algorithm>
#include <cmath>

#include "pa_tree.cuh"
#include "pa_tree_ring.h"

namespace pa {
namespace {

__device__ unsigned g_err_tree_attention;
std::atomic<bool> g_launched{false};  // in this process, on any device

constexpr int kRows = 128;  // query rows per tile (the MMA's M)
// Keys per K/V tile: two buffers of scores beside O fit half of tensor memory.  (One of 128
// keys makes each tile a chain scores -> softmax -> output -> scores: 60 -> 81 us.)
constexpr int kKeys = 64;
constexpr int kGroups = 4;  // row groups, at most: 64 nodes x 8 heads
constexpr int kWholeTiles = 6;  // longest segment (in tiles) that is never split
// A CTA's change to another segment (queries, epilogue) takes as long as this many
// tiles; ranges are cut with that weight when they are at least kLongRange tiles long.
constexpr int kLongRange = 12;
// The exponent's reference rises only when a score exceeds it by this (log2 units).
constexpr float kSlack = 8.0f;
constexpr uint32_t kCols = 256, kColO = 128;  // tensor memory: two S / P tiles, then O

struct TreeAttnArgs {
    __nv_bfloat16 *out;
    const __nv_bfloat16 *q;
    const void *kv;
    const int32_t *block_tables, *seq_lens;
    TreeGeom t;
    // [ctas] where each range starts: (sequence, KV head | tree nodes << 8 | row group << 16,
    // tile, first node row).
    int4 *starts;
    float *part_ml;  // [2 * ctas][part_rows][2]: m (log2 units), l
    // [2 * ctas][D / 4][part_rows][4]: a thread holds a row, so the lanes of a store (and of
    // the merge's loads) lie side by side.
    float *part_acc;
    int part_rows;
    int num_heads, num_kv_heads, group;
    int block_size, max_blocks, num_blocks, max_len;
    int q_tile;      // nodes per query tile: floor(128 / group)
    int q_recip;     // 2^16 / q_tile, rounded up
    int row_groups;  // of the largest tree
    int ctas;
    int whole_segments;  // ranges hold whole segments: nothing to merge
    int change;          // units of a change of segment
    int negate_q;
    float scale_log2;  // |scale| * log2(e), at least 1e-30
    // An FP8 pool: scale_log2 * k_scale = qk_mant 2^qk_exp, qk_mant in [0.5, 1).
    float qk_mant;
    int qk_exp;
    float v_scale;
};

// Two: queries of up to 64 rows, held twice.
template <int D, bool KV8, bool Two>
struct Tlay {
    static constexpr int kPanels = D / 64;
    static constexpr int kQPanel = kRows * 128;  // 64 dims of 128 rows
    static constexpr int kQ = kPanels * kQPanel;
    // Tiles of K and V as the products read them, in the places that the ring gives them.
    // An FP8 pool's K is read as codes; its V lands as codes and is converted.
    using Ring = TreeRing<D, KV8>;
    static constexpr int kVTile = kPanels * kKeys * 128;
    static constexpr int kKTile = KV8 ? kKeys * 128 : kVTile;
    static constexpr int kRing = Ring::kRing, kSlots = Ring::kSlots;
    static constexpr int kKSlots = Ring::kKSlots, kVSlots = Ring::kVSlots;
    static constexpr int kStages = KV8 ? 3 : 0;
    // The warp that issues the scores' products (1: the outputs' one), and the one that fetches
    // V (0: K's one).  A thread each for the products and a warp each for the copies let wide
    // bf16 trees run at 1400 cycles a tile instead of 1750.  Of up to 64 rows V stays with K
    // (32 trees of 12-16 nodes 60.2 -> 59.4 us), over an FP8 pool both do (64 chains 79 us,
    // 82 with the products and 90 with the copies apart).
    static constexpr int kScoreWarp = KV8 ? 1 : Two ? 3 : 6;
    static constexpr int kVWarp = KV8 || Two ? 0 : 7;
    static constexpr int kSplitWarp = KV8 && Two ? 2 : -1;
    static constexpr int kStage = kKeys * 128;
    // Where 8 keys x 64 dims (1 KB, swizzled) of panel p, keys 8 g .. lie in a 16-bit tile:
    // kGroup g + kPanel p.  A bf16 block lands in one copy with its panels side by side.
    static constexpr int kGroup = 1024 * kPanels;
    static constexpr int kPanel = 1024;
    static constexpr int kConv = KV8 ? 2 : 0;  // converting warps
    static constexpr int kThreads = (!KV8 && Two ? 6 : 8) * 32;
    static constexpr int kCodes =
        kQ + (KV8 ? kKSlots * kKTile + kVSlots * kVTile : kRing * kVTile);
    static constexpr int kOperands = kCodes + kStages * kStage;
    static constexpr size_t kSmem = (size_t)kOperands + 1024;  // + barriers

    // Where tile i's K and V lie: slot, how often it was filled before, byte offset.
    struct Place {
        int slot, use;
        uint32_t at;
        __device__ __forceinline__ uint32_t parity() const { return (uint32_t)use & 1u; }
    };
    static __device__ __forceinline__ Place k(int i) {
        const auto p = Ring::k(i);
        return {p.slot, p.use, (uint32_t)(kQ + p.slot * kKTile)};
    }
    static __device__ __forceinline__ Place v(int i) {
        const auto p = Ring::v(i);
        return {p.slot, p.use,
                (uint32_t)(KV8 ? kQ + kKSlots * kKTile + (p.slot - kKSlots) * kVTile
                               : kQ + p.slot * kVTile)};
    }
};

// A segment of a CTA's range: tiles [j0, j1) of KV head h of sequence s, for row group rg.
// The range ends with one of no tiles.
struct Seg {
    int s, row0, len, n_h_first;  // n | h << 8 | (the range starts in it) << 16 | rg << 17
    int j0, j1;
    __device__ __forceinline__ int n() const { return n_h_first & 255; }
    __device__ __forceinline__ int h() const { return (n_h_first >> 8) & 255; }
    __device__ __forceinline__ bool first() const { return (n_h_first >> 16) & 1; }
    __device__ __forceinline__ int rg() const { return n_h_first >> 17; }
};

// Segments in flight, at most: the producer publishes a segment when it opens the one
// before it, one tile ahead of its copies.  A copy of V waits for the output of at most
// seven tiles before, and that for every warp's P, so at most nine segments are unread.
constexpr int kSegs = 16;

// What follows the operands in shared memory.
struct Sync {
    // Per slot: its tile has arrived (of an FP8 pool's V: is converted).  Per tile i, by i % 4:
    // its scores, its output are done, and with that the slot that the product read is free.
    // (A commit costs the issuing thread some 200 cycles, as much as four products, so one
    // serves both.)
    uint64_t full[8], s_done[4], pv_done[4], staged[3], stage_free[3];
    uint64_t p_full[2], pv_issued[2];
    uint64_t q_raw[2], q_full[2], exp_read[2], o_free, sane[4], drain;
    uint64_t seg_full[kSegs];
    uint32_t tmem;
    int bad[4];
    uint8_t q_exp[kRows];  // an FP8 pool's queries: exponent + 127 of each row's scale
    Seg seg[kSegs];
};
static_assert(sizeof(Sync) <= 1024, "the barriers' room");

// Sequence s as this kernel sees it: no tiles where its data break the bounds.
struct SeqInfo {
    int row0, n, len;
    __device__ __forceinline__ int tiles() const {
        return n > 0 ? (len + kKeys - 1) / kKeys : 0;
    }
};

__device__ __forceinline__ SeqInfo seq_info(const TreeAttnArgs &a, int s, bool &bad) {
    const TreeSpan t = tree_span(a.t, s);
    const int len = a.seq_lens[s];
    bad = t.n < 0 || len < t.n || len > a.max_len;
    return bad ? SeqInfo{0, 0, 0} : SeqInfo{t.row0, t.n, len};
}

// Row groups of a tree of n <= 64 nodes (the quotient is exact for these sizes).
__device__ __forceinline__ int groups_of(const TreeAttnArgs &a, int n) {
    return ((n + a.q_tile - 1) * a.q_recip) >> 16;
}

// This CTA's range, walked by a whole warp in step: the sequences' data come 32 at a time,
// one per lane.
//
// The work of sequences with as many row groups is a list (per segment the change to it and
// its tiles), shared out evenly over teams of one CTA per row group, and the CTAs are shared
// out over those lists by their work.
template <bool Many>  // trees of several row groups
struct Walk {
    static constexpr int kG = Many ? kGroups : 1;
    int s, pre, x, end;        // sequence, units (per head) before it, position, range end
    int extra;                 // units of a segment besides its tiles
    int begin, at;             // the range's and the current segment's first position
    int base;                  // first sequence of the window, a multiple of 32
    int groups, rg;            // row groups of the sequences walked, this CTA's
    SeqInfo mine;              // sequence base + lane
    int mine_nt;               // its tiles (0: other row groups)
    int h, j0, j1, nt;         // the current segment's head, tiles [j0, j1) of nt
    SeqInfo cur;

    __device__ __forceinline__ void window(const TreeAttnArgs &a, int s0) {
        base = s0;
        const int i = s0 + (int)(threadIdx.x & 31);
        bool bad;
        mine = i < a.t.num_seqs ? seq_info(a, i, bad) : SeqInfo{0, 0, 0};
        mine_nt = !Many || groups_of(a, mine.n) == groups ? mine.tiles() : 0;
    }

    // To the range's start.  (Little code: it runs once and comes from memory each time.)
    __device__ __forceinline__ void start(const TreeAttnArgs &a) {
        const int lane = threadIdx.x & 31, Hkv = a.num_kv_heads, B = a.t.num_seqs;
        // Per number of row groups the tiles (below 2^31 with all heads) and sequences.
        int tiles[kG] = {}, seqs[kG] = {};
        bool any_bad = false;
#pragma unroll 1
        for (int i = lane; i < B; i += 64) {
            bool bad[2] = {};
            const SeqInfo x = seq_info(a, i, bad[0]);
            const SeqInfo y = i + 32 < B ? seq_info(a, i + 32, bad[1]) : SeqInfo{0, 0, 0};
            any_bad |= bad[0] || bad[1];
            const int cx = x.n ? groups_of(a, x.n) : 0, cy = y.n ? groups_of(a, y.n) : 0;
#pragma unroll
            for (int k = 0; k < kG; ++k) {
                tiles[k] += (cx == k + 1 ? x.tiles() : 0) + (cy == k + 1 ? y.tiles() : 0);
                seqs[k] += (cx == k + 1) + (cy == k + 1);
            }
        }
        if (any_bad) atomicOr(&g_err_tree_attention, kErrOob);
        long long all_tiles = 0;
#pragma unroll
        for (int k = 0; k < kG; ++k) {
            tiles[k] = __reduce_add_sync(0xffffffffu, tiles[k]);
            seqs[k] = __reduce_add_sync(0xffffffffu, seqs[k]);
            all_tiles += (long long)tiles[k] * (Hkv * (k + 1));
        }
        extra = all_tiles >= (long long)kLongRange * a.ctas ? a.change : 0;
        // This CTA's list and team.  A list gets the teams that its work comes to, rounded
        // up (a short one would else take twice as long), the longest what is left.
        int teams = a.ctas, team = blockIdx.x, total = tiles[0] + extra * seqs[0];
        groups = 1;
        rg = 0;
        if constexpr (Many) {
            int units[kGroups], n[kGroups], big = 0, rest = 0, left = a.ctas, at_cta = team;
            float all = 0.f, most = 0.f;
#pragma unroll
            for (int k = 0; k < kGroups; ++k) {
                units[k] = tiles[k] + extra * seqs[k];
                const float u = (float)units[k] * (float)(k + 1);
                if (u > most) big = k;
                most = fmaxf(most, u);
                all += u;
                rest += units[k] ? k + 1 : 0;
            }
            const float per = (float)a.ctas / all;
#pragma unroll
            for (int k = 0; k < kGroups; ++k) {
                n[k] = 0;
                if (k == big || !units[k]) continue;
                rest -= k + 1;  // one team of each list that is still to come
                n[k] = max(1, min((int)ceilf(per * (float)units[k]), (left - rest) / (k + 1)));
                left -= n[k] * (k + 1);
            }
            team = teams;  // left over
#pragma unroll
            for (int k = 0; k < kGroups; ++k) {
                if (k == big) n[k] = left / (k + 1);
                if (at_cta >= 0 && at_cta < n[k] * (k + 1)) {
                    groups = k + 1;
                    teams = n[k];
                    total = units[k];
                    team = at_cta / (k + 1);
                    rg = at_cta - team * (k + 1);
                }
                at_cta -= n[k] * (k + 1);
            }
        }
        // The first total % teams get one more.
        const int T = total * Hkv, share = T / teams, more = T - share * teams;
        begin = x = team < teams ? team * share + min(team, more) : 0;
        end = team < teams ? begin + share + (team < more ? 1 : 0) : 0;
        s = pre = base = 0;
        if (x >= end) return;
        // The sequence that holds x: its 32, itself.
#pragma unroll 1
        for (int b0 = 0; b0 < B; b0 += 32) {
            window(a, b0);
            const int units = mine_nt ? mine_nt + extra : 0;
            int incl = units;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int v = __shfl_up_sync(0xffffffffu, incl, o);
                if (lane >= o) incl += v;
            }
            const unsigned past = __ballot_sync(0xffffffffu, x < Hkv * (pre + incl));
            if (past) {
                const int at_lane = __ffs((int)past) - 1;
                s = b0 + at_lane;
                pre += __shfl_sync(0xffffffffu, incl - units, at_lane);
                return;
            }
            pre += __shfl_sync(0xffffffffu, incl, 31);
        }
        x = end;  // (not reached)
    }
    // The next segment; false at the range's end.
    __device__ __forceinline__ bool next(const TreeAttnArgs &a) {
        while (x < end) {
            if (s - base >= 32) window(a, s & ~31);
            cur.row0 = __shfl_sync(0xffffffffu, mine.row0, s - base);
            cur.n = __shfl_sync(0xffffffffu, mine.n, s - base);
            cur.len = __shfl_sync(0xffffffffu, mine.len, s - base);
            nt = __shfl_sync(0xffffffffu, mine_nt, s - base);
            const int units = nt ? nt + extra : 0;
            const int r = x - a.num_kv_heads * pre;
            if (r >= a.num_kv_heads * units) {
                pre += units;
                ++s;
                continue;
            }
            // Units [u0, u1) of the segment: first the change to it, then its tiles.  Whole
            // segments are those that start in the range.
            h = r / units;
            const int u0 = r - h * units;
            const int u1 = a.whole_segments ? units : min(units, u0 + end - x);
            at = x;
            x += u1 - u0;
            j0 = max(0, u0 - extra);
            j1 = max(0, u1 - extra);
            if (j0 < j1 && !(a.whole_segments && u0)) return true;
        }
        return false;
    }
};

__device__ __forceinline__ bool all_wait(uint64_t *bar, uint32_t parity) {
    return __all_sync(0xffffffffu, mbar_wait_bounded(bar, parity));
}

template <int D, bool KV8, bool Two>
__global__ void __launch_bounds__(Tlay<D, KV8, Two>::kThreads, 2)
    tree_attention_kernel(const __grid_constant__ CUtensorMap kv_map,
                          const __grid_constant__ CUtensorMap q_map, const TreeAttnArgs a) {
    using L = Tlay<D, KV8, Two>;
    // No static shared memory: the dynamic part then starts at the (1024-byte aligned)
    // beginning, and two CTAs' 112 KB of operands fit one SM.
    extern __shared__ __align__(1024) uint8_t smem[];
    uint8_t *sQ = smem;
    Sync &sy = *reinterpret_cast<Sync *>(smem + L::kOperands);
    if (smem_u32(smem) & 1023u) {  // the same for every thread: the swizzle needs it
        if (threadIdx.x == 0) atomicOr(&g_err_tree_attention, kErrPrecondition);
        return;
    }

    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int Hkv = a.num_kv_heads, G = a.group, QT = a.q_tile;
    // Queries of up to 64 rows are held twice, in the halves of their tile (the product
    // reads 128 rows from either: what lies behind a half comes out in rows that nobody
    // reads), and the two warps without rows load them a segment ahead.
    constexpr bool two_q = Two;
    constexpr uint32_t soft = two_q ? 2 : 4;  // softmax warps
    constexpr int s_warp = L::kScoreWarp, v_warp = L::kVWarp;

    // What needs no memory of the caller's, under the end of the launch before this one.
    if (tid == 0) {
        prefetch_tensormap(&kv_map);
        prefetch_tensormap(&q_map);
        for (int i = 0; i < L::kSlots; ++i)
            mbar_init(&sy.full[i], KV8 && i >= L::kKSlots ? L::kConv : 1);
        for (int i = 0; i < L::kStages; ++i) {
            mbar_init(&sy.staged[i], 1);
            mbar_init(&sy.stage_free[i], L::kConv);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sy.p_full[i], soft);
            mbar_init(&sy.pv_issued[i], 1);
            mbar_init(&sy.q_raw[i], 1);
            mbar_init(&sy.q_full[i], KV8 && !two_q ? soft : 1);
            mbar_init(&sy.exp_read[i], soft);
        }
        for (int i = 0; i < kSegs; ++i) mbar_init(&sy.seg_full[i], 1);
        mbar_init(&sy.o_free, soft);
        for (int i = 0; i < 4; ++i) {
            mbar_init(&sy.s_done[i], 1);
            mbar_init(&sy.pv_done[i], 1);
            mbar_init(&sy.sane[i], KV8 ? L::kConv : 1);
            sy.bad[i] = -1;
        }
        mbar_init(&sy.drain, s_warp == 1 ? 1 : 2);
        fence_barrier_init();
    }
    asm volatile("griddepcontrol.wait;" ::: "memory");
    // Tensor memory is taken after the launch before this one has ended, and the next one may
    // begin once this CTA has its own: a kernel that held some while it waits for the
    // other's end could keep the other from ever getting it.
    if (warp == 1) {
        tmem_alloc(&sy.tmem, kCols);
        tmem_relinquish();
        asm volatile("griddepcontrol.launch_dependents;" :::);
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sy.tmem;

    auto tile_wait = [&](uint64_t (&bars)[4], int i) {
        return all_wait(&bars[i & 3], (uint32_t)(i >> 2) & 1u);
    };
    // Segment k, once it is known.
    auto segment = [&](int k, Seg &g) -> bool {
        const bool ok = mbar_wait_bounded(&sy.seg_full[k % kSegs], (uint32_t)(k / kSegs) & 1u);
        g = sy.seg[k % kSegs];
        return ok;
    };

    // A segment's queries come by TMA: its nodes, the heads of its KV head, a panel of 64 dims
    // per copy.  (Rows behind the tree's are other queries: nobody reads what they give.)  One
    // thread.
    auto fetch_q = [&](const Seg &g, int b) {
        uint64_t *bar = KV8 ? &sy.q_raw[b] : &sy.q_full[b];
        mbar_arrive_expect_tx(bar, (uint32_t)(L::kPanels * a.part_rows * 128));
#pragma unroll
        for (int p = 0; p < L::kPanels; ++p)
            tma_load_3d(sQ + b * (64 * 128) + p * L::kQPanel, &q_map, bar, 64 * p, g.h() * G,
                        g.row0 + g.rg() * QT);
    };
    // K of an FP8 pool is multiplied as codes, so the query becomes the sum of two e4m3 rows:
    // scaled by the power of two that puts its largest element in [128, 256), q = hi + lo with
    // hi the nearest e4m3 number (4 significant bits of bf16's 8) and lo what is left.  That is
    // exact for elements down to 2^-9 of the largest; below, e4m3's smallest step leaves an
    // error of at most 2^-10, or 2^-17 of the largest element, no more than fp32 loses in the
    // 128-term sum.  The softmax takes the scaling back; a row with NaN or infinities becomes
    // NaN through it (exponent 255).
    //
    // Rows [first, end) of a segment's queries, in place, two at a time: a row's 256 bytes lie
    // where its two e4m3 rows will.  (Little code, since it runs once a segment and comes from
    // memory each time: unrolled eight times, with the loads, it took 15000 cycles.)
    auto split_q = [&](int b, int first, int end) {
        uint8_t *q = sQ + b * (64 * 128);
        const int c = lane & 15;
#pragma unroll 2
        for (int r = first + (lane >> 4); r < end + (lane >> 4); r += 2) {
            const uint4 v = *reinterpret_cast<const uint4 *>(
                q + (c >> 3) * L::kQPanel + r * 128 + (((c & 7) ^ (r & 7)) << 4));
            // The row's largest element, as bf16 bits without the sign.
            uint32_t top = 0u;
            auto up = [&](uint32_t x) { top = max(top, max(x & 0x7fffu, (x >> 16) & 0x7fffu)); };
            up(v.x);
            up(v.y);
            up(v.z);
            up(v.w);
#pragma unroll
            for (int o = 8; o > 0; o >>= 1)
                top = max(top, __shfl_xor_sync(0xffffffffu, top, o));
            const int ex = max(-119, min(127, top ? (int)(top >> 7) - 127 : 0));
            const float down = __uint_as_float((uint32_t)(127 + 7 - ex) << 23);
            uint32_t hi[2], lo[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                const uint32_t w0 = i ? v.z : v.x, w1 = i ? v.w : v.y;
                const float x0 = bf16_lo(w0) * down, x1 = bf16_hi(w0) * down;
                const float x2 = bf16_lo(w1) * down, x3 = bf16_hi(w1) * down;
                hi[i] = pack_e4m3x2(x0, x1) | pack_e4m3x2(x2, x3) << 16;
                uint32_t f0, f1;
                e4m3x4_to_f16x4(hi[i], f0, f1);
                lo[i] = pack_e4m3x2(x0 - f16_lo(f0), x1 - f16_hi(f0)) |
                        pack_e4m3x2(x2 - f16_lo(f1), x3 - f16_hi(f1)) << 16;
            }
            __syncwarp();  // the row is read
            uint8_t *at = q + r * 128 + (((c >> 1) ^ (r & 7)) << 4) + (c & 1) * 8;
            *reinterpret_cast<uint2 *>(at) = make_uint2(hi[0], hi[1]);
            *reinterpret_cast<uint2 *>(at + L::kQPanel) = make_uint2(lo[0], lo[1]);
            if (c == 0)
                sy.q_exp[b * 64 + r] = (uint8_t)(top >= 0x7f80u ? 255 : 127 + ex - 7);
        }
        fence_proxy_async_smem();
        __syncwarp();
    };
    auto rows_of = [&](const Seg &g) { return min(QT, g.n() - g.rg() * QT) * G; };
    // What a row's scores are multiplied with, always above zero (a hidden key's -inf stays what
    // it is).  FP8: with its own power of two too, held to the normal fp32 numbers: a smaller
    // factor than 2^-126 leaves every visible key the same weight as well.
    auto row_scale = [&](int exponent) -> float {
        if constexpr (!KV8) return a.scale_log2;
        const int e = max(-125, min(127, a.qk_exp + exponent - 127));
        return exponent == 255 ? NAN
                               : a.qk_mant * __uint_as_float((uint32_t)(e + 127) << 23);
    };

    // K and V come through the block table, a block's rows of one head per copy (a box), the
    // boxes of a tile issued by as many lanes.
    const int bs = a.block_size, bs_bits = 31 - __clz(bs), nbox = kKeys / bs;
    const uint64_t policy = policy_evict_first();
    // This lane's table entry for tile j; -1 << 30 for no box: outside the tile or past the
    // sequence.
    auto entry = [&](const int32_t *bt, int j, int len) {
        const int tok = j * kKeys + lane * bs;
        return lane < nbox && tok < len ? bt[tok >> bs_bits] : -(1 << 30);
    };
    // Its TMA row for K, wholly outside the map (zeros, nothing read) for no box or a bad
    // block id; and V's.
    auto row_of = [&](int blk, int head) {
        if (blk == -(1 << 30)) return blk;
        if (blk < 0 || blk >= a.num_blocks) {
            atomicOr(&g_err_tree_attention, kErrOob);
            return -(1 << 30);
        }
        return ((blk * 2) * Hkv + head) * bs;
    };
    auto v_row = [&](int r) { return r < -(1 << 29) ? r : r + Hkv * bs; };
    auto copy = [&](uint8_t *dst, uint64_t *bar, uint32_t bytes, int row) {
        if (lane == 0) mbar_arrive_expect_tx(bar, bytes);
        __syncwarp();
        if (lane < nbox) {
            if constexpr (KV8)
                tma_load_2d_hint(dst + lane * bs * 128, &kv_map, bar, 0, row, policy);
            else  // the pool's rows in groups of 8 (blocks are whole groups)
                tma_load_4d_hint(dst + lane * (bs / 8) * L::kGroup, &kv_map, bar, row >> 3,
                                 policy);
        }
    };
    auto read_wait = [&](typename L::Ring::After r) -> bool {
        return r.what == TreeRead::scores   ? tile_wait(sy.s_done, r.tile)
               : r.what == TreeRead::output ? tile_wait(sy.pv_done, r.tile)
                                            : true;
    };
    // K / V of tile i, once what lay in the slot before is read.
    auto load_k = [&](int i, int row) -> bool {
        const auto p = L::k(i);
        const bool ok = read_wait(L::Ring::k_after(i));
        if (ok) copy(smem + p.at, &sy.full[p.slot], (uint32_t)L::kKTile, row);
        return ok;
    };
    auto load_v = [&](int i, int row) -> bool {
        if constexpr (KV8) {
            const int st = i % L::kStages;
            if (i >= L::kStages &&
                !all_wait(&sy.stage_free[st], (uint32_t)(i / L::kStages - 1) & 1u))
                return false;
            copy(smem + L::kCodes + st * L::kStage, &sy.staged[st], (uint32_t)L::kStage, row);
            return true;
        } else {
            const auto p = L::v(i);
            const bool ok = read_wait(L::Ring::v_after(i));
            if (ok) copy(smem + p.at, &sy.full[p.slot], (uint32_t)L::kVTile, row);
            return ok;
        }
    };
    // The copies of the first n tiles have landed.
    auto land_k = [&](int n) {
        for (int i = max(0, n - L::Ring::kInFlight); i < n; ++i) {
            if constexpr (L::Ring::kKLandsByScores)
                tile_wait(sy.s_done, i);
            else
                mbar_wait_bounded(&sy.full[L::k(i).slot], L::k(i).parity());
        }
    };
    auto land_v = [&](int n) {
        for (int i = max(0, n - L::Ring::kInFlight); i < n; ++i) {
            if constexpr (KV8)
                mbar_wait_bounded(&sy.staged[i % L::kStages], (uint32_t)(i / L::kStages) & 1u);
            else
                mbar_wait_bounded(&sy.full[L::v(i).slot], L::v(i).parity());
        }
    };

    if (warp == 0) {
        // ------------------------------------------------------------ K (and the segments)
        Walk<!Two> w;  // this CTA's range
        w.start(a);
        // The walk is a segment ahead of the copies; what it finds, for every warp.
        int segs = 0;
        bool have = true;
        auto publish = [&]() {
            have = w.next(a);
            if (lane == 0) {
                const int i = segs % kSegs;
                sy.seg[i] = {w.s, w.cur.row0, w.cur.len,
                             w.cur.n | w.h << 8 | (w.at == w.begin ? 1 : 0) << 16 | w.rg << 17,
                             have ? w.j0 : 0, have ? w.j1 : 0};
                mbar_arrive(&sy.seg_full[i]);
            }
            ++segs;
        };
        // The table entries come one tile ahead of the copies: entry `blk` is tile it's.
        int j = 0, j1 = 0, head = 0, len = 0, blk = 0, blk_head = 0;
        const int32_t *bt = nullptr;
        int it = 0, prev = 0;
        bool ok = true, held = false;
        for (;;) {
            if (j == j1 && have) {
                if (segs > 0) {
                    j = w.j0;
                    j1 = w.j1;
                    head = w.h;
                    len = w.cur.len;
                    bt = a.block_tables + (size_t)w.s * a.max_blocks;
                }
                publish();
                if (segs == 1) {
                    if (lane == 0 && !a.whole_segments)
                        a.starts[blockIdx.x] =
                            have && w.at == w.begin
                                ? make_int4(w.s, w.h | w.cur.n << 8 | w.rg << 16, w.j0, w.cur.row0)
                                : make_int4(-1, 0, 0, 0);
                    continue;
                }
            }
            const bool more = j < j1;
            const int next = more ? entry(bt, j++, len) : 0;
            if (held) {
                const int row = row_of(blk, blk_head);
                if (!(ok = load_k(it, row))) break;
                // (One warp for both: V a tile behind, as the products go.)
                if (v_warp == 0 && it > 0 && !(ok = load_v(it - 1, v_row(prev)))) break;
                prev = row;
                ++it;
            }
            if (!more) break;
            held = true;
            blk = next;
            blk_head = head;
        }
        if (v_warp == 0 && ok && it > 0) ok = load_v(it - 1, v_row(prev));
        if (!ok && lane == 0) atomicOr(&g_err_tree_attention, kErrTimeout);
        // Never leave with copies in flight into this CTA's shared memory.
        land_k(it);
        if (v_warp == 0) land_v(it);
    } else if (warp == v_warp) {
        // ------------------------------------------------------------ V
        int it = 0, k = 0, j = 0, j1 = 0, head = 0, blk = 0;
        bool ok = true, held = false;
        Seg g = {};
        for (;;) {
            bool more = true;
            if (j == j1) {
                if (!(ok = __all_sync(0xffffffffu, segment(k, g)))) break;
                more = g.j0 < g.j1;
                j = g.j0;
                j1 = g.j1;
                ++k;
            }
            const int next =
                more ? entry(a.block_tables + (size_t)g.s * a.max_blocks, j++, g.len) : 0;
            if (held) {
                if (!(ok = load_v(it, v_row(row_of(blk, head))))) break;
                ++it;
            }
            if (!more) break;
            held = true;
            blk = next;
            head = g.h();
        }
        if (!ok && lane == 0) atomicOr(&g_err_tree_attention, kErrTimeout);
        land_v(it);
    } else if (warp == L::kSplitWarp) {
        // ------------------------------------------------------------ an FP8 pool's queries
        // Of up to 64 rows, once the softmax has read the exponents of the segment before the
        // last.
        bool ok = true;
        for (int k = 0;; ++k) {
            Seg g;
            const int b = k & 1;
            const uint32_t par = (uint32_t)(k >> 1) & 1u;
            if (!(ok = __all_sync(0xffffffffu, segment(k, g))) || g.j0 >= g.j1) break;
            if (k >= 2 && !(ok = all_wait(&sy.exp_read[b], par ^ 1u))) break;
            if (!(ok = all_wait(&sy.q_raw[b], par))) break;
            split_q(b, 0, rows_of(g));
            if (lane == 0) mbar_arrive(&sy.q_full[b]);
        }
        if (!ok && lane == 0) atomicOr(&g_err_tree_attention, kErrTimeout);
    } else if (warp == 1 || warp == s_warp) {
        // ------------------------------------------------------------ products
        const uint32_t idesc_s =
            KV8 ? tc_idesc_e4m3(kRows, kKeys) : tc_idesc_bf16(kRows, kKeys, 0);
        const uint32_t idesc_pv = KV8 ? tc_idesc_f16(kRows, D, 1) : tc_idesc_bf16(kRows, D, 1);
        const uint64_t q_desc = tc_desc_sw128(smem_u32(sQ), 16, 1024);
        const uint64_t k_desc = tc_desc_sw128(smem_u32(smem), 16, KV8 ? 1024 : L::kGroup);
        const uint64_t v_desc = tc_desc_sw128(smem_u32(smem), L::kPanel, L::kGroup);
        // S_i = Q.K^T into buffer i & 1, over tile i - 2's P: the product that reads it was
        // issued before (products run in the order of their issue, between two threads that
        // which the fences and the barrier give).  half: 64-row half of the query tile, in
        // units of 16 bytes.
        auto scores = [&](int i, uint32_t half) -> bool {
            const auto p = L::k(i);
            const int b = i & 1;
            if (s_warp != 1 && i >= 2 &&
                !mbar_wait_bounded(&sy.pv_issued[b], (uint32_t)(i / 2 - 1) & 1u))
                return false;
            if (!mbar_wait_bounded(&sy.full[p.slot], p.parity())) return false;
            tc_fence_after();
            const uint64_t kd = k_desc + (uint64_t)(p.at >> 4);
            if constexpr (KV8) {
                // The queries' two e4m3 parts, 32 dims at a time.
#pragma unroll
                for (int k = 0; k < 2 * (D / 32); ++k) {
                    const uint32_t ko = (k & 3) * 32;
                    tc_mma_f8_ss(tmem + b * kKeys,
                                 q_desc + half + (((k >> 2) * L::kQPanel + ko) >> 4),
                                 kd + (ko >> 4), idesc_s, k > 0 ? 1u : 0u);
                }
            } else {
#pragma unroll
                for (int k = 0; k < D / 16; ++k) {
                    const uint32_t qo = ((k >> 2) * L::kQPanel + (k & 3) * 32) >> 4;
                    const uint32_t ko = ((k >> 2) * L::kPanel + (k & 3) * 32) >> 4;
                    tc_mma_ss(tmem + b * kKeys, q_desc + half + qo, kd + ko, idesc_s,
                              k > 0 ? 1u : 0u);
                }
            }
            tc_commit(&sy.s_done[i & 3]);
            return true;
        };
        // O += P_i.V (over O's old contents for a segment's first tile).
        auto output = [&](int i, bool first) -> bool {
            const auto p = L::v(i);
            const int b = i & 1;
            if (!mbar_wait_bounded(&sy.p_full[b], (uint32_t)(i / 2) & 1u)) return false;
            if (!mbar_wait_bounded(&sy.full[p.slot], p.parity())) return false;
            tc_fence_after();
            const uint64_t vd = v_desc + (uint64_t)(p.at >> 4);
#pragma unroll
            for (int kk = 0; kk < kKeys / 16; ++kk)
                tc_mma_ts(tmem + kColO, tmem + b * kKeys + kk * 8,
                          vd + (uint64_t)((kk * 2 * L::kGroup) >> 4), idesc_pv,
                          (!first || kk > 0) ? 1u : 0u);
            if (s_warp != 1) {  // scores may be issued over P_i
                tc_fence_before();
                mbar_arrive(&sy.pv_issued[b]);
            }
            tc_commit(&sy.pv_done[i & 3]);
            return true;
        };
        // Tile i's V in keys [r0, 64), past the context: rows from r1 on (behind the sequence)
        // are zeroed, tree nodes' cleared of NaN and infinities.  True if there were any.
        auto clean = [&](int i, int r0, int r1) -> bool {
            constexpr int kC = 8 * L::kPanels, kN = 4;  // 16-byte chunks of a key; loads at once
            uint8_t *vs = smem + L::v(i).at +
                          ((lane % kC) >> 3) * L::kPanel + (lane & 7) * 16;
            auto at = [&](int r) {
                return reinterpret_cast<uint4 *>(vs + (r >> 3) * L::kGroup + (r & 7) * 128);
            };
            bool bad = false;
            for (int r = r0 + lane / kC; r < r1; r += kN * (32 / kC)) {
                uint4 v[kN];
#pragma unroll
                for (int k = 0; k < kN; ++k)
                    v[k] = r + k * (32 / kC) < r1 ? *at(r + k * (32 / kC))
                                                  : make_uint4(0, 0, 0, 0);
#pragma unroll
                for (int k = 0; k < kN; ++k) {
                    bool hit = false;
                    auto clear = [&](uint32_t x) {
                        if ((x & 0x7F80u) == 0x7F80u) {
                            x &= 0xffff0000u;
                            hit = true;
                        }
                        if ((x & 0x7F800000u) == 0x7F800000u) {
                            x &= 0x0000ffffu;
                            hit = true;
                        }
                        return x;
                    };
                    v[k].x = clear(v[k].x);
                    v[k].y = clear(v[k].y);
                    v[k].z = clear(v[k].z);
                    v[k].w = clear(v[k].w);
                    if (hit) {
                        *at(r + k * (32 / kC)) = v[k];
                        bad = true;
                    }
                }
            }
            for (int r = max(r0, r1) + lane / kC; r < kKeys; r += 32 / kC)
                *at(r) = make_uint4(0, 0, 0, 0);
            // Every lane's stores, before lane 0 issues the product that reads them (a vote
            // orders no memory).
            fence_proxy_async_smem();
            __syncwarp();
            return bad;
        };
        // Up to `last` tiles' scores, of segments up to max_seg, one thread.  It also fetches the
        // queries: with a place for two segments' in the middle of the segment
        // before, when the scores of the one before that are done, else after the segment's.
        int s_next = 0, s_left = 0, s_seg = 0;  // next tile, tiles left of its segment, segments
        int s_first = 0, q_seg = 0;             // the segment's first tile; queries fetched
        uint32_t half = 0;
        bool s_end = false;
        auto next_q = [&](int tile) -> bool {  // after that tile's scores
            Seg g;
            if (!segment(q_seg, g)) return false;
            if (g.j0 < g.j1) {
                if (tile >= 0 &&
                    !mbar_wait_bounded(&sy.s_done[tile & 3], (uint32_t)(tile >> 2) & 1u))
                    return false;
                fetch_q(g, two_q ? q_seg & 1 : 0);
            }
            ++q_seg;
            return true;
        };
        auto fill = [&](int last, int max_seg) -> bool {
            while (s_next < last && !s_end) {
                if (s_left == 0) {
                    if (s_seg > max_seg) break;
                    Seg g;
                    if (!segment(s_seg, g)) return false;
                    s_left = g.j1 - g.j0;
                    s_end = s_left == 0;
                    if (s_end) break;
                    if (q_seg == s_seg && !next_q(s_next - 1)) return false;
                    const int b = two_q ? s_seg & 1 : 0;
                    if (!mbar_wait_bounded(&sy.q_full[b],
                                           (uint32_t)(two_q ? s_seg >> 1 : s_seg) & 1u))
                        return false;
                    half = b ? 64 * 128 >> 4 : 0;
                    s_first = s_next;
                    ++s_seg;
                }
                if (!scores(s_next, half)) return false;
                ++s_next;
                --s_left;
                if (two_q && q_seg == s_seg && (s_next - s_first == 3 || s_left == 0) &&
                    !next_q(s_first - 1))
                    return false;
            }
            return true;
        };
        bool ok = true;
        if (warp != 1 && lane == 0) ok = fill(1 << 30, 1 << 30);
        // The outputs: a segment's first after the epilogue of the one before has read O.  With
        // the scores in the same thread, those come up to two tiles ahead, into the next
        // segment where its queries have a place of their own.  Of a bf16 pool the (at most
        // two) tiles that reach past the context are cleaned by the warp first.
        int it = 0;
        for (int seg = 0; ok && warp == 1; ++seg) {
            Seg g;
            if (!(ok = __all_sync(0xffffffffu, segment(seg, g)))) break;
            const int n = g.j1 - g.j0, ctx = g.len - g.n();
            if (n == 0) break;
            const int plain = KV8 ? n : min(n, max(0, ctx / kKeys - g.j0));
            auto ahead = [&](int tiles) {
                return s_warp != 1 || fill(it + tiles, seg + (two_q ? 1 : 0));
            };
            if (lane == 0) {
                ok = ahead(2) &&
                     (seg == 0 || mbar_wait_bounded(&sy.o_free, (uint32_t)(seg - 1) & 1u));
                for (int j = 0; ok && j < plain; ++j) ok = output(it + j, j == 0) && ahead(j + 3);
            }
            ok = __all_sync(0xffffffffu, ok);
            bool bad = false;
            for (int j = plain; ok && j < n; ++j) {
                const int i = it + j, k0 = (g.j0 + j) * kKeys;
                ok = all_wait(&sy.full[L::v(i).slot], L::v(i).parity());
                if (!ok) break;
                bad |= clean(i, max(ctx - k0, 0), min(g.len - k0, kKeys));
                bad = __any_sync(0xffffffffu, bad);
                if (j == n - 1 && bad && lane == 0) sy.bad[seg & 3] = seg;
                if (lane == 0) ok = output(i, j == 0) && ahead(j + 3);
                ok = __all_sync(0xffffffffu, ok);
            }
            if (!KV8 && lane == 0) mbar_arrive(&sy.sane[seg & 3]);
            it += n;
        }
        if (!ok && lane == 0) atomicOr(&g_err_tree_attention, kErrTimeout);
        if (!ok && lane == 0 && warp == s_warp && q_seg > 0) {  // queries in flight
            const int b = two_q ? (q_seg - 1) & 1 : 0;
            mbar_wait_bounded(KV8 ? &sy.q_raw[b] : &sy.q_full[b],
                              (uint32_t)(two_q ? (q_seg - 1) >> 1 : q_seg - 1) & 1u);
        }
        // Every product must be done before tensor memory is freed.
        if (lane == 0) tc_commit(&sy.drain);
        __syncwarp();
        if (warp == 1) mbar_wait_bounded(&sy.drain, 0);
    } else if (two_q && warp < 4) {
        // (Without a task.)
    } else if (warp < 6) {
        // ------------------------------------------------------------ softmax
        const int row = 32 * (warp & 3) + lane;  // TMEM lane = query row of the tile
        const uint32_t trow = tmem + ((uint32_t)(32 * (warp & 3)) << 16);
        const int r_node = row / G, r_head = row - r_node * G;
        const bool in_tile = row < QT * G;
        // Ancestors of the current sequence's nodes (lane and lane + 32), and of this row.
        int anc_seq = -1;
        uint64_t anc_lo = 0, anc_hi = 0;
        auto real_in = [&](const Seg &g) { return in_tile && g.rg() * QT + r_node < g.n(); };
        // Ancestors of every node of the current sequence: node lane in anc_lo, node
        // lane + 32 in anc_hi.  Each of six rounds joins a node's set with that of the
        // node its pointer has reached, and doubles the pointer's stride.
        auto ancestors = [&](const Seg &g) {
            if (anc_seq == g.s) return;
            anc_seq = g.s;
            int p0 = -1, p1 = -1;
            auto parent = [&](int i) {
                if (i >= g.n()) return -1;
                const int p = a.t.parents[g.row0 + i];
                if (p < -1 || p >= i) {
                    atomicOr(&g_err_tree_attention, kErrOob);
                    return -1;
                }
                return p;
            };
            p0 = parent(lane);
            p1 = parent(lane + 32);
            anc_lo = 1ull << lane;
            anc_hi = 1ull << (lane + 32);
#pragma unroll 1
            for (int k = 0; k < 6; ++k) {
                auto up = [&](int p, uint64_t &m, int &pp) {
                    const uint64_t x = __shfl_sync(0xffffffffu, anc_lo, p & 31);
                    const uint64_t y = __shfl_sync(0xffffffffu, anc_hi, p & 31);
                    const int u = __shfl_sync(0xffffffffu, p0, p & 31);
                    const int v = __shfl_sync(0xffffffffu, p1, p & 31);
                    m = p < 0 ? 0ull : (p < 32 ? x : y);
                    pp = p < 0 ? -1 : (p < 32 ? u : v);
                };
                uint64_t m0, m1;
                int q0, q1;
                up(p0, m0, q0);
                up(p1, m1, q1);
                anc_lo |= m0;
                anc_hi |= m1;
                p0 = q0;
                p1 = q1;
            }
        };
        int it = 0, seg = 0;
        Seg si;
        bool ok = __all_sync(0xffffffffu, segment(0, si));
        // More than 64 rows over an FP8 pool: a segment's queries, 32 rows per warp.
        auto queries = [&](const Seg &g, int k) -> bool {
            if (!all_wait(&sy.q_raw[0], (uint32_t)k & 1u)) return false;
            split_q(0, row - lane, min(row - lane + 32, rows_of(g)));
            if (lane == 0) mbar_arrive(&sy.q_full[0]);
            return true;
        };
        if (KV8 && !two_q && ok && si.j0 < si.j1) ok = queries(si, 0);
        while (ok && si.j0 < si.j1) {
            const int s_h = si.h(), s_n = si.n(), j0 = si.j0, j1 = si.j1, rg = si.rg();
            const bool whole = j0 == 0 && j1 * kKeys >= si.len;
            const int which = si.first() ? 0 : 1;  // record of a piece: first in the range?
            const int ctx = si.len - s_n;
            const bool real = real_in(si);
            const bool busy = __any_sync(0xffffffffu, real);
            const bool tree = j1 * kKeys > ctx;  // the piece holds tree nodes
            int exponent = 0;
            if constexpr (KV8) {
                if (two_q) {
                    const int b = seg & 1;
                    if (!(ok = all_wait(&sy.q_full[b], (uint32_t)(seg >> 1) & 1u))) break;
                    exponent = sy.q_exp[64 * b + (row & 63)];
                } else {
                    exponent = sy.q_exp[row];
                }
            }
            const float scale = row_scale(exponent);
            uint64_t anc = 0;
            if (tree) {
                ancestors(si);
                const int i = real ? rg * QT + r_node : 0;
                const uint64_t x = __shfl_sync(0xffffffffu, anc_lo, i & 31);
                const uint64_t y = __shfl_sync(0xffffffffu, anc_hi, i & 31);
                anc = i < 32 ? x : y;
            }
            // The next segment (published when this one was opened): its data come to L2.
            Seg next;
            if (!(ok = __all_sync(0xffffffffu, segment(seg + 1, next)))) break;
            const bool more = next.j0 < next.j1;
            if (!two_q && more && real_in(next)) {
                const __nv_bfloat16 *next_q =
                    a.q + ((size_t)(next.row0 + rg * QT + r_node) * a.num_heads +
                           (size_t)next.h() * G + r_head) * D;
#pragma unroll
                for (int c = 0; c < D / 64; ++c)
                    asm volatile("prefetch.global.L2 [%0];" ::"l"(next_q + 64 * c));
            }
            if (more && next.s != si.s && lane < 2)
                asm volatile("prefetch.global.L2 [%0];" ::"l"(a.t.parents + next.row0 +
                                                             min(32 * lane, next.n() - 1)));
            float m = -INFINITY, l = 0.f;
            for (int j = j0; j < j1; ++j, ++it) {
                const int b = it & 1;
                const uint32_t cs = trow + b * kKeys;  // this tile's scores, then P
                if (!(ok = tile_wait(sy.s_done, it))) break;
                tc_fence_after();
                const int k0 = j * kKeys;
                const bool past = k0 + kKeys > ctx;
                float s0 = 0.f, s1 = 0.f, s2 = 0.f, s3 = 0.f, nm = 0.f, cr = 1.f;
                bool rescale = false;
                float x[kKeys];
                // Visible keys of 32-key group g, as a bit word.
                auto seen = [&](int g) -> uint32_t {
                    const int d = ctx - k0 - 32 * g;  // context keys in or before this group
                    if (d >= 32) return 0xffffffffu;
                    if (d > 0) return ((1u << d) - 1u) | (uint32_t)(anc << d);
                    return d > -64 ? (uint32_t)(anc >> (-d)) : 0u;
                };
                auto mask = [&](float *v, int g) {
                    const uint32_t word = seen(g);
#pragma unroll
                    for (int c = 0; c < 32; ++c)
                        if (!((word >> c) & 1u)) v[c] = -INFINITY;
                };
                // 32 scores of group g to P, packed into columns 16 g ..
                auto probs = [&](const float *v, int g) {
                    uint32_t pk[16];
#pragma unroll
                    for (int c = 0; c < 16; c += 2) {
                        float t0, t1, t2, t3;
                        fma2(t0, t1, v[2 * c], v[2 * c + 1], scale, scale, nm, nm);
                        fma2(t2, t3, v[2 * c + 2], v[2 * c + 3], scale, scale, nm, nm);
                        const float p0 = fast_exp2(t0), p1 = fast_exp2(t1);
                        const float p2 = fast_exp2(t2), p3 = fast_exp2(t3);
                        add2(s0, s1, p0, p1);
                        add2(s2, s3, p2, p3);
                        pk[c] = KV8 ? pack_f16(p0, p1) : pack_bf16(p0, p1);
                        pk[c + 1] = KV8 ? pack_f16(p2, p3) : pack_bf16(p2, p3);
                    }
                    tmem_st16(cs + 16 * g, pk);
                };
                if (busy) {
                    // Row maximum of the raw scores (the scale goes into the exponent).
                    tmem_ld32(cs, *reinterpret_cast<float(*)[32]>(x));
                    tmem_ld32(cs + 32, *reinterpret_cast<float(*)[32]>(x + 32));
                    tc_wait_ld();
                    if (a.negate_q) {
#pragma unroll
                        for (int c = 0; c < kKeys; ++c) x[c] = -x[c];
                    }
                    if (past) {
                        mask(x, 0);
                        mask(x + 32, 1);
                    }
                    float mx = -INFINITY, my = -INFINITY, mz = -INFINITY, mw = -INFINITY;
#pragma unroll
                    for (int c = 0; c < kKeys; c += 8) {
                        mx = fmax3(mx, x[c], x[c + 1]);
                        my = fmax3(my, x[c + 2], x[c + 3]);
                        mz = fmax3(mz, x[c + 4], x[c + 5]);
                        mw = fmax3(mw, x[c + 6], x[c + 7]);
                    }
                    mx = fmaxf(mx, mz);
                    my = fmaxf(my, mw);
                    mx = fmaxf(mx, my) * scale;
                    const bool grow = real && mx > m + kSlack;  // (other rows hold anything)
                    rescale = __any_sync(0xffffffffu, grow);
                    if (rescale) {
                        const float mn = grow ? fmaxf(m, mx) : m;
                        cr = grow ? fast_exp2(m - mn) : 1.f;
                        l *= cr;
                        m = mn;
                    }
                    // A row that has seen no key yet keeps m = -inf and P = 0.
                    nm = m == -INFINITY ? 0.f : -m;
                    probs(x, 0);
                    probs(x + 32, 1);
                    l += (s0 + s1) + (s2 + s3);
                    if (rescale && j > j0) {
                        // The product before this one must be done; the next one waits.
                        if (!(ok = tile_wait(sy.pv_done, it - 1))) break;
                        tc_fence_after();
#pragma unroll 1
                        for (int c = 0; c < D / 32; ++c) {
                            float o[32];
                            tmem_ld32(trow + kColO + 32 * c, o);
                            tc_wait_ld();
#pragma unroll
                            for (int e = 0; e < 32; ++e) o[e] *= cr;
                            tmem_st32(trow + kColO + 32 * c,
                                      *reinterpret_cast<const uint32_t(*)[32]>(o));
                        }
                    }
                    tc_wait_st();
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&sy.p_full[b]);
            }
            if (!ok) break;
            if (KV8 && two_q) {  // (the exponents were used)
                __syncwarp();
                if (lane == 0) mbar_arrive(&sy.exp_read[seg & 1]);
            }
            // This segment's scores are all done: the next one's queries are on their way.
            if (KV8 && !two_q && more && !(ok = queries(next, seg + 1))) break;
            bool bad = false;
            if (tree) {  // NaN or infinities in the tree's V?
                if (!(ok = all_wait(&sy.sane[seg & 3], (uint32_t)(seg >> 2) & 1u))) break;
                bad = *reinterpret_cast<volatile int *>(&sy.bad[seg & 3]) == seg;
            }
            if (!(ok = tile_wait(sy.pv_done, it - 1))) break;
            tc_fence_after();
            if (busy) {
                const float vsc = KV8 ? a.v_scale : 1.f;
                const size_t rec = (size_t)blockIdx.x * 2 + which;
                const size_t orow = ((size_t)(si.row0 + rg * QT + r_node) * a.num_heads +
                                     (size_t)s_h * G + r_head) * D;
                const float mul = whole ? vsc / l : vsc;
                const uint64_t keep = policy_evict_last();
#pragma unroll 1
                for (int c = 0; c < D / 32; ++c) {
                    float o[32];
                    tmem_ld32(trow + kColO + 32 * c, o);
                    tc_wait_ld();
                    if (c == D / 32 - 1) {  // O is read
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&sy.o_free);
                    }
                    if (bad && real) {
                        // What this row sees of the values that were cleared.
                        const int32_t *bt = a.block_tables + (size_t)si.s * a.max_blocks;
                        for (int i = 0; i < s_n; ++i) {
                            const int pos = ctx + i;
                            if (!((anc >> i) & 1ull) || pos < j0 * kKeys || pos >= j1 * kKeys)
                                continue;
                            const int blk = bt[pos / a.block_size];
                            if (blk < 0 || blk >= a.num_blocks) continue;
                            const size_t v0 =
                                ((((size_t)blk * 2 + 1) * Hkv + s_h) * a.block_size +
                                 pos % a.block_size) * D + 32 * c;
                            const uint8_t *kv = reinterpret_cast<const uint8_t *>(a.kv);
#pragma unroll 1
                            for (int e = 0; e < 32; ++e) {
                                float v;
                                if constexpr (KV8)
                                    v = (kv[v0 + e] & 0x7f) == 0x7f ? NAN : 0.f;
                                else
                                    v = __bfloat162float(
                                        reinterpret_cast<const __nv_bfloat16 *>(kv)[v0 + e]);
                                if (!isfinite(v)) {
#pragma unroll
                                    for (int f = 0; f < 32; ++f)
                                        if (f == e) o[f] += v;
                                }
                            }
                        }
                    }
#pragma unroll
                    for (int e = 0; e < 32; ++e) o[e] *= mul;
                    if (real && whole) {
                        uint4 *dst = reinterpret_cast<uint4 *>(a.out + orow) + 4 * c;
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            dst[e] = make_uint4(pack_bf16(o[8 * e], o[8 * e + 1]),
                                                pack_bf16(o[8 * e + 2], o[8 * e + 3]),
                                                pack_bf16(o[8 * e + 4], o[8 * e + 5]),
                                                pack_bf16(o[8 * e + 6], o[8 * e + 7]));
                    } else if (real) {
                        float4 *dst = reinterpret_cast<float4 *>(a.part_acc) +
                                      (rec * (D / 4) + 8 * c) * a.part_rows + row;
#pragma unroll
                        for (int e = 0; e < 8; ++e)
                            st_hint(dst + e * a.part_rows,
                                    make_float4(o[4 * e], o[4 * e + 1], o[4 * e + 2],
                                                o[4 * e + 3]),
                                    keep);
                    }
                    __syncwarp();
                }
                if (real && !whole)
                    st_hint(reinterpret_cast<float2 *>(a.part_ml) + rec * a.part_rows + row,
                            make_float2(m, l), keep);
            } else if (lane == 0) {
                mbar_arrive(&sy.o_free);
            }
            ++seg;
            si = next;
        }
        if (!ok && lane == 0) atomicOr(&g_err_tree_attention, kErrTimeout);
    } else if constexpr (KV8) {
        // ------------------------------------------------------------ V: e4m3 -> f16
        // A lane converts a key's 128 codes (128B-swizzled as TMA left them) to f16 in the
        // layout a bf16 tile has.  Keys behind the sequence become zeros, NaN of tree nodes'
        // keys too.
        const int r = (warp - 6) * 32 + lane;
        auto tile = [&](int i, int key, const Seg &g, bool &bad) -> bool {
            const int ss = i % L::kStages;
            const auto p = L::v(i);
            if (!all_wait(&sy.staged[ss], (uint32_t)(i / L::kStages) & 1u)) return false;
            const uint8_t *codes = smem + L::kCodes + ss * L::kStage + r * 128;
            uint4 in[8];
#pragma unroll
            for (int c = 0; c < 8; ++c)
                in[c] = *reinterpret_cast<const uint4 *>(codes + ((c ^ (r & 7)) << 4));
            if (key >= g.len - g.n()) {
                const bool none = key >= g.len;
                auto clear = [&](uint32_t x) {
                    const uint32_t nan = ((x & 0x7f7f7f7fu) + 0x01010101u) & 0x80808080u;
                    bad |= !none && nan != 0u;
                    return none ? 0u : x & ~((nan >> 7) * 0xffu);
                };
#pragma unroll
                for (int c = 0; c < 8; ++c)
                    in[c] = make_uint4(clear(in[c].x), clear(in[c].y), clear(in[c].z),
                                       clear(in[c].w));
            }
            if (!read_wait(L::Ring::v_after(i))) return false;
            uint8_t *base = smem + p.at + (r >> 3) * L::kGroup + (r & 7) * 128;
#pragma unroll
            for (int c = 0; c < 8; ++c) {
                uint32_t f[8];
                e4m3x4_to_f16x4(in[c].x, f[0], f[1]);
                e4m3x4_to_f16x4(in[c].y, f[2], f[3]);
                e4m3x4_to_f16x4(in[c].z, f[4], f[5]);
                e4m3x4_to_f16x4(in[c].w, f[6], f[7]);
                uint8_t *dst = base + (c >> 2) * L::kPanel;
                const int ch = 2 * (c & 3);
                *reinterpret_cast<uint4 *>(dst + ((ch ^ (r & 7)) << 4)) =
                    make_uint4(f[0], f[1], f[2], f[3]);
                *reinterpret_cast<uint4 *>(dst + (((ch + 1) ^ (r & 7)) << 4)) =
                    make_uint4(f[4], f[5], f[6], f[7]);
            }
            fence_proxy_async_smem();
            __syncwarp();
            // (The stage is freed after the codes' use: freed after their loads alone, the next
            // tile's copy could overtake them.)
            if (lane == 0) {
                mbar_arrive(&sy.stage_free[ss]);
                mbar_arrive(&sy.full[p.slot]);
            }
            return true;
        };
        int it = 0;
        bool ok = true;
        for (int k = 0; ok; ++k) {
            Seg g;
            if (!(ok = __all_sync(0xffffffffu, segment(k, g))) || g.j0 >= g.j1) break;
            bool bad = false;
            for (int j = g.j0; ok && j < g.j1; ++j, ++it) ok = tile(it, j * kKeys + r, g, bad);
            if (bad) sy.bad[k & 3] = k;
            __syncwarp();
            if (lane == 0) mbar_arrive(&sy.sane[k & 3]);
        }
        if (!ok && lane == 0) atomicOr(&g_err_tree_attention, kErrTimeout);
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) {
        tc_fence_after();
        tmem_dealloc(tmem, kCols);
    }
}

// Merge the pieces of segments that were split across CTAs: a lane per row, a warp per
// D / 16 dims, joined by log-sum-exp in one pass, several pieces' loads in flight.
//
// With many segments block w looks whether CTA w's range starts inside a segment whose first
// piece is that of the team before, and takes its rows 32 at a time.  Few segments (at most a
// quarter of the CTAs) are split into many pieces: a block per segment, 32 rows and quarter of
// the dims, whose warps also share the pieces out among four groups, joined through shared
// memory (8 sequences of 1024 .. 131072 tokens, up to some 80 pieces: 143.6 -> 142.4 us for the
// whole call).
constexpr int kMergeWarps = 16, kMaxCtas = 512;

template <int D, bool kFew>
__global__ void __launch_bounds__(kMergeWarps * 32, 2) tree_merge_kernel(const TreeAttnArgs a) {
    constexpr int kUnits = D / 4 / kMergeWarps;  // float4 of a row that a thread joins
    constexpr int kSplit = kFew ? 4 : 1;         // groups of warps that share the pieces
    __shared__ int s_first, s_count;
    __shared__ float s_part[kFew ? kMergeWarps : 1][4 * kUnits + 2][32];
    __shared__ int4 s_start[kMaxCtas];
    pdl_begin();
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    // Every range's start at once: looked up one after the other they cost a memory latency
    // each.
    for (int i = threadIdx.x; i < a.ctas; i += blockDim.x) s_start[i] = a.starts[i];
    if (kFew && threadIdx.x == 0) {
        s_first = a.ctas;
        s_count = 0;
    }
    __syncthreads();
    auto start_of = [&](int i) {
        return i >= 0 && i < a.ctas ? s_start[i] : make_int4(-1, 0, 0, 0);
    };
    auto step_of = [&](int key) {  // a team's CTAs
        return a.row_groups == 1 ? 1 : max(1, groups_of(a, (key >> 8) & 255));
    };
    int w, n, key, node0, step;  // first CTA that starts inside, pieces
    bool prev_same;
    if constexpr (kFew) {
        const int rg = blockIdx.x % a.row_groups, sh = blockIdx.x / a.row_groups;
        const int seq = sh / a.num_kv_heads, head = sh - seq * a.num_kv_heads;
        for (int i = threadIdx.x; i < a.ctas; i += blockDim.x) {
            const int4 e = s_start[i];
            if (e.x == seq && (e.y & 255) == head && e.y >> 16 == rg && e.z > 0) {
                atomicMin(&s_first, i);
                atomicAdd(&s_count, 1);
            }
        }
        __syncthreads();
        if (s_count == 0) return;
        w = s_first;
        n = s_count + 1;
        const int4 st = start_of(w);
        key = st.y;
        node0 = st.w;
        step = step_of(key);
        const int4 before = start_of(w - step);
        prev_same = before.x == seq && before.y == key;
    } else {
        w = blockIdx.x;
        step = a.row_groups == 1 ? 1 : step_of(start_of(w).y);
        // The team before w's, w's and the next, one per lane.
        const int4 st = start_of(w + (lane - 1) * step);
        const int seq = __shfl_sync(0xffffffffu, st.x, 1);
        key = __shfl_sync(0xffffffffu, st.y, 1);
        node0 = __shfl_sync(0xffffffffu, st.w, 1);
        // Idle, or a segment's start.
        if (seq < 0 || __shfl_sync(0xffffffffu, st.z, 1) == 0) return;
        prev_same = __shfl_sync(0xffffffffu, st.x == seq && st.y == key, 0);
        if (prev_same && __shfl_sync(0xffffffffu, st.z, 0) > 0) return;  // an earlier one's
        n = 1;
        for (int base = w;; base += 32 * step) {
            const int4 e = start_of(base + lane * step);
            const unsigned in = __ballot_sync(0xffffffffu, e.x == seq && e.y == key);
            n += __popc(in);
            if (in != 0xffffffffu) break;
        }
    }
    const int nodes = (key >> 8) & 255, head = key & 255, rg = key >> 16;
    const int rows = min(a.q_tile, nodes - rg * a.q_tile) * a.group;
    const int unit0 = (kFew ? blockIdx.z * (kMergeWarps / kSplit) + warp % (kMergeWarps / kSplit)
                            : warp) * kUnits;
    const int first = kFew ? warp / (kMergeWarps / kSplit) : 0;
    const float2 *ml = reinterpret_cast<const float2 *>(a.part_ml);
    const float4 *acc = reinterpret_cast<const float4 *>(a.part_acc);
    for (int row0 = 32 * blockIdx.y; row0 < rows; row0 += 32 * gridDim.y) {
        const int row = min(row0 + lane, rows - 1);
        float M = -INFINITY, den = 0.f;
        float4 num[kUnits];
#pragma unroll
        for (int i = 0; i < kUnits; ++i) num[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        constexpr int kBatch = 4;
        for (int k0 = first; k0 < n; k0 += kBatch * kSplit) {
            auto at = [&](int k) { return k0 + k * kSplit; };  // the batch's k-th piece
            float2 e[kBatch];
            float4 v[kBatch][kUnits];
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                if (at(k) < n) {
                    const size_t cta = (size_t)(w + (at(k) - 1) * step);
                    const size_t rec = cta * 2 + (at(k) == 0 && !prev_same ? 1 : 0);
                    e[k] = ml[rec * a.part_rows + row];
#pragma unroll
                    for (int i = 0; i < kUnits; ++i)
                        v[k][i] = acc[(rec * (D / 4) + unit0 + i) * a.part_rows + row];
                }
            }
            // A row that sees no key of a piece has m = -inf and nothing in it.
            float mn = M;
#pragma unroll
            for (int k = 0; k < kBatch; ++k)
                if (at(k) < n) mn = fmaxf(mn, e[k].x);
            const float ref = mn == -INFINITY ? 0.f : mn, c = fast_exp2(M - ref);
            M = mn;
            den *= c;
#pragma unroll
            for (int i = 0; i < kUnits; ++i) {
                num[i].x *= c;
                num[i].y *= c;
                num[i].z *= c;
                num[i].w *= c;
            }
#pragma unroll
            for (int k = 0; k < kBatch; ++k) {
                if (at(k) >= n) break;
                const float g = fast_exp2(e[k].x - ref);
                den += g * e[k].y;
#pragma unroll
                for (int i = 0; i < kUnits; ++i) {
                    num[i].x += g * v[k][i].x;
                    num[i].y += g * v[k][i].y;
                    num[i].z += g * v[k][i].z;
                    num[i].w += g * v[k][i].w;
                }
            }
        }
        if constexpr (kFew) {
            float *own = &s_part[warp][0][lane];
            own[0] = M;
            own[32] = den;
#pragma unroll
            for (int i = 0; i < kUnits; ++i) {
                own[32 * (2 + 4 * i)] = num[i].x;
                own[32 * (3 + 4 * i)] = num[i].y;
                own[32 * (4 + 4 * i)] = num[i].z;
                own[32 * (5 + 4 * i)] = num[i].w;
            }
            __syncthreads();
            if (first != 0) continue;
#pragma unroll
            for (int p = 1; p < kSplit; ++p) {
                const float *o = &s_part[warp + p * (kMergeWarps / kSplit)][0][lane];
                const float mn = fmaxf(M, o[0]), ref = mn == -INFINITY ? 0.f : mn;
                const float c = fast_exp2(M - ref), g = fast_exp2(o[0] - ref);
                M = mn;
                den = den * c + g * o[32];
#pragma unroll
                for (int i = 0; i < kUnits; ++i) {
                    num[i].x = num[i].x * c + g * o[32 * (2 + 4 * i)];
                    num[i].y = num[i].y * c + g * o[32 * (3 + 4 * i)];
                    num[i].z = num[i].z * c + g * o[32 * (4 + 4 * i)];
                    num[i].w = num[i].w * c + g * o[32 * (5 + 4 * i)];
                }
            }
        }
        if (row0 + lane >= rows) continue;
        const float inv = 1.f / den;
        const int node = node0 + rg * a.q_tile + row / a.group;
        const size_t orow = (size_t)node * a.num_heads + (size_t)head * a.group + row % a.group;
        uint2 *dst = reinterpret_cast<uint2 *>(a.out + orow * D) + unit0;
        uint2 o[kUnits];
#pragma unroll
        for (int i = 0; i < kUnits; ++i)
            o[i] = make_uint2(pack_bf16(num[i].x * inv, num[i].y * inv),
                              pack_bf16(num[i].z * inv, num[i].w * inv));
        if constexpr (kUnits == 2)
            *reinterpret_cast<uint4 *>(dst) = make_uint4(o[0].x, o[0].y, o[1].x, o[1].y);
        else
            dst[0] = o[0];
    }
}

// Launch shape for trees of at most max_tree nodes.
struct Shape {
    int q_tile, row_groups, ctas, part_rows;
    size_t ml_off, acc_off, bytes;
};

Shape shape_of(int max_tree, int group, int head_size, int sm_count) {
    Shape s;
    s.q_tile = kRows / group;
    s.row_groups = (max_tree + s.q_tile - 1) / s.q_tile;
    // A team of every list at least, two CTAs per SM.
    s.ctas = std::min(kMaxCtas, std::max(kGroups * (kGroups + 1) / 2, 2 * sm_count));
    s.part_rows = std::min(s.q_tile, max_tree) * group;
    const size_t recs = (size_t)s.ctas * 2 * s.part_rows;
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    s.ml_off = up((size_t)s.ctas * sizeof(int4));
    s.acc_off = s.ml_off + up(recs * 8);
    s.bytes = s.acc_off + recs * head_size * 4;
    return s;
}

template <int D, bool KV8, bool Two>
cudaError_t launch_rows(const CUtensorMap &map, const CUtensorMap &q_map, const TreeAttnArgs &a,
                        cudaStream_t stream) {
    using L = Tlay<D, KV8, Two>;
    g_launched.store(true);
    cudaError_t e = ensure_smem<tree_attention_kernel<D, KV8, Two>>(L::kSmem);
    if (e != cudaSuccess) return e;
    e = launch_pdl(tree_attention_kernel<D, KV8, Two>, dim3((unsigned)a.ctas),
                   L::kThreads, L::kSmem, 1, stream, map, q_map, a);
    if (e != cudaSuccess || a.whole_segments || a.ctas < 2) return e;
    const unsigned rows = (unsigned)((a.part_rows + 31) / 32);
    const long long segments = (long long)a.t.num_seqs * a.num_kv_heads * a.row_groups;
    if (4 * segments <= a.ctas)
        return launch_pdl(tree_merge_kernel<D, true>, dim3((unsigned)segments, rows, 4),
                          kMergeWarps * 32, 0, 1, stream, a);
    return launch_pdl(tree_merge_kernel<D, false>, dim3((unsigned)a.ctas), kMergeWarps * 32, 0, 1,
                      stream, a);
}

template <int D, bool KV8>
cudaError_t launch(const CUtensorMap &map, const CUtensorMap &q_map, const TreeAttnArgs &a,
                   cudaStream_t stream) {
    return a.part_rows <= 64 ? launch_rows<D, KV8, true>(map, q_map, a, stream)
                             : launch_rows<D, KV8, false>(map, q_map, a, stream);
}

}  // namespace

cudaError_t take_error_tree_attention(unsigned *bits) {
    return take_error_word(g_launched, g_err_tree_attention, bits);
}

size_t tree_attention_workspace_bytes(int num_seqs, int max_tree, int group, int head_size,
                                      int sm_count) {
    return shape_of(max_tree, group, head_size, sm_count).bytes;
}

cudaError_t launch_tree_attention(void *out, const void *q, const TreeGeom &t,
                                  const void *kv_cache, const KvGeom &g, int num_heads,
                                  const int32_t *block_tables, int max_blocks_per_seq,
                                  const int32_t *seq_lens, int max_seq_len, float scale, bool kv8,
                                  float k_scale, float v_scale, void *workspace,
                                  cudaStream_t stream) {
    CUtensorMap map;
    if (kv8 ? !encode_kv_map_fp8(&map, kv_cache, g, g.block_size)
            : !encode_kv_map_groups(&map, kv_cache, g))
        return cudaErrorInvalidValue;
    TreeAttnArgs a;
    a.group = num_heads / g.num_kv_heads;
    const Shape sh = shape_of(t.max_tree, a.group, g.head_size, device_sm_count());
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.q = static_cast<const __nv_bfloat16 *>(q);
    a.kv = kv_cache;
    a.block_tables = block_tables;
    a.seq_lens = seq_lens;
    a.t = t;
    a.starts = reinterpret_cast<int4 *>(ws);
    a.part_ml = reinterpret_cast<float *>(ws + sh.ml_off);
    a.part_acc = reinterpret_cast<float *>(ws + sh.acc_off);
    a.part_rows = sh.part_rows;
    a.num_heads = num_heads;
    a.num_kv_heads = g.num_kv_heads;
    a.block_size = g.block_size;
    a.max_blocks = max_blocks_per_seq;
    a.num_blocks = g.num_blocks;
    a.max_len = max_seq_len;
    a.q_tile = sh.q_tile;
    a.q_recip = ((1 << 16) + sh.q_tile - 1) / sh.q_tile;
    a.row_groups = sh.row_groups;
    // No more teams than tiles.
    const long long tiles = (long long)t.num_seqs * g.num_kv_heads *
                            (((long long)max_seq_len + kKeys - 1) / kKeys);
    a.ctas = (int)std::min<long long>(sh.ctas, std::max(1LL, tiles) * sh.row_groups);
    // A positive scale is folded into the exponent; a negative one negates Q (exact),
    // zero becomes a value far too small to change any finite score.
    a.negate_q = scale < 0.f ? 1 : 0;
    a.scale_log2 = std::max(std::fabs(scale) * 1.4426950408889634f, 1e-30f);
    a.qk_mant = (float)std::frexp((double)a.scale_log2 * (double)k_scale, &a.qk_exp);
    a.v_scale = v_scale;
    // Contexts of a few tiles: a range of whole segments costs at most those tiles (about
    // 0.6 us each) and saves the merge's launch (one short sequence 9 us, 15-17 with it).
    a.whole_segments = max_seq_len <= kWholeTiles * kKeys;
    // A change costs some 7000 cycles, a tile 2400 where HBM bounds it (without: 32 sequences
    // 62.7 us, 61.2 with), 1400 to 1800 from an FP8 pool or with several row groups (without:
    // 64 FP8 chains 93 us, 79 with; 16 wide trees 151, 141).  A tile of head size 64 moves half
    // the bytes; its weight is the same here, unmeasured.
    a.change = kv8 || sh.row_groups > 1 ? 6 : 2;
    CUtensorMap q_map = {};
    if (!encode_rows_map(&q_map, q, g.head_size, num_heads, t.total_nodes, a.group,
                         sh.part_rows / a.group))
        return cudaErrorInvalidValue;
    if (kv8) return launch<128, true>(map, q_map, a, stream);
    if (g.head_size == 128) return launch<128, false>(map, q_map, a, stream);
    return launch<64, false>(map, q_map, a, stream);
}

}  // namespace pa
