// pa_tree_verify.cu - accept drafted tokens against the target's probabilities.
//
// Per sequence a walk from the root: at the last accepted node n, r = p_n and
// Z = 1; child c (token t) is accepted when u_c q_n(t) Z < r(t), else
// r := max(r / Z - q_n, 0), Z := sum r (without draft probabilities: accepted when
// u_c Z < r(t), else r(t) := 0, Z -= r(t)).  When no child is accepted the next
// token is the smallest x with r(0) + .. + r(x) > u sum r.
//
// Bound: one row of p (and of q) per sequence for the draw, 4 or 8 bytes a token of the
// vocabulary, from HBM; with few sequences the chain of dependent steps.
//
// Split: a cluster of CTAs per sequence, each over a contiguous slice of the
// vocabulary, each warp over a contiguous part of the slice.  Warp 0 of every CTA
// makes the same walk over the tree's scalars (gathered once by 64 threads, two nodes a
// lane; children are found by ballots, and a child that is the first to be tried, or all
// children without draft probabilities, are decided at once).  Only a rejection with draft
// probabilities and the final draw touch the vocabulary, by one coalesced pass that leaves
// each warp's sum.  Where the slice fits, r and q stay in shared memory between rejections
// at a node; else r is recomputed from p and q.  CTA sums cross the cluster through
// distributed shared memory, in rank order, so every CTA continues with the same bits.  For
// the draw the CTA and the warp's part that hold the goal are scanned again.
//
// Precision: whole numbers come out, so a sum must not be off by what separates
// neighbouring tokens.  r and its sums are held as unevaluated pairs of fp32 numbers
// (a head and the rounding error of the operation before; about 48 bits an operation), since
// this GPU's 64-bit units are some 60 times slower than its 32-bit ones: one CTA of 64-bit
// sums took 1433 us where the batch's bytes take 40 (256 chains, 131072 tokens), and
// 64-bit sums across the 16 warps of each CTA alone some 2 us a pass.  A thread's sum of up
// to 512 numbers takes 64 additions to each of two accumulators, each off by at most 5 2^-48
// of it, and 12 more join the threads': below 2^-38 of the whole, at random some 2^-44.
//
// Measured (GB300): those 256 chains 53 us, 5.1 TB/s; 48 trees of 9-31 nodes with sibling
// rounds, 50021 tokens, 23-28 us; 64 trees of 33-64 proposed nodes, 131072 tokens, 19 us; one
// chain of 6, 32000 tokens, 7 us (13 000 cycles: gathers 2000, walk 1200, pass 3000, cluster
// sum 2000, draw 4500).
#include <algorithm>

#include "pa_tree.cuh"

namespace pa {
namespace {

__device__ unsigned g_err_tree_verify;
std::atomic<bool> g_launched{false};  // in this process, on any device

constexpr int kNodes = 64;
constexpr int kWarps = 16;
constexpr int kMaxCluster = 8;
// What a thread loads at once: groups of four tokens of p and q (twice as many of p alone;
// 256 chains 56.0 -> 53.5 us, 64 wide trees 22.8 -> 20.6, against eight tokens one by one),
// or of a short slice kept in shared memory tokens one by one.  (A kernel per kind of
// probabilities keeps all that in registers: 51.9 and 18.3 us, 48 trees 28 -> 24.)
constexpr int kU = 2, kS = 8;

struct VerifyArgs {
    int32_t *accepted, *num_accepted, *next;
    const float *target, *draft;
    int64_t target_stride, draft_stride;
    const int32_t *tokens;
    const float *accept_u, *sample_u;
    TreeGeom t;
    int vocab;
    int cluster;     // CTAs per sequence
    int cta_slice;   // tokens per CTA, a multiple of 32
    int warp_slice;  // tokens per warp, a multiple of 32
};

// A number held as head + tail.
struct __align__(8) Pair {
    float h, l;
};

// a + b exactly, as a pair.
__device__ __forceinline__ Pair two_sum(float a, float b) {
    const float s = __fadd_rn(a, b), bb = __fadd_rn(s, -a);
    return {s, __fadd_rn(__fadd_rn(a, -__fadd_rn(s, -bb)), __fadd_rn(b, -bb))};
}

__device__ __forceinline__ void add_to(Pair &acc, Pair x) {
    const Pair s = two_sum(acc.h, x.h);
    acc.h = s.h;
    acc.l = __fadd_rn(acc.l, __fadd_rn(s.l, x.l));
}

// The same into a thread's long sum, the tail folded into the head: a tail that only gathers
// the errors of the heads grows with every addition and loses bits of its own (256 additions
// left sums off by 2^-34).
__device__ __forceinline__ void add_long(Pair &acc, Pair x) {
    add_to(acc, x);
    const float h = __fadd_rn(acc.h, acc.l);
    acc.l = __fadd_rn(acc.l, -__fadd_rn(h, -acc.h));
    acc.h = h;
}

// Four numbers' sum, by halves: fewer additions stand behind each other than in a chain.
__device__ __forceinline__ Pair sum4(const float (&v)[4]) {
    Pair a = two_sum(v[0], v[1]);
    add_to(a, two_sum(v[2], v[3]));
    return a;
}
__device__ __forceinline__ Pair sum4(Pair (&v)[4]) {
    add_to(v[0], v[1]);
    add_to(v[2], v[3]);
    add_to(v[0], v[2]);
    return v[0];
}

// The sum over kLanes consecutive lanes (those behind them hold nothing where fewer
// than 32 are summed), the same bits in each of them.
template <int kLanes = 32>
__device__ __forceinline__ Pair warp_sum(Pair x) {
#pragma unroll
    for (int o = kLanes / 2; o > 0; o >>= 1)
        add_to(x, {__shfl_xor_sync(0xffffffffu, x.h, o), __shfl_xor_sync(0xffffffffu, x.l, o)});
    return x;
}

// h + l with |l| at most half a unit of h: such pairs compare by h, then l.
__device__ __forceinline__ Pair normal(Pair x) { return two_sum(x.h, x.l); }
__device__ __forceinline__ bool above(Pair x, Pair y) {
    return x.h > y.h || (x.h == y.h && x.l > y.l);
}

// x * y to about 47 bits.
__device__ __forceinline__ Pair times(Pair x, Pair y) {
    const float m = __fmul_rn(x.h, y.h);
    return normal({m, __fmaf_rn(x.h, y.l, __fmaf_rn(x.l, y.h, __fmaf_rn(x.h, y.h, -m)))});
}

// 1 / Z: (head, tail) of 1 / (Z 2^-e) by one Newton step from the fp32 reciprocal
// (whose error e1 it leaves squared, below 2^-46), and 2^-e in two factors.
__device__ __forceinline__ float4 reciprocal(Pair z) {
    int e;
    const float h = frexpf(z.h, &e);  // z.h = h 2^e, h in [0.5, 1)
    const int e1 = -e / 2;
    const float f1 = __int_as_float((127 + e1) << 23), f2 = __int_as_float((127 - e - e1) << 23);
    const float l = __fmul_rn(__fmul_rn(z.l, f1), f2);
    const float x = __frcp_rn(h);
    const float err = __fmaf_rn(-l, x, __fmaf_rn(-h, x, 1.f));
    return make_float4(x, __fmul_rn(x, err), f1, f2);
}

// max(p - q, 0), the difference exact (NaN stays).
__device__ __forceinline__ Pair first_residual(float p, float q) {
    const Pair r = two_sum(p, -q);
    return r.h <= 0.f ? Pair{0.f, 0.f} : r;
}

// max(r / Z - q, 0), z = reciprocal(Z).
__device__ __forceinline__ Pair next_residual(Pair r, float q, float4 z) {
    const float h = __fmul_rn(__fmul_rn(r.h, z.z), z.w), l = __fmul_rn(__fmul_rn(r.l, z.z), z.w);
    const float m = __fmul_rn(h, z.x);
    const float n = __fmaf_rn(h, z.y, __fmaf_rn(l, z.x, __fmaf_rn(h, z.x, -m)));
    const Pair d = two_sum(m, -q);
    const float e = __fadd_rn(d.l, n);
    const float s = __fadd_rn(d.h, e);
    return s <= 0.f ? Pair{0.f, 0.f} : Pair{s, __fadd_rn(e, -__fadd_rn(s, -d.h))};
}

// r at a token after nrej > 0 rejections with draft probabilities.
__device__ __forceinline__ Pair residual(float p, float q, int nrej, const float4 *zinv) {
    Pair r = first_residual(p, q);
    for (int k = 1; k < nrej && r.h != 0.f; ++k) r = next_residual(r, q, zinv[k]);
    return r;
}

// The first lane whose running sum (of the lanes' weights, >= 0) exceeds goal, with
// goal lessened by the sum before it and found set; where there is none the last lane
// with weight (-1 without any), with goal lessened by the whole.
template <int kLanes = 32>
__device__ __forceinline__ int locate(Pair mine, Pair &goal, bool &found) {
    const int lane = threadIdx.x & 31;
    Pair incl = mine;
#pragma unroll
    for (int o = 1; o < kLanes; o <<= 1) {
        const Pair u = {__shfl_up_sync(0xffffffffu, incl.h, o),
                        __shfl_up_sync(0xffffffffu, incl.l, o)};
        if (lane >= o) add_to(incl, u);
    }
    incl = normal(incl);
    const unsigned some = __ballot_sync(0xffffffffu, mine.h > 0.f);
    const unsigned over = __ballot_sync(0xffffffffu, above(incl, goal)) & some;
    found = over != 0;
    const int at = found ? __ffs((int)over) - 1 : 31 - __clz((int)some);  // clz(0) = 32
    const int upto = found ? at - 1 : kLanes - 1;
    const float h = __shfl_sync(0xffffffffu, incl.h, max(upto, 0));
    const float l = __shfl_sync(0xffffffffu, incl.l, max(upto, 0));
    if (upto >= 0) add_to(goal, {-h, -l});
    goal = normal(goal);
    return at;
}

// r[x .. x + 3], 0 outside [v0, v1); wide: r + x is 16-byte aligned.
__device__ __forceinline__ void load4(const float *r, int x, int v0, int v1, bool wide,
                                      float (&v)[4]) {
    if (wide && x >= v0 && x + 3 < v1) {
        const float4 t = *reinterpret_cast<const float4 *>(r + x);
        v[0] = t.x;
        v[1] = t.y;
        v[2] = t.z;
        v[3] = t.w;
        return;
    }
#pragma unroll
    for (int e = 0; e < 4; ++e) v[e] = x + e >= v0 && x + e < v1 ? r[x + e] : 0.f;
}

__device__ __forceinline__ uint32_t peer_addr(const void *p, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}

__device__ __forceinline__ void cluster_arrive() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_wait() {
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void cluster_sync() {
    cluster_arrive();
    cluster_wait();
}

// kDraft: with draft probabilities; kKept: r and q of the slice are kept in shared memory.
template <bool kDraft, bool kKept>
__global__ void __launch_bounds__(kWarps * 32, 32 / kWarps)
    tree_verify_kernel(const VerifyArgs a) {
    __shared__ int s_par[kNodes], s_tok[kNodes];
    __shared__ float s_p[kNodes], s_q[kNodes], s_u[kNodes];
    __shared__ float4 s_zinv[kNodes];    // 1 / Z before each rejection at the current node
    __shared__ Pair s_tot[kWarps];       // warp sums of the last pass
    __shared__ Pair s_cta[2][kMaxCluster];  // CTA sums of the cluster, by turns
    __shared__ int s_cmd[3];             // what warp 0 asks for: node, rejections, last pass
    __shared__ Pair s_goal;
    __shared__ Pair s_sub[kWarps];       // the same over the parts of the drawn warp's part
    __shared__ int s_pick;
    __shared__ float s_best[kWarps > kMaxCluster ? kWarps : kMaxCluster];
    __shared__ int s_arg[kWarps > kMaxCluster ? kWarps : kMaxCluster];
    __shared__ float s_cbest[kMaxCluster];
    __shared__ int s_carg[kMaxCluster];
    // Without draft: a bit per token of the slice.  With, where the slice fits (cached):
    // r's heads and tails, and q, after the last rejection.
    extern __shared__ uint32_t s_dyn[];
    uint32_t *s_gone = s_dyn;
    float *s_rh = reinterpret_cast<float *>(s_dyn), *s_rl = s_rh + a.cta_slice,
          *s_qc = s_rl + a.cta_slice;

    pdl_begin();
    const int C = a.cluster, s = blockIdx.x / C, rank = blockIdx.x - s * C;
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const TreeSpan span = tree_span(a.t, s);
    int32_t *path = a.accepted + (size_t)s * a.t.max_tree;
    if (span.n <= 0) {  // the same for the whole cluster
        if (rank != 0) return;
        if (span.n < 0) {
            if (tid == 0) atomicOr(&g_err_tree_verify, kErrOob);
            return;
        }
        for (int i = tid; i < a.t.max_tree; i += blockDim.x) path[i] = -1;
        if (tid == 0) {
            a.num_accepted[s] = 0;
            a.next[s] = -1;
        }
        return;
    }
    // A CTA's shared memory may be written by its peers once it has started: every CTA says so
    // here, and waits for the others before its first store to them (a pass later, so that the
    // gathers and the pass cover the wait).
    if (C > 1) cluster_arrive();
    bool peers = C == 1;  // the others have started
    const int n = span.n, V = a.vocab;
    constexpr bool with = kDraft;
    if (tid < kNodes) {
        int par = -1, tok = -1;
        float p = 0.f, q = 0.f, u = 0.f;
        if (tid > 0 && tid < n) {
            par = a.t.parents[span.row0 + tid];
            tok = a.tokens[span.row0 + tid];
            u = a.accept_u[span.row0 + tid];
            if (par < -1 || par >= tid) {
                if (rank == 0) atomicOr(&g_err_tree_verify, kErrOob);
                par = -1;
            }
            if (tok < 0 || tok >= V) {
                if (rank == 0) atomicOr(&g_err_tree_verify, kErrOob);
                tok = -1;
            } else if (par >= 0) {
                p = a.target[(int64_t)(span.row0 + par) * a.target_stride + tok];
                if (with) q = a.draft[(int64_t)(span.row0 + par) * a.draft_stride + tok];
            }
        }
        s_par[tid] = par;
        s_tok[tid] = tok;
        s_p[tid] = p;
        s_q[tid] = q;
        s_u[tid] = u;
    }
    const int c0 = min(V, rank * a.cta_slice), c1 = min(V, c0 + a.cta_slice);
    if (!with)
        for (int i = tid; i < (c1 - c0 + 31) / 32; i += blockDim.x) s_gone[i] = 0u;
    __syncthreads();

    const int v0 = min(c1, c0 + warp * a.warp_slice), v1 = min(c1, v0 + a.warp_slice);
    // Warp 0's walk; lane i holds nodes i and i + 32.
    int cur = 0, nrej = 0, count = 1;
    Pair mass = {1.f, 0.f};  // Z
    uint64_t todo = 0;   // children of cur still to be tried
    uint64_t ok_first = 0;  // nodes that are accepted when they are tried with Z = 1
    uint64_t twin = 0;   // nodes with an earlier sibling of the same token
    int my_par[2] = {-1, -1}, my_tok[2] = {-1, -1};
    float my_p[2] = {0.f, 0.f}, my_u[2] = {0.f, 0.f};
    auto nodes = [&](bool lo, bool hi) {
        const unsigned x = __ballot_sync(0xffffffffu, lo), y = __ballot_sync(0xffffffffu, hi);
        return (uint64_t)y << 32 | x;
    };
    auto children = [&](int node) { return nodes(my_par[0] == node, my_par[1] == node); };
    if (warp == 0) {
        bool first[2];
        for (int i = 0; i < 2; ++i) {
            my_par[i] = s_par[lane + 32 * i];
            my_tok[i] = s_tok[lane + 32 * i];
            my_p[i] = s_p[lane + 32 * i];
            my_u[i] = s_u[lane + 32 * i];
            // u q < p with the product exact (u < p without draft): its rounding error
            // decides only where the rounded product equals p.
            const float q = with ? s_q[lane + 32 * i] : 1.f;
            const float x = __fmul_rn(my_u[i], q), e = __fmaf_rn(my_u[i], q, -x);
            first[i] = x < my_p[i] || (x == my_p[i] && e < 0.f);
        }
        ok_first = nodes(first[0], first[1]);
        if (!with) {
            const unsigned key0 = (unsigned)(my_par[0] + 1) << 21 | (unsigned)(my_tok[0] + 1);
            const unsigned key1 = (unsigned)(my_par[1] + 1) << 21 | (unsigned)(my_tok[1] + 1);
            const unsigned below = (1u << lane) - 1u;
            bool t0 = __match_any_sync(0xffffffffu, key0) & below;
            bool t1 = __match_any_sync(0xffffffffu, key1) & below;
            for (int i = 0; i < 32; ++i) t1 |= __shfl_sync(0xffffffffu, key0, i) == key1;
            twin = nodes(t0, t1);
        }
        todo = children(0);
        if (rank == 0 && lane == 0) path[0] = 0;
    }
    auto row_of = [&](const float *m, int64_t stride, int node) {
        return m + (int64_t)(span.row0 + node) * stride;
    };
    // Four tokens at a time from where the row is 16-byte aligned: the first such group that
    // touches v0 (it may begin before).
    auto first4 = [&](const float *r) {
        return v0 - (int)((reinterpret_cast<uintptr_t>(r + v0) >> 2) & 3u);
    };
    auto aligned4 = [](const float *r, int x) {
        return (reinterpret_cast<uintptr_t>(r + x) & 15u) == 0;
    };
    int turn = 0, last_node = 0, last_rej = 0;
    bool have = false;  // the warp sums are those of (cur, nrej)
    Pair whole = {0.f, 0.f};
    for (;;) {
        if (warp == 0) {
            // On to the next pass: a rejection's sum, or the last one.
            bool ask = false;
            uint64_t tried = 0;  // without draft: cur's children that were tried
            while (todo && mass.h > 0.f) {
                int i = __ffsll((long long)todo) - 1;  // the child that is accepted, or -1
                if (nrej == 0) {
                    if (!((ok_first >> i) & 1ull)) i = -1;
                } else {
                    const float q = s_q[i];
                    const Pair r = residual(s_p[i], q, nrej, s_zinv);
                    const Pair need = times(times({s_u[i], 0.f}, {q, 0.f}), mass);
                    if (!above(normal(r), need)) i = -1;
                }
                if (i < 0 && with) {  // rejected: Z of the next round is a pass's sum
                    todo &= todo - 1;
                    // The first round's Z is 1.
                    if (nrej > 0 && lane == 0) s_zinv[nrej] = reciprocal(mass);
                    __syncwarp();
                    ++nrej;
                    ask = true;
                    break;
                }
                if (i < 0) {
                    // The first child is rejected: the others at once, Z before each from
                    // the running sum of the probabilities before it.
                    Pair sum[2];
                    float own[2];
                    for (int k = 0; k < 2; ++k) {
                        const bool in = (todo >> (lane + 32 * k)) & 1ull;
                        const bool gone = (twin >> (lane + 32 * k)) & 1ull;
                        own[k] = in && !gone ? my_p[k] : 0.f;
                        sum[k] = {own[k], 0.f};
#pragma unroll
                        for (int o = 1; o < 32; o <<= 1) {
                            const Pair u = {__shfl_up_sync(0xffffffffu, sum[k].h, o),
                                            __shfl_up_sync(0xffffffffu, sum[k].l, o)};
                            if (lane >= o) add_to(sum[k], u);
                        }
                    }
                    add_to(sum[1], {__shfl_sync(0xffffffffu, sum[0].h, 31),
                                    __shfl_sync(0xffffffffu, sum[0].l, 31)});
                    bool ok[2], may[2];
                    for (int k = 0; k < 2; ++k) {
                        Pair z = {1.f, 0.f};
                        add_to(z, {-sum[k].h, -sum[k].l});
                        add_to(z, {own[k], 0.f});
                        z = normal(z);
                        may[k] = ((todo >> (lane + 32 * k)) & 1ull) && z.h > 0.f;
                        ok[k] = may[k] && above({own[k], 0.f}, times({my_u[k], 0.f}, z));
                    }
                    const uint64_t hit = nodes(ok[0], ok[1]);
                    if (!hit) {
                        tried = nodes(may[0], may[1]);
                        break;
                    }
                    i = __ffsll((long long)hit) - 1;
                }
                if (rank == 0 && lane == 0) path[count] = i;
                ++count;
                cur = i;
                nrej = 0;
                mass = {1.f, 0.f};
                have = false;
                todo = children(i);
            }
            // The last pass: nothing to try after it.
            const bool last = !ask || !todo;
            if (last && !with) {
                for (int i = 0; i < 2; ++i) {
                    const int t = my_tok[i] - c0;
                    if (((tried >> (lane + 32 * i)) & 1ull) && my_tok[i] >= c0 && my_tok[i] < c1)
                        atomicOr(&s_gone[t >> 5], 1u << (t & 31));
                }
            }
            if (lane == 0) {
                s_cmd[0] = cur;
                s_cmd[1] = nrej;
                s_cmd[2] = (last ? 1 : 0) | (!ask && have ? 2 : 0);
            }
        }
        __syncthreads();
        const int node = s_cmd[0], rej = s_cmd[1], flags = s_cmd[2];
        last_node = node;
        last_rej = rej;
        if (!(flags & 2)) {
            const float *p = row_of(a.target, a.target_stride, node);
            const float *q = with ? row_of(a.draft, a.draft_stride, node) : p;
            // Every load of a step is issued before the first is used; what lies past the
            // warp's part counts as p = q = 0, which leaves r = 0.
            Pair acc[2] = {};
            if (with && rej > 1 && kKept) {
                // A thread's tokens are the same in every pass.
                for (int i = v0 + lane - c0; i < v1 - c0; i += 32) {
                    const Pair r = next_residual({s_rh[i], s_rl[i]}, s_qc[i], s_zinv[rej - 1]);
                    s_rh[i] = r.h;
                    s_rl[i] = r.l;
                    add_long(acc[0], r);
                }
            } else if (with && rej > 0 && kKept) {
                // A short slice: one token per lane, so that r's places lie side by side.
                for (int x = v0 + lane; x < v1; x += 32 * kS) {
                    float pv[kS], qv[kS];
#pragma unroll
                    for (int k = 0; k < kS; ++k) {
                        pv[k] = x + 32 * k < v1 ? p[x + 32 * k] : 0.f;
                        qv[k] = x + 32 * k < v1 ? q[x + 32 * k] : 0.f;
                    }
#pragma unroll
                    for (int k = 0; k < kS; ++k) {
                        const Pair r = first_residual(pv[k], qv[k]);
                        if (x + 32 * k < v1) {
                            s_rh[x + 32 * k - c0] = r.h;
                            s_rl[x + 32 * k - c0] = r.l;
                            s_qc[x + 32 * k - c0] = qv[k];
                        }
                        add_long(acc[k & 1], r);
                    }
                }
            } else if (with && rej > 0) {
                const int x0 = first4(p);
                const bool wide = aligned4(p, x0) && aligned4(q, x0);
                for (int x = x0 + 4 * lane; x < v1; x += 128 * kU) {
                    float pv[kU][4], qv[kU][4];
#pragma unroll
                    for (int k = 0; k < kU; ++k) {
                        load4(p, x + 128 * k, v0, v1, wide, pv[k]);
                        load4(q, x + 128 * k, v0, v1, wide, qv[k]);
                    }
#pragma unroll
                    for (int k = 0; k < kU; ++k) {
                        Pair r[4];
#pragma unroll
                        for (int e = 0; e < 4; ++e)
                            r[e] = residual(pv[k][e], qv[k][e], rej, s_zinv);
                        add_long(acc[k & 1], sum4(r));
                    }
                }
            } else {
                const int x0 = first4(p);
                const bool wide = aligned4(p, x0);
                for (int x = x0 + 4 * lane; x < v1; x += 128 * 2 * kU) {
                    float pv[2 * kU][4];
#pragma unroll
                    for (int k = 0; k < 2 * kU; ++k)
                        load4(p, x + 128 * k, v0, v1, wide, pv[k]);
#pragma unroll
                    for (int k = 0; k < 2 * kU; ++k) {
#pragma unroll
                        for (int e = 0; e < 4; ++e) {
                            const int y = x + 128 * k + e, b = y - c0;
                            if (!with && y >= v0 && y < v1 && ((s_gone[b >> 5] >> (b & 31)) & 1u))
                                pv[k][e] = 0.f;
                        }
                        add_long(acc[k & 1], sum4(pv[k]));
                    }
                }
            }
            add_to(acc[0], acc[1]);
            const Pair t = warp_sum(acc[0]);
            if (lane == 0) s_tot[warp] = t;
            __syncthreads();
            if (!peers) cluster_wait();
            peers = true;
            if (warp == 0) {
                // This CTA's sum to every CTA of the cluster.
                const Pair sum =
                    warp_sum<kWarps>(lane < kWarps ? s_tot[lane] : Pair{0.f, 0.f});
                if (lane < C)
                    asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(
                                     peer_addr(&s_cta[turn][rank], lane)),
                                 "f"(sum.h), "f"(sum.l)
                                 : "memory");
            }
            __syncwarp();
            if (C > 1)
                cluster_sync();
            else
                __syncthreads();
            if (warp == 0) {
                whole = normal(warp_sum<kMaxCluster>(lane < C ? s_cta[turn][lane]
                                                              : Pair{0.f, 0.f}));
                whole.h = __shfl_sync(0xffffffffu, whole.h, 0);
                whole.l = __shfl_sync(0xffffffffu, whole.l, 0);
                mass = whole;
                have = true;
            }
            turn ^= 1;
        }
        if (flags & 1) break;
    }
    // The next token.
    if (warp == 0) {
        if (rank == 0) {
            for (int i = count + lane; i < a.t.max_tree; i += 32) path[i] = -1;
            if (lane == 0) a.num_accepted[s] = count;
        }
        // The CTA, and there the warp, that holds the goal u * whole; where rounding leaves
        // none (or sample_u >= 1) the last with weight, to the last token with weight.
        const float u = a.sample_u[s];
        Pair goal = times({u, 0.f}, whole);
        bool found;
        const int pick = locate<kMaxCluster>(
            lane < C ? s_cta[turn ^ 1][lane] : Pair{0.f, 0.f}, goal, found);
        int w_pick = pick < 0 ? -2 : -1;
        if (pick == rank) {
            if (!found) goal = {INFINITY, 0.f};
            w_pick = locate<kWarps>(lane < kWarps ? s_tot[lane] : Pair{0.f, 0.f}, goal, found);
            if (!found) goal = {INFINITY, 0.f};
        }
        if (lane == 0) {
            s_goal = goal;
            s_pick = w_pick;
        }
    }
    __syncthreads();
    const float *p = row_of(a.target, a.target_stride, last_node);
    if (s_pick == -1) return;  // another CTA draws
    if (s_pick >= 0) {
        // The drawn warp's part again, shared by all warps; then the part of that which
        // holds the goal, 256 tokens at a time, eight consecutive ones per lane.
        const float *q = with ? row_of(a.draft, a.draft_stride, last_node) : p;
        const int w0 = min(c1, c0 + s_pick * a.warp_slice), w1 = min(c1, w0 + a.warp_slice);
        // (A part of at most 512 tokens is scanned by its own warp at once.)
        const bool shared = w1 - w0 > 512;
        if (!shared && warp != s_pick) return;
        const int sub = ((w1 - w0 + kWarps - 1) / kWarps + 31) / 32 * 32;
        const int y0 = shared ? min(w1, w0 + warp * sub) : w0;
        const int y1 = shared ? min(w1, y0 + sub) : w1;
        Pair goal = s_goal, acc = {0.f, 0.f};
        // r of eight tokens x0, x0 + step, ..: their p and q are loaded first.
        auto eight = [&](int x0, int step, int end, Pair (&r)[8]) {
            if (with && last_rej > 0 && kKept) {
#pragma unroll
                for (int k = 0; k < 8; ++k) {
                    const int x = x0 + k * step, i = x - c0;
                    r[k] = x < end ? Pair{s_rh[i], s_rl[i]} : Pair{0.f, 0.f};
                }
                return;
            }
            float pv[8], qv[8];
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int x = x0 + k * step;
                pv[k] = x < end ? p[x] : 0.f;
                qv[k] = with && last_rej > 0 && x < end ? q[x] : 0.f;
            }
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                const int x = x0 + k * step, i = x - c0;
                if (!with && x < end && ((s_gone[i >> 5] >> (i & 31)) & 1u)) pv[k] = 0.f;
                r[k] = with && last_rej ? residual(pv[k], qv[k], last_rej, s_zinv)
                                        : Pair{pv[k], 0.f};
            }
        };
        Pair r[8];
        bool found;
        if (shared) {
            for (int x = y0 + lane; x < y1; x += 256) {
                eight(x, 32, y1, r);
#pragma unroll
                for (int k = 0; k < 8; ++k) add_to(acc, r[k]);
                acc = normal(acc);
            }
            acc = warp_sum(acc);
            if (lane == 0) s_sub[warp] = acc;
            __syncthreads();
            const int at =
                locate<kWarps>(lane < kWarps ? s_sub[lane] : Pair{0.f, 0.f}, goal, found);
            if (warp != max(at, 0)) return;
            if (!found) goal = {INFINITY, 0.f};
        }
        int last = y0;
        for (int b = y0; b < y1; b += 256) {
            const int x = b + 8 * lane;
            eight(x, 1, y1, r);
            Pair mine = {0.f, 0.f};
#pragma unroll
            for (int k = 0; k < 8; ++k) add_to(mine, r[k]);
            const int hit = locate(mine, goal, found);
            if (hit < 0) continue;
            // In that lane: the first token past the goal, else its last with weight.
            int tok = x;
            bool done = false;
            Pair run = {0.f, 0.f};
#pragma unroll
            for (int k = 0; k < 8; ++k) {
                add_to(run, r[k]);
                if (!done && r[k].h > 0.f) {
                    tok = x + k;
                    done = found && above(normal(run), goal);
                }
            }
            last = __shfl_sync(0xffffffffu, tok, hit);
            if (found) break;
        }
        if (lane == 0) a.next[s] = min(last, V - 1);
        return;
    }
    // Nothing left to draw from: the lowest token of the largest p.
    float best = -1.f;
    int arg = 0x7fffffff;
    auto better = [](float b, int g, float &best, int &arg) {
        if (b > best || (b == best && g < arg)) {
            best = b;
            arg = g;
        }
    };
    for (int x = v0 + lane; x < v1; x += 32) better(p[x], x, best, arg);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        better(__shfl_xor_sync(0xffffffffu, best, o), __shfl_xor_sync(0xffffffffu, arg, o), best,
               arg);
    if (lane == 0) {
        s_best[warp] = best;
        s_arg[warp] = arg;
    }
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < kWarps; ++w) better(s_best[w], s_arg[w], best, arg);
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(peer_addr(&s_cbest[rank], 0)),
                     "f"(best)
                     : "memory");
        asm volatile("st.shared::cluster.u32 [%0], %1;" ::"r"(peer_addr(&s_carg[rank], 0)),
                     "r"(arg)
                     : "memory");
    }
    __syncwarp();
    if (C > 1)
        cluster_sync();
    else
        __syncthreads();
    if (rank == 0 && tid == 0) {
        for (int c = 1; c < C; ++c) better(s_cbest[c], s_carg[c], best, arg);
        a.next[s] = arg < V ? arg : 0;
    }
}

}  // namespace

cudaError_t take_error_tree_verify(unsigned *bits) {
    return take_error_word(g_launched, g_err_tree_verify, bits);
}

cudaError_t launch_tree_verify(int32_t *accepted, int32_t *num_accepted, int32_t *next_tokens,
                               const float *target, int64_t target_stride, const float *draft,
                               int64_t draft_stride, const int32_t *tokens, const TreeGeom &t,
                               int vocab, const float *accept_u, const float *sample_u,
                               cudaStream_t stream) {
    VerifyArgs a;
    a.accepted = accepted;
    a.num_accepted = num_accepted;
    a.next = next_tokens;
    a.target = target;
    a.draft = draft;
    a.target_stride = target_stride;
    a.draft_stride = draft_stride;
    a.tokens = tokens;
    a.accept_u = accept_u;
    a.sample_u = sample_u;
    a.t = t;
    a.vocab = vocab;
    // CTAs per sequence: as many as fit the GPU at once, two per SM; with draft
    // probabilities up to one and a half times that, since sequences end after very
    // different numbers of passes and the last CTAs start where others have ended (48 trees,
    // 50021 tokens, before r was kept between rejections: 41 us with 8 CTAs each, 384 of
    // which 304 fit, 63 with 4).  Each with at least 2048 tokens, and slices whose bit sets
    // fit 32 KB.
    const int sms = device_sm_count();
    const long long room = (draft ? 3LL : 2LL) * sms;
    int c = 1;
    while (c < kMaxCluster && (2LL * c * t.num_seqs <= room || vocab / c > (1 << 18)) &&
           vocab / (2 * c) >= 2048)
        c *= 2;
    a.cluster = c;
    auto up32 = [](int x) { return (x + 31) / 32 * 32; };
    a.cta_slice = up32((vocab + c - 1) / c);
    a.warp_slice = up32((a.cta_slice + kWarps - 1) / kWarps);
    // r and q in shared memory where two CTAs of that size share an SM, or one is enough
    // for the batch; else a later rejection starts again from p and q.
    const size_t keep = (size_t)a.cta_slice * 12;
    const bool kept = draft && t.max_tree > 2 &&
               (keep <= 100 << 10 || (keep <= 200 << 10 && (long long)c * t.num_seqs <= sms));
    const size_t smem = draft ? (kept ? keep : 0) : (size_t)a.cta_slice / 8;
    if (kept) {
        const cudaError_t e = ensure_smem<tree_verify_kernel<true, true>>(keep);
        if (e != cudaSuccess) return e;
    }
    g_launched.store(true);
    const dim3 grid((unsigned)(t.num_seqs * c));
    auto *kern = kept    ? tree_verify_kernel<true, true>
                 : draft ? tree_verify_kernel<true, false>
                         : tree_verify_kernel<false, false>;
    return launch_pdl(kern, grid, kWarps * 32, smem, c, stream, a);
}

}  // namespace pa
