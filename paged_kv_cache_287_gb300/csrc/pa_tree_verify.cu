// pa_tree_verify.cu - accept drafted tokens against the target's probabilities.
//
// Per sequence a walk from the root: at the last accepted node n, r = p_n and
// Z = 1; child c (token t) is accepted when u_c q_n(t) Z < r(t), else
// r := max(r / Z - q_n, 0), Z := sum r (without draft probabilities: accepted when
// u_c Z < r(t), else r(t) := 0, Z -= r(t)).  When no child is accepted the next
// token is the smallest x with r(0) + .. + r(x) > u sum r.
//
// Split: a cluster of CTAs per sequence, each over a contiguous slice of the
// vocabulary, each warp over a contiguous part of the slice.  Warp 0 of every CTA
// makes the same walk over the tree's scalars (gathered once by 64 threads); only a
// rejection with draft probabilities and the final draw touch the vocabulary, by one
// coalesced pass that recomputes r from p and q (nothing of the vocabulary's size is
// kept between passes: a second pass over the same rows hits L2) and leaves each
// warp's sum.  CTA sums cross the cluster through distributed shared memory, in rank
// order, so every CTA continues with the same bits.  For the draw the warp that holds
// the goal scans its own part: 32 contiguous shares, then the share that holds it.
//
// Precision: whole numbers come out, so a sum must not be off by what separates
// neighbouring tokens.  r and its sums are held as unevaluated pairs of fp32 numbers
// (a head and the rounding error of the operation before; about 48 bits), since this
// GPU's 64-bit units are some 60 times slower than its 32-bit ones: one CTA of 64-bit
// sums took 1433 us where the batch's bytes take 40 (256 chains, 131072 tokens).
#include <algorithm>

#include "pa_tree.cuh"

namespace pa {
namespace {

__device__ unsigned g_err_tree_verify;

constexpr int kNodes = 64;
constexpr int kWarps = 16;
constexpr int kMaxCluster = 8;

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
struct Pair {
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

__device__ __forceinline__ double value(Pair x) { return (double)x.h + (double)x.l; }

// 1 / Z as (head, tail) of 1 / (Z 2^-e), and 2^-e in two factors (e up to 149).
__device__ __forceinline__ float4 reciprocal(double z) {
    int e;
    const double m = frexp(z, &e);  // z = m 2^e, m in [0.5, 1)
    const double inv = 1.0 / m;
    const float h = (float)inv;
    const int e1 = -e / 2;
    return make_float4(h, (float)(inv - (double)h), ldexpf(1.f, e1), ldexpf(1.f, -e - e1));
}

// r at a token after nrej rejections with draft probabilities: first p - q (exact),
// then r / Z - q with each later Z.
__device__ __forceinline__ Pair residual(float p, float q, int nrej, const float4 *zinv) {
    Pair r = two_sum(p, -q);
    if (!(r.h > 0.f)) return {r.h != r.h ? r.h : 0.f, 0.f};
    for (int k = 1; k < nrej; ++k) {
        const float4 z = zinv[k];
        const float h = __fmul_rn(__fmul_rn(r.h, z.z), z.w), l = __fmul_rn(__fmul_rn(r.l, z.z), z.w);
        const float m = __fmul_rn(h, z.x);
        const float n = __fmaf_rn(h, z.y, __fmaf_rn(l, z.x, __fmaf_rn(h, z.x, -m)));
        const Pair d = two_sum(m, -q);
        const float e = __fadd_rn(d.l, n);
        r.h = __fadd_rn(d.h, e);
        r.l = __fadd_rn(e, -__fadd_rn(r.h, -d.h));
        if (!(r.h > 0.f)) return {r.h != r.h ? r.h : 0.f, 0.f};
    }
    return r;
}

__device__ __forceinline__ uint32_t peer_addr(const void *p, int rank) {
    uint32_t r;
    asm("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}

__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
}

__global__ void __launch_bounds__(kWarps * 32) tree_verify_kernel(const VerifyArgs a) {
    __shared__ int s_par[kNodes], s_tok[kNodes];
    __shared__ float s_p[kNodes], s_q[kNodes], s_u[kNodes];
    __shared__ double s_z[kNodes];       // Z before each rejection at the current node
    __shared__ float4 s_zinv[kNodes];
    __shared__ double s_tot[kWarps];     // warp sums of the last pass
    __shared__ double s_cta[2][kMaxCluster];  // CTA sums of the cluster, by turns
    __shared__ int s_cmd[3];             // what warp 0 asks for: node, rejections, last pass
    __shared__ double s_goal;
    __shared__ int s_pick;
    __shared__ float s_best[kWarps > kMaxCluster ? kWarps : kMaxCluster];
    __shared__ int s_arg[kWarps > kMaxCluster ? kWarps : kMaxCluster];
    __shared__ float s_cbest[kMaxCluster];
    __shared__ int s_carg[kMaxCluster];
    extern __shared__ uint32_t s_gone[];  // without draft: a bit per token of the slice

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
    const int n = span.n, V = a.vocab;
    const bool with = a.draft != nullptr;
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
    // Warp 0's walk.
    int cur = 0, nrej = 0, count = 1;
    double mass = 1.0;
    uint64_t todo = 0;  // children of cur still to be tried
    int my_par[2] = {-1, -1}, my_tok[2] = {-1, -1};
    auto children = [&](int node) {
        const unsigned lo = __ballot_sync(0xffffffffu, my_par[0] == node);
        const unsigned hi = __ballot_sync(0xffffffffu, my_par[1] == node);
        return (uint64_t)hi << 32 | lo;
    };
    if (warp == 0) {
        for (int i = 0; i < 2; ++i) {
            my_par[i] = s_par[lane + 32 * i];
            my_tok[i] = s_tok[lane + 32 * i];
        }
        todo = children(0);
        if (rank == 0 && lane == 0) path[0] = 0;
    }
    auto row_of = [&](const float *m, int64_t stride, int node) {
        return m + (int64_t)(span.row0 + node) * stride;
    };
    // r at token x of this CTA's slice.
    auto r_at = [&](const float *p, const float *q, int rej, int x) -> Pair {
        if (!with) {
            const int i = x - c0;
            return {(s_gone[i >> 5] >> (i & 31)) & 1u ? 0.f : p[x], 0.f};
        }
        if (rej == 0) return {p[x], 0.f};
        return residual(p[x], q[x], rej, s_zinv);
    };
    int turn = 0, last_node = 0, last_rej = 0;
    bool have = false;  // the warp sums are those of (cur, nrej)
    double whole = 0.0;
    for (;;) {
        if (warp == 0) {
            // On to the next pass: a rejection's sum, or the last one.
            bool ask = false;
            while (!ask && todo && mass > 0.0) {
                const int i = __ffsll((long long)todo) - 1;
                todo &= todo - 1;
                const int tok = s_tok[i];
                const double p = s_p[i], q = s_q[i], u = s_u[i];
                bool ok;
                double r = p;
                if (with) {
                    for (int k = 0; k < nrej; ++k) r = fmax(r / s_z[k] - q, 0.0);
                    ok = u * q * mass < r;
                } else {
                    // Gone already when an earlier sibling had the same token.
                    const bool twin =
                        (my_par[0] == cur && lane < i && my_tok[0] == tok) ||
                        (my_par[1] == cur && lane + 32 < i && my_tok[1] == tok);
                    if (__any_sync(0xffffffffu, twin)) r = 0.0;
                    ok = u * mass < r;
                }
                if (ok) {
                    if (rank == 0 && lane == 0) path[count] = i;
                    ++count;
                    cur = i;
                    nrej = 0;
                    mass = 1.0;
                    have = false;
                    todo = children(i);
                } else if (with) {
                    if (lane == 0) {
                        s_z[nrej] = mass;
                        s_zinv[nrej] = reciprocal(mass);
                    }
                    __syncwarp();
                    ++nrej;
                    ask = true;
                } else {
                    mass -= r;
                }
            }
            const bool last = !ask;
            if (last && !with) {  // every child of cur was tried and rejected
                for (int i = 0; i < 2; ++i) {
                    const int t = my_tok[i] - c0;
                    // Only those tried: mass may have run out before the others.
                    const bool tried = my_par[i] == cur && !((todo >> (lane + 32 * i)) & 1ull);
                    if (tried && my_tok[i] >= c0 && my_tok[i] < c1)
                        atomicOr(&s_gone[t >> 5], 1u << (t & 31));
                }
            }
            if (lane == 0) {
                s_cmd[0] = cur;
                s_cmd[1] = nrej;
                s_cmd[2] = (last ? 1 : 0) | (last && have ? 2 : 0);
            }
        }
        __syncthreads();
        const int node = s_cmd[0], rej = s_cmd[1], flags = s_cmd[2];
        last_node = node;
        last_rej = rej;
        if (!(flags & 2)) {
            const float *p = row_of(a.target, a.target_stride, node);
            const float *q = with ? row_of(a.draft, a.draft_stride, node) : p;
            Pair acc[4] = {};
            int x = v0 + lane;
            for (; x + 96 < v1; x += 128) {
                Pair r[4];
                if (with && rej > 0) {
                    float pv[4], qv[4];
#pragma unroll
                    for (int k = 0; k < 4; ++k) {
                        pv[k] = p[x + 32 * k];
                        qv[k] = q[x + 32 * k];
                    }
#pragma unroll
                    for (int k = 0; k < 4; ++k) r[k] = residual(pv[k], qv[k], rej, s_zinv);
                } else {
#pragma unroll
                    for (int k = 0; k < 4; ++k) r[k] = r_at(p, q, rej, x + 32 * k);
                }
#pragma unroll
                for (int k = 0; k < 4; ++k) add_to(acc[k], r[k]);
            }
            for (; x < v1; x += 32) add_to(acc[0], r_at(p, q, rej, x));
            double t = (value(acc[0]) + value(acc[1])) + (value(acc[2]) + value(acc[3]));
#pragma unroll
            for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
            if (lane == 0) s_tot[warp] = t;
            __syncthreads();
            if (warp == 0) {
                // This CTA's sum, in warp order, to every CTA of the cluster.
                double sum = 0.0;
                for (int w = 0; w < kWarps; ++w) sum += s_tot[w];
                if (lane < C)
                    asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(
                                     peer_addr(&s_cta[turn][rank], lane)),
                                 "d"(sum)
                                 : "memory");
            }
            __syncwarp();
            if (C > 1)
                cluster_sync();
            else
                __syncthreads();
            if (warp == 0) {
                whole = 0.0;
                for (int c = 0; c < C; ++c) whole += s_cta[turn][c];
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
        // The CTA, and there the warp, that holds the goal; where rounding leaves none
        // (or sample_u >= 1) the last with weight, and the last token with weight in it.
        const double *cta = s_cta[turn ^ 1];
        double goal = (double)a.sample_u[s] * whole, before = 0.0;
        int pick = -1;
        for (int c = 0; c < C && pick < 0; ++c) {
            if (before + cta[c] > goal)
                pick = c;
            else
                before += cta[c];
        }
        if (pick < 0) {
            goal = INFINITY;
            for (int c = 0; c < C; ++c)
                if (cta[c] > 0.0) pick = c;
        }
        int w_pick = pick < 0 ? -2 : -1;
        if (pick == rank) {
            for (int w = 0; w < kWarps && w_pick < 0; ++w) {
                if (before + s_tot[w] > goal)
                    w_pick = w;
                else
                    before += s_tot[w];
            }
            if (w_pick < 0) {
                goal = INFINITY;
                for (int w = 0; w < kWarps; ++w)
                    if (s_tot[w] > 0.0) w_pick = w;
            }
        }
        if (lane == 0) {
            s_goal = goal - before;
            s_pick = w_pick;
        }
    }
    __syncthreads();
    const float *p = row_of(a.target, a.target_stride, last_node);
    if (s_pick != -2) {
        if (warp != s_pick) return;
        const float *q = with ? row_of(a.draft, a.draft_stride, last_node) : p;
        double goal = s_goal;
        // 32 contiguous shares of the warp's tokens, one per lane, then the share that
        // holds the goal, 32 tokens at a time.
        const int per = (v1 - v0 + 31) / 32;
        const int x0 = min(v1, v0 + lane * per), x1 = min(v1, x0 + per);
        Pair acc = {0.f, 0.f};
        for (int x = x0; x < x1; ++x) add_to(acc, r_at(p, q, last_rej, x));
        const double mine = value(acc);
        double incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const double u = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o) incl += u;
        }
        const unsigned over = __ballot_sync(0xffffffffu, mine > 0.0 && incl > goal);
        const unsigned some = __ballot_sync(0xffffffffu, mine > 0.0);
        int at = 0;
        if (over) {
            at = __ffs((int)over) - 1;
            goal -= __shfl_sync(0xffffffffu, incl - mine, at);
        } else {
            at = some ? 31 - __clz((int)some) : 0;
            goal = INFINITY;
        }
        const int y0 = min(v1, v0 + at * per), y1 = min(v1, y0 + per);
        int last = y0;
        for (int b = y0; b < y1; b += 32) {
            const int x = b + lane;
            const double r = x < y1 ? value(r_at(p, q, last_rej, x)) : 0.0;
            double c = r;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const double u = __shfl_up_sync(0xffffffffu, c, o);
                if (lane >= o) c += u;
            }
            const unsigned hit = __ballot_sync(0xffffffffu, r > 0.0 && c > goal);
            const unsigned any = __ballot_sync(0xffffffffu, r > 0.0);
            if (hit) {
                last = b + __ffs((int)hit) - 1;
                break;
            }
            if (any) last = b + 31 - __clz((int)any);
            goal -= __shfl_sync(0xffffffffu, c, 31);
        }
        if (lane == 0) a.next[s] = last;
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
    unsigned zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(bits, g_err_tree_verify, sizeof(unsigned));
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_err_tree_verify, &zero, sizeof(unsigned));
    return e;
}

#ifndef PA_VERIFY_CTAS
#define PA_VERIFY_CTAS 8
#endif

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
    // CTAs per sequence: a few per SM over the batch, each with at least four tokens
    // per thread, and slices whose bit sets fit the default shared memory.
    int c = 1;
    while (c < kMaxCluster && ((long long)c * t.num_seqs < PA_VERIFY_CTAS * device_sm_count() ||
                               vocab / c > (1 << 18)) &&
           vocab / (2 * c) >= kWarps * 32 * 4)
        c *= 2;
    a.cluster = c;
    auto up32 = [](int x) { return (x + 31) / 32 * 32; };
    a.cta_slice = up32((vocab + c - 1) / c);
    a.warp_slice = up32((a.cta_slice + kWarps - 1) / kWarps);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(t.num_seqs * c));
    cfg.blockDim = dim3(kWarps * 32);
    cfg.dynamicSmemBytes = draft ? 0 : (size_t)a.cta_slice / 8;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = (unsigned)c;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, tree_verify_kernel, a);
}

}  // namespace pa
