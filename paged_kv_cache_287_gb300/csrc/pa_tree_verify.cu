// pa_tree_verify.cu - accept drafted tokens against the target's probabilities.
//
// Per sequence a walk from the root: at the last accepted node n, r = p_n and
// Z = 1; child c (token t) is accepted when u_c q_n(t) Z < r(t), else
// r := max(r / Z - q_n, 0), Z := sum r (without draft probabilities: accepted when
// u_c Z < r(t), else r(t) := 0, Z -= r(t)).  When no child is accepted the next
// token is the smallest x with r(0) + .. + r(x) > u sum r.
//
// One CTA per sequence; every thread makes the same walk over the tree's scalars
// in shared memory, and the vocabulary is only touched by the sums: each warp sums
// a contiguous range of it, and the range that holds the goal is scanned again.
#include <algorithm>

#include "pa_tree.cuh"

namespace pa {
namespace {

__device__ unsigned g_err_tree_verify;

constexpr int kNodes = 64;
constexpr int kWarps = 16;

struct VerifyArgs {
    int32_t *accepted, *num_accepted, *next;
    const float *target, *draft;
    int64_t target_stride, draft_stride;
    const int32_t *tokens;
    const float *accept_u, *sample_u;
    TreeGeom t;
    int vocab;
};

__global__ void __launch_bounds__(kWarps * 32) tree_verify_kernel(const VerifyArgs a) {
    __shared__ int s_par[kNodes], s_tok[kNodes], s_rej[kNodes];
    __shared__ float s_p[kNodes], s_q[kNodes], s_u[kNodes];
    __shared__ double s_tot[kWarps];
    __shared__ double s_z[kNodes];
    __shared__ int s_arg[kWarps];
    __shared__ float s_best[kWarps];
    extern __shared__ uint32_t s_gone[];  // without draft: a bit per rejected token

    const int s = blockIdx.x, tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const TreeSpan span = tree_span(a.t, s);
    int32_t *path = a.accepted + (size_t)s * a.t.max_tree;
    if (span.n <= 0) {
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
    if (tid < n) {
        int par = a.t.parents[span.row0 + tid];
        if (par < -1 || par >= tid) {
            atomicOr(&g_err_tree_verify, kErrOob);
            par = -1;
        }
        int tok = tid > 0 ? a.tokens[span.row0 + tid] : 0;
        float p = 0.f, q = 0.f;
        if (tok < 0 || tok >= V) {
            atomicOr(&g_err_tree_verify, kErrOob);
            tok = -1;
        } else if (tid > 0 && par >= 0) {
            p = a.target[(int64_t)(span.row0 + par) * a.target_stride + tok];
            if (a.draft) q = a.draft[(int64_t)(span.row0 + par) * a.draft_stride + tok];
        }
        s_par[tid] = par;
        s_tok[tid] = tok;
        s_p[tid] = p;
        s_q[tid] = q;
        s_u[tid] = a.accept_u[span.row0 + tid];
    }
    const int words = (V + 31) / 32;
    if (!a.draft)
        for (int i = tid; i < words; i += blockDim.x) s_gone[i] = 0u;
    __syncthreads();

    const int chunk = ((V + kWarps - 1) / kWarps + 31) / 32 * 32;
    const int v0 = min(V, warp * chunk), v1 = min(V, v0 + chunk);
    int cur = 0, nrej = 0, count = 1;
    double mass = 1.0;
    bool have_tot = false;
    // r at x after the rejections so far, from p and q there.
    auto residual = [&](float p, float q) {
        double r = p;
        for (int k = 0; k < nrej; ++k) r = fmax(r / s_z[k] - (double)q, 0.0);
        return r;
    };
    auto r_at = [&](int x) -> double {
        const float p = a.target[(int64_t)(span.row0 + cur) * a.target_stride + x];
        if (!a.draft) return (s_gone[x >> 5] >> (x & 31)) & 1u ? 0.0 : (double)p;
        if (nrej == 0) return p;
        return residual(p, a.draft[(int64_t)(span.row0 + cur) * a.draft_stride + x]);
    };
    // Warp totals of r into s_tot.
    auto totals = [&]() {
        __syncthreads();
        double t = 0.0;
        for (int x = v0 + lane; x < v1; x += 32) t += r_at(x);
        for (int o = 16; o > 0; o >>= 1) t += __shfl_xor_sync(0xffffffffu, t, o);
        if (lane == 0) s_tot[warp] = t;
        __syncthreads();
        have_tot = true;
    };
    if (tid == 0) path[0] = 0;
    for (int i = 1; i < n; ++i) {
        if (s_par[i] != cur || !(mass > 0.0)) continue;
        const int tok = s_tok[i];
        double have = 0.0, need = (double)s_u[i] * mass;
        if (a.draft) {
            have = residual(s_p[i], s_q[i]);
            need = (double)s_u[i] * (double)s_q[i] * mass;
        } else if (tok >= 0) {
            have = (s_gone[tok >> 5] >> (tok & 31)) & 1u ? 0.0 : (double)s_p[i];
        }
        __syncthreads();
        if (need < have) {  // accepted
            if (!a.draft && tid < nrej) s_gone[s_rej[tid] >> 5] = 0u;
            if (tid == 0) path[count] = i;
            ++count;
            cur = i;
            nrej = 0;
            mass = 1.0;
            have_tot = false;
        } else if (a.draft) {
            if (tid == 0) s_z[nrej] = mass;
            ++nrej;
            totals();
            mass = 0.0;
            for (int w = 0; w < kWarps; ++w) mass += s_tot[w];
        } else {
            if (tok >= 0) {
                if (tid == 0) {
                    s_gone[tok >> 5] |= 1u << (tok & 31);
                    s_rej[nrej] = tok;
                }
                ++nrej;
            }
            mass -= have;
            have_tot = false;
        }
        __syncthreads();
    }
    for (int i = count + tid; i < a.t.max_tree; i += blockDim.x) path[i] = -1;
    if (tid == 0) a.num_accepted[s] = count;

    // The next token.
    if (!have_tot) totals();
    double whole = 0.0;
    for (int w = 0; w < kWarps; ++w) whole += s_tot[w];
    double goal = (double)a.sample_u[s] * whole;
    double before = 0.0;
    int pick = -1;
    for (int w = 0; w < kWarps && pick < 0; ++w) {
        if (before + s_tot[w] > goal)
            pick = w;
        else
            before += s_tot[w];
    }
    if (pick < 0) {  // rounding, or sample_u >= 1: the last x with r(x) > 0
        goal = INFINITY;
        for (int w = 0; w < kWarps; ++w)
            if (s_tot[w] > 0.0) pick = w;
    }
    if (pick >= 0) {
        if (warp != pick) return;
        int last = v0;
        for (int x0 = v0; x0 < v1; x0 += 32) {
            const int x = x0 + lane;
            const double r = x < v1 ? r_at(x) : 0.0;
            double c = r;
            for (int o = 1; o < 32; o <<= 1) {
                const double u = __shfl_up_sync(0xffffffffu, c, o);
                if (lane >= o) c += u;
            }
            const unsigned over = __ballot_sync(0xffffffffu, r > 0.0 && before + c > goal);
            const unsigned some = __ballot_sync(0xffffffffu, r > 0.0);
            if (over) {
                last = x0 + __ffs((int)over) - 1;
                break;
            }
            if (some) last = x0 + 31 - __clz((int)some);
            before += __shfl_sync(0xffffffffu, c, 31);
        }
        if (lane == 0) a.next[s] = last;
        return;
    }
    // Nothing left to draw from: the lowest x of the largest p.
    float best = -1.f;
    int arg = 0x7fffffff;
    for (int x = v0 + lane; x < v1; x += 32) {
        const float p = a.target[(int64_t)(span.row0 + cur) * a.target_stride + x];
        if (p > best) {
            best = p;
            arg = x;
        }
    }
    for (int o = 16; o > 0; o >>= 1) {
        const float b = __shfl_xor_sync(0xffffffffu, best, o);
        const int g = __shfl_xor_sync(0xffffffffu, arg, o);
        if (b > best || (b == best && g < arg)) {
            best = b;
            arg = g;
        }
    }
    if (lane == 0) {
        s_best[warp] = best;
        s_arg[warp] = arg;
    }
    __syncthreads();
    if (tid == 0) {
        for (int w = 1; w < kWarps; ++w)
            if (s_best[w] > s_best[0] || (s_best[w] == s_best[0] && s_arg[w] < s_arg[0])) {
                s_best[0] = s_best[w];
                s_arg[0] = s_arg[w];
            }
        a.next[s] = s_arg[0] < V ? s_arg[0] : 0;
    }
}

}  // namespace

cudaError_t take_error_tree_verify(unsigned *bits) {
    unsigned zero = 0;
    cudaError_t e = cudaMemcpyFromSymbol(bits, g_err_tree_verify, sizeof(unsigned));
    if (e == cudaSuccess) e = cudaMemcpyToSymbol(g_err_tree_verify, &zero, sizeof(unsigned));
    return e;
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
    const size_t smem = draft ? 0 : (size_t)(vocab + 31) / 32 * 4;
    if (smem > 40 << 10) {
        const cudaError_t e = ensure_smem<tree_verify_kernel>(smem);
        if (e != cudaSuccess) return e;
    }
    tree_verify_kernel<<<(unsigned)t.num_seqs, kWarps * 32, smem, stream>>>(a);
    return cudaGetLastError();
}

}  // namespace pa
