"""Draft trees for the tests: random trees, and plain 64-bit implementations.

The implementations here follow the formulas of ``include/pa.h`` with loops over
sequences and nodes; they share no code with the CUDA kernels.
"""

from __future__ import annotations

from dataclasses import dataclass
from typing import List, Optional, Sequence

import numpy as np
import torch

from paged_kv_cache_287_gb300.workloads import FP8_K_SCALE, FP8_V_SCALE


def random_parents(g: np.random.Generator, n: int, shape: str = "tree") -> List[int]:
    """Parents of n nodes: "chain", "star", "tree" (random recursive) or "forest"
    (a tree whose nodes may have no parent)."""
    if n == 0:
        return []
    if shape == "chain":
        return [-1] + list(range(n - 1))
    if shape == "star":
        return [-1] + [0] * (n - 1)
    lo = -1 if shape == "forest" else 0
    return [-1] + [int(g.integers(lo, i)) for i in range(1, n)]


def cu_of(lens: Sequence[int]) -> np.ndarray:
    return np.concatenate([[0], np.cumsum(lens)]).astype(np.int32)


def path_to(parents: Sequence[int], i: int) -> List[int]:
    out = []
    while i >= 0:
        out.append(i)
        i = parents[i]
    return out


def pool_values(pool: torch.Tensor, kv_scales=None) -> np.ndarray:
    """The pool's values in 64 bits (a uint8 pool holds e4m3 codes)."""
    if pool.dtype == torch.uint8:
        v = pool.cpu().view(torch.float8_e4m3fn).double().numpy().copy()
        v[:, 0] *= float(np.float32(kv_scales[0]))
        v[:, 1] *= float(np.float32(kv_scales[1]))
        return v
    return pool.cpu().double().numpy()


def tree_attention(q, pool, tables, seq_lens, tree_lens, parents, scale, kv_scales=None):
    """(result, tolerance) of tree attention, [rows, Hq, D] float64 each.

    The tolerance counts the kernel's roundings.  With A = sum_t softmax_t |v_t|:
    the output's rounding to bf16, 2^-8 |out|; P's rounding before P.V (bf16 2^-8,
    f16 2^-11 and 2^-25 below its normal range, on P >= 1 at the largest score)
    against an unrounded sum, that much of A; and in fp32 the products and sums of a
    score, at most (D + 8) 2^-24 sum_d |q_d k_d| |scale| each, twice (numerator and
    sum), with 2^-20 for exp2 and the accumulation of P.V in blocks of at least 16.  Over
    an FP8 pool a query is held as the sum of two e4m3 numbers after scaling its row's
    largest element into [128, 256): e4m3's step is at least 2^-9, so an element is off
    by at most 2^-10, that is 2^-17 of the largest, and the score by at most 2^-17
    max|q| sum_d |k_d| |scale|, again twice.
    """
    fp8 = pool.dtype == torch.uint8
    vals = pool_values(pool, kv_scales)
    qd = q.cpu().double().numpy()
    tables = tables.cpu().numpy()
    scale = float(np.float32(scale))
    bs = pool.shape[3]
    Hq, D = qd.shape[1:]
    Hkv = pool.shape[2]
    G = Hq // Hkv
    out, tol = np.zeros_like(qd), np.zeros_like(qd)
    cu = cu_of(tree_lens)
    for s, T in enumerate(tree_lens):
        n = int(seq_lens[s])
        ids = tables[s, :-(-n // bs)]
        kv = vals[ids].transpose(1, 2, 0, 3, 4).reshape(2, Hkv, -1, D)[:, :, :n]
        up = list(parents[cu[s]:cu[s + 1]])
        for i in range(T):
            seen = np.r_[0:n - T, sorted(n - T + j for j in path_to(up, i))].astype(int)
            for h in range(Hkv):
                k, v = kv[0, h][seen], kv[1, h][seen]
                qh = qd[cu[s] + i, h * G:(h + 1) * G]
                x = (qh @ k.T) * scale
                mag = (np.abs(qh) @ np.abs(k).T) * abs(scale)
                p = np.exp(x - x.max(axis=1, keepdims=True))
                l = p.sum(axis=1, keepdims=True)
                o = (p / l) @ v
                a = (p / l) @ np.abs(v)
                t = 2.0 ** -8 * np.abs(o) + 1e-30
                t += a * (2.0 ** -11 if fp8 else 2.0 ** -8)
                if fp8:
                    t += 2.0 ** -25 * np.abs(v).sum(axis=0) / l
                off = (D + 8) * 2.0 ** -24 * mag.max(axis=1, keepdims=True)
                if fp8:
                    off = off + 2.0 ** -17 * np.abs(qh).max(axis=1, keepdims=True) * \
                        np.abs(k).sum(axis=1).max() * abs(scale)
                t += a * (2 * off + 2.0 ** -20)
                out[cu[s] + i, h * G:(h + 1) * G] = o
                tol[cu[s] + i, h * G:(h + 1) * G] = t * (1 + 2.0 ** -7)
    return out, tol


def assert_attention(got: torch.Tensor, want: np.ndarray, tol: np.ndarray, what: str = ""):
    g = got.float().cpu().double().numpy()
    assert np.isfinite(g).all(), f"{what}: not finite"
    over = np.abs(g - want) - tol
    i = int(np.argmax(over)) if over.size else 0
    assert over.size == 0 or over.flat[i] <= 0, (
        f"{what}: |d| {abs(g.flat[i] - want.flat[i]):.3e} > {tol.flat[i]:.3e} at "
        f"{np.unravel_index(i, g.shape)}")


def verify(target, draft, tokens, tree_lens, parents, accept_u, sample_u):
    """The walk of every sequence in 64 bits: (paths, next tokens)."""
    cu = cu_of(tree_lens)
    V = target.shape[1]
    paths, nexts = [], []
    for s, T in enumerate(tree_lens):
        if T == 0:
            paths.append([])
            nexts.append(-1)
            continue
        lo = cu[s]
        path, r = [0], None
        while True:
            at = path[-1]
            r, z, found = target[lo + at].astype(np.float64), 1.0, None
            for c in range(1, T):
                if parents[lo + c] != at or not z > 0:
                    continue
                t, u = int(tokens[lo + c]), float(accept_u[lo + c])
                have = r[t] if 0 <= t < V else 0.0
                if draft is None:
                    if u * z < have:
                        found = c
                        break
                    if 0 <= t < V:
                        r[t] = 0.0
                    z -= have
                else:
                    q = draft[lo + at].astype(np.float64)
                    if u * (q[t] if 0 <= t < V else 0.0) * z < have:
                        found = c
                        break
                    r = np.maximum(r / z - q, 0.0)
                    z = r.sum()
            if found is None:
                break
            path.append(found)
        total = r.cumsum()
        if total[-1] > 0:
            over = np.nonzero(total > float(sample_u[s]) * total[-1])[0]
            nexts.append(int(over[0]) if over.size else int(np.nonzero(r)[0][-1]))
        else:
            nexts.append(int(np.argmax(target[lo + path[-1]])))
        paths.append(path)
    return paths, nexts


def accept(pool: np.ndarray, paths, tables, seq_lens, tree_lens):
    """Pool bits after the accepted rows moved, and the new lengths."""
    new, bs = pool.copy(), pool.shape[3]
    lens = []
    for s, path in enumerate(paths):
        base = int(seq_lens[s]) - tree_lens[s]
        for i, p in enumerate(path):
            src, dst = base + p, base + i
            new[tables[s, dst // bs], :, :, dst % bs] = pool[tables[s, src // bs], :, :, src % bs]
        lens.append(base + len(path))
    return new, np.array(lens, np.int32)


@dataclass
class Drafts:
    """Inputs of a verification, on the CPU."""

    target: torch.Tensor
    draft: Optional[torch.Tensor]
    tokens: torch.Tensor
    parents: torch.Tensor
    cu: torch.Tensor
    accept_u: torch.Tensor
    sample_u: torch.Tensor
    tree_lens: List[int]

    @property
    def reference(self):
        return verify(self.target.numpy(), None if self.draft is None else self.draft.numpy(),
                      self.tokens.numpy(), self.tree_lens, self.parents.tolist(),
                      self.accept_u.numpy(), self.sample_u.numpy())


def random_drafts(seed: int, tree_lens: Sequence[int], vocab: int, with_draft: bool,
                  shape: str = "tree", sharp: float = 2.0, near: float = 0.7) -> Drafts:
    """Random distributions, and tokens drawn from the draft's after their parent."""
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    rows = int(sum(tree_lens))
    logits = torch.randn(rows, vocab, generator=g) * sharp
    target = torch.softmax(logits, dim=1)
    draft = torch.softmax(logits + near * torch.randn(rows, vocab, generator=g), dim=1)
    parents, tokens, lo = [], [], 0
    for n in tree_lens:
        up = random_parents(rng, n, shape)
        for i in range(n):
            tokens.append(int(torch.multinomial(draft[lo + max(up[i], 0)], 1, generator=g)))
        parents += up
        lo += n
    i32 = torch.int32
    return Drafts(target, draft if with_draft else None, torch.tensor(tokens, dtype=i32),
                  torch.tensor(parents, dtype=i32), torch.from_numpy(cu_of(tree_lens)),
                  torch.rand(rows, generator=g), torch.rand(len(tree_lens), generator=g),
                  list(tree_lens))


FP8_SCALES = (FP8_K_SCALE, FP8_V_SCALE)
