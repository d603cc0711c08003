"""Draft trees on the GPU in the regimes that large batches and vocabularies bring:
clusters of CTAs per sequence, ranges of many tiles, many segments per range.
"""

from __future__ import annotations

import time

import numpy as np
import pytest
import torch

from paged_kv_cache_287_gb300 import binding
from tests import _tree
from tests.test_gpu_tree import Case, run_verify

pytestmark = pytest.mark.gpu

DEV = torch.device("cuda:0")
I32 = torch.int32


@pytest.fixture(autouse=True)
def _clean_errors():
    binding.pa_error_check()
    yield
    binding.pa_error_check()


# ---------------------------------------------------------------- attention
def check_some(c, which, out=None, what=""):
    """The rows of sequences `which` of a batch, each against the definition over its own
    blocks."""
    out = c.run() if out is None else out
    b, cu = c.b, _tree.cu_of(c.T)
    for s in which:
        n = int(b.seq_lens[s])
        ids = b.block_tables[s, :-(-n // b.block_size)].long()
        rows = slice(int(cu[s]), int(cu[s + 1]))
        table = torch.arange(len(ids)).view(1, -1)
        want, tol = _tree.tree_attention(b.q[rows], c.pool[ids], table, [n], [c.T[s]],
                                         c.up[rows], b.scale, c.scales)
        _tree.assert_attention(out[rows], want, tol, f"{what} sequence {s}")
    assert torch.isfinite(out.float()).all()


def workers():
    """CTAs of a large batch: two per SM."""
    return 2 * torch.cuda.get_device_properties(0).multi_processor_count


@pytest.mark.parametrize("tiles", [3, 4, 5, 8, 9, 13])
@pytest.mark.parametrize("heads,T", [(8, 6), (64, 40)])  # up to 64 rows, and more
def test_ranges_of_few_tiles_of_head_size_64(tiles, heads, T):
    """Every CTA walks this many 64-key tiles (the ring of K and V holds four of each): no
    wait runs out, which would take seconds and be flagged."""
    kv_heads = 8
    groups = -(-T * (heads // kv_heads) // 128)
    per_seq = max(7, -(-workers() * tiles // (kv_heads * groups * 2)))
    ctx = [per_seq * 64 - T - i for i in range(2)]
    c = Case(ctx, [T] * 2, heads, kv_heads, 64, 16, seed=tiles)
    c.run()
    torch.cuda.synchronize()
    ws, out = c.workspace(), torch.empty_like(c.b.q)
    start = time.perf_counter()
    for _ in range(20):
        c.run(out=out, ws=ws)
    torch.cuda.synchronize()
    assert time.perf_counter() - start < 1.0
    check_some(c, [0, 1], out)


@pytest.mark.parametrize("T,heads", [(5, 4), (64, 16)])
def test_cleared_values_are_handed_over_on_every_call(T, heads):
    """V of unseen nodes and of what lies behind the sequences holds NaN and infinities, in
    tiles that are cleared by 32 lanes and read by a product that one issues: fifty calls,
    the same finite result."""
    c = Case([70, 500, 129, 60], [T, T, 1, T], heads, 2, 128, 16, seed=33, shape="star")
    b = c.b
    ends = b.seq_lens.tolist()
    want, tol = c.reference()
    for s, n in enumerate(ends):  # behind the sequence, to the end of its block
        blk = int(b.block_tables[s, (n - 1) // 16])
        if n % 16:
            c.pool[blk, :, :, n % 16:] = float("nan")
    rows = []
    for s, lo in enumerate(b.cu_q_lens.tolist()[:-1]):
        if c.T[s] > 2:  # node 2 is seen by itself alone
            slot = int(b.slot_mapping[lo + 2])
            c.pool[slot // 16, 1, :, slot % 16, ::3] = float("inf")
            rows.append(lo + 2)
    keep = [r for r in range(b.q.shape[0]) if r not in rows]
    first, ws = c.run(), c.workspace()
    _tree.assert_attention(first[keep], want[keep], tol[keep])
    out = torch.empty_like(first)
    for i in range(50):
        out.fill_(float("nan"))
        c.run(out=out, ws=ws)
        assert torch.equal(out.view(torch.int16), first.view(torch.int16)), i


KINDS = [(64, False), (128, False), (128, True)]  # head size, FP8 pool


@pytest.mark.parametrize("D,fp8", KINDS)
@pytest.mark.parametrize("wide", [False, True])
def test_ranges_of_many_tiles_and_segments(D, fp8, wide):
    """At least 14 tiles per CTA, so that ranges are cut with the weight of a change: rings
    that wrap, many segments per range, ragged contexts, empty trees in between; wide: trees
    of one to four row groups, whose CTAs walk side by side."""
    rng = np.random.default_rng(40 + D + 2 * fp8 + wide)
    B, heads, kv_heads = (24, 32, 4) if wide else (40, 32, 8)
    T = [int(t) for t in rng.integers(1, 65 if wide else 17, B)]
    T[:4] = [64, 1, 33, 17] if wide else [16, 1, 0, 9]
    mean = 14 * workers() * 64 // (B * kv_heads)
    ctx = [int(x) for x in rng.integers(mean // 4, 2 * mean, B)]
    ctx[1], ctx[3] = 6 * mean, 5
    c = Case(ctx, T, heads, kv_heads, D, 16, seed=41, fp8=fp8)
    tiles = [-(-(a + t) // 64) * -(-t * heads // kv_heads // 128) for a, t in zip(ctx, T)]
    assert kv_heads * sum(tiles) >= 12 * workers()
    check_some(c, [0, 1, 3, int(rng.integers(4, B)), B - 1])


@pytest.mark.parametrize("less", [0, 1])
@pytest.mark.parametrize("D,fp8", KINDS)
def test_ranges_on_both_sides_of_the_weight_of_a_change(less, D, fp8):
    """Batches of exactly 12 tiles per CTA, and of one tile less."""
    B, kv_heads = 2, 2
    per_seq = 12 * workers() // (B * kv_heads)
    lens = [64 * (per_seq + 5), 64 * (per_seq - 5 - less) - 3]
    T = [6, 3]
    assert kv_heads * sum(-(-n // 64) for n in lens) == 12 * workers() - kv_heads * less
    check_some(Case([n - t for n, t in zip(lens, T)], T, 8, kv_heads, D, 32, seed=42, fp8=fp8),
               [0, 1], what=f"less {less}")


@pytest.mark.parametrize("n", [1, 40, 900])
@pytest.mark.parametrize("heads,hi", [(8, 12), (64, 64)])
def test_ranges_that_begin_and_end_inside_a_change(n, heads, hi):
    """Segments of n tokens of context, thousands of ranges' borders among them: borders fall
    on every unit of a change and of its tiles."""
    rng = np.random.default_rng(n + heads)
    kv_heads = 8
    per = -(-(n + hi) // 64)
    B = min(1500, 13 * workers() // (per * kv_heads) + 1)
    T = [int(t) for t in rng.integers(1, hi + 1, B)]
    c = Case([n + i % 7 for i in range(B)], T, heads, kv_heads, 64, 8, seed=43)
    check_some(c, sorted({0, B - 1, *rng.integers(0, B, 14).tolist()}))


@pytest.mark.parametrize("D,fp8", KINDS)
@pytest.mark.parametrize("heads", [8, 32])
def test_attention_in_other_batch_orders(D, fp8, heads):
    """The same sequences in three orders: ranges are cut elsewhere, every result within the
    definition's tolerance."""
    rng = np.random.default_rng(44)
    T = [9, 40, 16, 1, 64, 0, 5]
    c = Case([700, 90, 4000, 64, 2000, 0, 1500], T, heads, 4, D, 16, seed=45, fp8=fp8)
    b, cu = c.b, _tree.cu_of(T)
    want, tol = c.reference()
    for _ in range(3):
        order = rng.permutation(len(T))
        rows = np.concatenate([np.arange(cu[s], cu[s + 1]) for s in order])
        at = torch.from_numpy(rows).to(DEV)
        out = torch.full_like(b.q, float("nan"))
        binding.pa_tree_attention(
            out, b.q[at].contiguous(), torch.from_numpy(_tree.cu_of([T[s] for s in order])).to(DEV),
            c.parents[at].contiguous(), c.max_tree, c.pool,
            b.block_tables[torch.from_numpy(order).to(DEV)].contiguous(),
            b.seq_lens[torch.from_numpy(order).to(DEV)].contiguous(), c.max_len, b.scale,
            c.workspace(), kv_scales=c.scales)
        _tree.assert_attention(out, want[rows], tol[rows], str(order))


@pytest.mark.parametrize("seed", range(24))
def test_attention_of_random_shapes(seed):
    rng = np.random.default_rng(1000 + seed)
    fp8 = bool(rng.integers(0, 2))
    kv_heads, group = int(rng.choice([1, 2, 3, 8])), int(rng.integers(1, 9))
    D, bs = (128 if fp8 else int(rng.choice([64, 128]))), int(rng.choice([8, 16, 32]))
    B, hi = int(rng.integers(1, 9)), int(rng.choice([2, 8, 17, 64]))
    T = [int(t) for t in rng.integers(0, hi + 1, B)]
    T[0] = max(T[0], 1)
    edges = [0, 1, 7, 63, 64, 65, 127, 128, 383, 384, 385, 1000]
    ctx = [int(rng.choice(edges)) if rng.random() < 0.6 else int(rng.integers(0, 3000))
           for _ in T]
    shape = str(rng.choice(["tree", "chain", "star", "forest"]))
    c = Case([x if t else 0 for x, t in zip(ctx, T)], T, kv_heads * group, kv_heads, D, bs,
             seed=seed, shape=shape, fp8=fp8, scale=float(rng.choice([0.05, 0.2, -0.1])))
    c.check(f"{kv_heads}x{group} D {D} block {bs} T {T} ctx {ctx} {shape}")


@pytest.mark.parametrize("T", [9, 64])  # up to 64 rows, and more
@pytest.mark.parametrize("scale,k_scale", [(0.0, None), (0.1, 1e-9), (1e-12, 1e-30)])
def test_tiny_queries_and_scales_over_an_fp8_pool(T, scale, k_scale):
    """A row's factor (scale, K's scale and the row's own power of two) may lie below the
    smallest fp32 number: the row still takes the mean of what it sees, and of nothing
    else."""
    c = Case([100, 700], [T, 5], 8, 2, 128, 16, seed=26, fp8=True, scale=scale)
    if k_scale is not None:
        c.scales = (k_scale, c.scales[1])
    q = c.b.q
    q[1] = 0.0
    q[2] *= 2.0 ** -40
    q[3] *= 2.0 ** -100
    q[4, 1] = 1e-39  # a subnormal
    c.check()


# ---------------------------------------------------------------- verification in clusters
@pytest.mark.parametrize("vocab", [5000, 16384, 40000])  # 2, 8 and 8 CTAs per sequence
@pytest.mark.parametrize("with_draft", [True, False])
def test_verify_in_clusters_beside_other_work(vocab, with_draft):
    """Clusters that start while other kernels hold parts of the GPU: every call gives the
    walk's result."""
    d = _tree.random_drafts(vocab, [20, 0, 3, 64, 1], vocab, with_draft, "star")
    args = [x if x is None else x.to(DEV)
            for x in (d.target, d.draft, d.tokens, d.cu, d.parents, d.accept_u, d.sample_u)]
    paths, nexts = d.reference
    a = torch.randn(1500, 1500, device=DEV)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    outs = [[torch.empty(5, 64, dtype=I32, device=DEV), torch.empty(5, dtype=I32, device=DEV),
             torch.empty(5, dtype=I32, device=DEV)] for _ in range(40)]
    for s in streams:
        s.wait_stream(torch.cuda.current_stream())
    for i, out in enumerate(outs):
        if i % 3 == 0:
            with torch.cuda.stream(streams[1 - i % 2]):
                a = (a @ a).clamp_(-1, 1)
        with torch.cuda.stream(streams[i % 2]):
            binding.pa_tree_verify(*out, *args)
    torch.cuda.synchronize()
    for acc, num, nxt in outs:
        assert nxt.tolist() == nexts
        assert [acc[i, :n].tolist() for i, n in enumerate(num.tolist())] == paths


@pytest.mark.parametrize("with_draft", [True, False])
@pytest.mark.parametrize("B,vocab", [(2, 1 << 20), (170, 600011)])
def test_verify_of_the_largest_vocabularies(B, vocab, with_draft):
    """Up to 1048576 tokens; and so large a batch that the clusters' size goes by the
    vocabulary alone (four CTAs, each of at most 2^18 tokens)."""
    T = [4 if s == B // 2 else 1 for s in range(B)]
    g = torch.Generator(device=DEV).manual_seed(B)
    target = torch.softmax(torch.randn(sum(T), vocab, generator=g, device=DEV) * 2, dim=1)
    draft = torch.softmax(target.log() + torch.randn(sum(T), vocab, generator=g, device=DEV), 1)
    up = sum((([-1, 0, 0, 1]) if t > 1 else [-1] for t in T), [])
    cu = _tree.cu_of(T)
    base = np.repeat(cu[:-1], T)
    tokens = torch.tensor([int(draft[b + max(p, 0)].argmax()) if p >= 0 else 0
                           for b, p in zip(base, up)], dtype=I32)
    d = _tree.Drafts(target.cpu(), draft.cpu() if with_draft else None, tokens,
                     torch.tensor(up, dtype=I32), torch.from_numpy(cu),
                     torch.rand(sum(T), generator=torch.Generator().manual_seed(1)),
                     torch.rand(B, generator=torch.Generator().manual_seed(2)), T)
    del target, draft
    assert run_verify(d) == d.reference


@pytest.mark.parametrize("vocab", [16384, 50021])
def test_verify_falls_back_in_clusters(vocab):
    """Nothing left to draw from, with eight CTAs per sequence: the lowest token of the
    target's largest probability, wherever its CTA's slice; and a draw whose goal no running
    sum exceeds: the last token with weight."""
    for lo, hi in ((3, vocab - 2), (vocab // 2 - 1, vocab // 2 + 1), (vocab - 9, vocab - 3)):
        p = torch.zeros(4, vocab)
        p[:, lo], p[:, hi] = 0.5, 0.5
        cu = torch.tensor([0, 4], dtype=I32)
        star = torch.tensor([-1, 0, 0, 0], dtype=I32)
        tokens = torch.tensor([0, hi, hi, lo], dtype=I32)
        d = _tree.Drafts(p, p.clone(), tokens, star, cu, torch.ones(4), torch.tensor([0.7]), [4])
        assert run_verify(d) == d.reference == ([[0]], [lo])
        d = _tree.Drafts(p, None, torch.tensor([0, hi, lo, lo], dtype=I32), star, cu,
                         torch.ones(4), torch.tensor([0.7]), [4])
        assert run_verify(d) == d.reference == ([[0]], [lo])
        one = torch.tensor([0, 1], dtype=I32)
        d = _tree.Drafts(p[:1], None, tokens[:1], star[:1], one, torch.zeros(1),
                         torch.tensor([1.0]), [1])
        assert run_verify(d) == d.reference == ([[0]], [hi])


# ---------------------------------------------------------------- verification's sums
def lossy_row(vocab):
    """Probabilities whose sum a head with a tail in plain fp32 gets wrong by some 2^-34, and
    a sample_u whose goal lies between: token 0 has 1, 255 tokens of the same thread a little
    less than 2^-24 each, chosen so that the tail's rounding loses nearly half a unit every
    time."""
    at = [128 * (j // 2) + 2 * (j % 2) for j in range(256)]
    step, tail, lost, t = 2.0 ** -48, np.float32(0), 0.0, [1.0]
    for _ in range(1, 255):
        x = 0.9 * 2.0 ** -24 // step * step
        unit = 2.0 ** (np.floor(np.log2(float(tail) + x)) - 23)
        if unit > step:
            x += (0.5 * unit - step - (float(tail) + x) % unit) % unit
            x -= unit * (x >= 2.0 ** -24)
        assert x == float(np.float32(x)) and 0 < x < 2.0 ** -24
        new = np.float32(float(tail) + x)
        lost += float(tail) + x - float(new)
        tail = new
        t.append(x)
    cum = np.cumsum(t)  # exact: multiples of 2^-48 below 2
    # The last number puts u times the whole a third of what is lost past token j's sum.
    u, j, x = next((u, j, x) for u in 1.0 - np.arange(40, 200) * 2.0 ** -24
                   for j in range(100, 250) for x in [(cum[j] + lost / 3) / u - cum[-1]]
                   if 2.0 ** -25 < x < 2.0 ** -24)
    t.append(float(np.float32(x)))
    total = cum[-1] + t[-1]
    assert lost > 2.0 ** -35 and u * (total - lost) < cum[j] < u * total
    row = torch.zeros(vocab)
    row[at] = torch.tensor(t, dtype=torch.float64).float()
    return row, float(u), at[j + 1]


def test_verify_sums_many_small_numbers_to_more_than_a_heads_and_a_tails_bits():
    """As many sequences as give each one CTA, so that a thread adds 256 numbers: the draw
    depends on bits that a tail in plain fp32 loses."""
    B, vocab = workers() // 2 + 8, 1 << 18
    row, u, want = lossy_row(vocab)
    target = torch.zeros(B, vocab)
    target[:, 7] = 1.0
    target[B // 2] = row
    d = _tree.Drafts(target, None, torch.zeros(B, dtype=I32),
                     torch.full((B,), -1, dtype=I32), torch.arange(B + 1, dtype=I32),
                     torch.zeros(B), torch.full((B,), u), [1] * B)
    got = run_verify(d)
    assert d.reference[1][B // 2] == want
    assert got == d.reference
