"""Draft trees on the GPU: attention, verification and acceptance against plain
64-bit implementations, their awkward shapes and data, and a whole speculative step.
"""

from __future__ import annotations

import math

import numpy as np
import pytest
import torch

import oracle
from paged_kv_cache_287_gb300 import binding
from paged_kv_cache_287_gb300.workloads import fp8_pool_of, make_batch
from tests import _tree
from tests._gpu import bits, gpu_write, oracle_pool, workspace_for

pytestmark = pytest.mark.gpu

if not torch.cuda.is_available():
    pytest.skip("no CUDA device", allow_module_level=True)

DEV = torch.device("cuda:0")
I32 = torch.int32


@pytest.fixture(autouse=True)
def _clean_errors():
    binding.pa_error_check()
    yield
    binding.pa_error_check()


def ints(x):
    return torch.as_tensor(np.asarray(x, dtype=np.int32)).to(DEV)


class Case:
    """A batch of trees whose K/V are written, and its parents."""

    def __init__(self, ctx, T, heads, kv_heads, D, bs, seed=1, shape="tree", fp8=False,
                 scale=None, q_mult=1.0, **kw):
        rng = np.random.default_rng(seed)
        self.T, self.fp8 = list(T), fp8
        self.b = b = make_batch(
            name="tree", seq_lens=[c + t for c, t in zip(ctx, T)], q_lens=list(T),
            num_heads=heads, num_kv_heads=kv_heads, head_size=D, block_size=bs,
            scale=D ** -0.5 if scale is None else scale, seed=seed, q_scale=q_mult, device=DEV,
            **kw)
        self.scales = _tree.FP8_SCALES if fp8 else None
        if fp8:
            self.pool = fp8_pool_of(b)
            if b.slot_mapping.numel():
                binding.pa_cache_write_fp8(self.pool, b.k_new, b.v_new, b.slot_mapping,
                                           *self.scales)
        else:
            gpu_write(b)
            self.pool = b.kv_cache
        self.up = sum((_tree.random_parents(rng, t, shape) for t in T), [])
        self.parents = ints(self.up)
        self.max_tree = max(1, max(T, default=1))
        self.max_len = b.max_seq_len  # read once: a captured call must not synchronise

    def workspace(self):
        b = self.b
        return torch.empty(binding.pa_tree_attention_workspace_bytes(
            b.num_seqs, self.max_tree, b.num_heads, b.num_kv_heads, b.head_size),
            dtype=torch.uint8, device=DEV)

    def run(self, out=None, ws=None, **kw):
        b = self.b
        out = torch.full_like(b.q, float("nan")) if out is None else out
        binding.pa_tree_attention(out, kw.pop("q", b.q), b.cu_q_lens,
                                  kw.pop("parents", self.parents), self.max_tree, self.pool,
                                  b.block_tables, kw.pop("seq_lens", b.seq_lens), self.max_len,
                                  b.scale, self.workspace() if ws is None else ws,
                                  kv_scales=self.scales, **kw)
        return out

    def reference(self, up=None):
        b = self.b
        return _tree.tree_attention(b.q, self.pool, b.block_tables, b.seq_lens.tolist(), self.T,
                                    self.up if up is None else up, b.scale, self.scales)

    def check(self, what=""):
        _tree.assert_attention(self.run(), *self.reference(), what)


# ---------------------------------------------------------------- attention
SHAPES = [  # heads, kv heads, D, block size
    (1, 1, 64, 8), (2, 2, 128, 16), (4, 2, 64, 32), (6, 2, 128, 8), (8, 2, 64, 16),
    (10, 2, 128, 32), (6, 1, 64, 8), (14, 2, 128, 16), (16, 2, 64, 32), (8, 1, 128, 16)]


@pytest.mark.parametrize("heads,kv_heads,D,bs", SHAPES)
def test_attention_over_ragged_trees_and_contexts(heads, kv_heads, D, bs):
    """Tree sizes 1 .. 64 and contexts of none up to a few tiles, tile and block
    borders and their neighbours among them."""
    ctx = [0, 1, 0, 7, 63, 64, 120, 127, 128, 129, 255, 300, 0, 511]
    T = [1, 1, 64, 9, 33, 64, 8, 1, 17, 2, 31, 16, 13, 5]
    Case(ctx, T, heads, kv_heads, D, bs, seed=heads + D).check(f"{heads}/{kv_heads}/{D}/{bs}")


@pytest.mark.parametrize("heads,kv_heads,bs", [(1, 1, 8), (6, 2, 16), (8, 2, 32), (16, 2, 8)])
def test_attention_over_an_fp8_pool(heads, kv_heads, bs):
    ctx = [0, 1, 120, 128, 129, 300, 64, 700]
    T = [1, 64, 9, 33, 2, 16, 7, 48]
    Case(ctx, T, heads, kv_heads, 128, bs, seed=heads, fp8=True).check()


@pytest.mark.parametrize("shape", ["chain", "star", "forest"])
@pytest.mark.parametrize("fp8", [False, True])
def test_attention_of_chains_stars_and_forests(shape, fp8):
    Case([200, 3, 130], [20, 64, 6], 8, 2, 128, 16, seed=4, shape=shape, fp8=fp8).check(shape)


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("ctx,T,heads,kv_heads", [
    ([9000], [5], 4, 1), ([3, 5000, 1200], [64, 12, 40], 16, 2), ([2500] * 5, [3] * 5, 8, 8),
    ([40] * 90, [2] * 90, 4, 2)])
def test_attention_of_long_skewed_and_many_sequences(ctx, T, heads, kv_heads, fp8):
    """Contexts split over the GPU (and their pieces merged), and more sequences
    than that."""
    Case(ctx, T, heads, kv_heads, 128, 16, seed=7, fp8=fp8, q_mult=2.0).check()


@pytest.mark.parametrize("scale", [0.0, -0.1, 1e-3, 4.0])
def test_attention_scales(scale):
    Case([100, 260], [7, 30], 4, 2, 64, 16, seed=2, scale=scale).check(str(scale))


@pytest.mark.parametrize("fp8", [False, True])
def test_one_node_trees_are_the_decode_and_chains_the_prefill(fp8):
    c = Case([30, 500, 129], [1, 1, 1], 8, 2, 128, 16, seed=3, fp8=fp8)
    b, want = c.b, torch.empty_like(c.b.q)
    args = (want, b.q, c.pool, b.block_tables, b.seq_lens, b.max_seq_len, b.scale)
    binding.pa_decode_fp8(*args, *c.scales, workspace_for(b)) if fp8 else \
        binding.pa_decode(*args, workspace_for(b))
    _, tol = c.reference()
    _tree.assert_attention(c.run(), want.cpu().double().numpy(), 2 * tol)
    c = Case([30, 500, 129], [4, 64, 33], 8, 2, 128, 16, seed=3, fp8=fp8, shape="chain")
    b, want = c.b, torch.empty_like(c.b.q)
    args = (want, b.q, b.cu_q_lens, 64, c.pool, b.block_tables, b.seq_lens, b.scale)
    binding.pa_prefill_chunk_fp8(*args, *c.scales) if fp8 else binding.pa_prefill_chunk(*args)
    _, tol = c.reference()
    _tree.assert_attention(c.run(), want.cpu().double().numpy(), 2 * tol)


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("T,ctx", [(9, 20), (64, 100), (40, 0)])
def test_what_a_node_does_not_see_has_no_part_in_its_result(bad, T, ctx):
    """Node j's K and V hold NaN or infinities: rows that do not see node j are what
    they were, bit for bit (the same work is done for them)."""
    c = Case([ctx, 33], [T, 3], 4, 2, 128, 16, seed=T)
    before = c.run()
    b, j = c.b, T // 3
    slot = int(b.slot_mapping[j])
    c.pool[slot // 16, :, :, slot % 16] = bad
    after = c.run()
    sees = torch.tensor([j in _tree.path_to(c.up[:T], i) for i in range(T)] + [False] * 3)
    assert torch.equal(before[~sees].view(torch.int16), after[~sees].view(torch.int16))
    assert not torch.isfinite(after[sees].float()).all(dim=-1).any()


def test_a_visible_infinity_in_v_reaches_the_rows_that_see_it():
    """V of one node holds infinities in some dims: exactly the rows that see it are
    infinite there, and finite elsewhere."""
    T = 12
    c = Case([50], [T], 2, 1, 128, 16, seed=5)
    j, slot = 3, int(c.b.slot_mapping[3])
    c.pool[slot // 16, 1, 0, slot % 16, 10:20] = float("inf")
    got = c.run().float().cpu()
    for i in range(T):
        sees = j in _tree.path_to(c.up, i)
        assert bool((got[i, :, 10:20] == float("inf")).all()) == sees
        assert torch.isfinite(got[i, :, :10]).all() and torch.isfinite(got[i, :, 20:]).all()
        assert sees or torch.isfinite(got[i]).all()


@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("T", [9, 64])
def test_queries_of_zeros_tiny_huge_and_nan_rows(fp8, T):
    """Each query row has its own scale over an FP8 pool; a NaN or an infinity stays in
    its row (and head)."""
    c = Case([100, 700], [T, 5], 8, 2, 128, 16, seed=25, fp8=fp8, scale=1e-3)
    q = c.b.q
    q[1, 0] = 0.0
    q[2, 1] = 1e-39  # a subnormal: scores far below one
    q[3, 2] *= 1000.0
    q[4, 3, ::2] *= 2.0 ** -12  # elements far below the row's largest
    want, tol = c.reference()
    _tree.assert_attention(c.run(), want, tol)
    clean = q.clone()
    q[0, 4, 5], q[T, 7, 127], q[T + 1, 0, 0] = float("nan"), float("inf"), float("-inf")
    out = c.run()
    hit = torch.zeros(out.shape[:2], dtype=torch.bool)
    hit[0, 4] = hit[T, 7] = hit[T + 1, 0] = True
    assert out.cpu()[hit].isnan().all()
    q.copy_(clean)
    assert np.array_equal(bits(out.cpu()[~hit]), bits(c.run().cpu()[~hit]))


def test_an_infinity_or_nan_in_the_context_reaches_every_row():
    c = Case([200], [6], 2, 1, 64, 16, seed=6)
    blk, off = int(c.b.block_tables[0, 3]), 5
    c.pool[blk, 1, 0, off, 7] = float("inf")
    got = c.run().float()
    assert (got[:, :, 7] == float("inf")).all()
    assert torch.isfinite(got[:, :, :7]).all() and torch.isfinite(got[:, :, 8:]).all()
    c.pool[blk, 0, 0, off, 3] = float("nan")
    assert torch.isnan(c.run().float()).all()


def test_empty_trees_and_rows_behind_the_last_sequence_are_left_alone():
    """Sequences without drafts between others; q and out hold more rows than the
    trees."""
    T = [0, 5, 0, 3, 0]
    c = Case([9, 60, 0, 200, 128], T, 4, 2, 64, 16, seed=9)
    b = c.b
    q = torch.cat([b.q, torch.full((7, 4, 64), float("nan"), dtype=torch.bfloat16, device=DEV)])
    out = torch.full_like(q, 7.0)
    parents = ints(c.up + [99] * 7)
    c.run(out=out, q=q, parents=parents)
    _tree.assert_attention(out[:8], *c.reference())
    assert (out[8:] == 7.0).all()


def test_attention_gives_the_same_bits_on_every_call_and_in_every_batch_order():
    c = Case([700, 90, 4000], [9, 40, 16], 8, 2, 128, 16, seed=12)
    first = c.run()
    ws = c.workspace()
    for _ in range(3):
        ws.fill_(255)
        assert torch.equal(c.run(ws=ws).view(torch.int16), first.view(torch.int16))


def test_attention_flags_bad_data_and_skips_what_it_concerns():
    T = [4, 6, 5]
    c = Case([30, 40, 50], T, 4, 2, 64, 16, seed=13)
    want, tol = c.reference()
    # A length beyond the table, and one shorter than the tree: those sequences are skipped.
    for bad in (10 ** 6, 3, -5):
        lens = c.b.seq_lens.clone()
        lens[1] = bad
        out = c.run(out=torch.full_like(c.b.q, 7.0), seq_lens=lens)
        with pytest.raises(binding.PaError, match="OOB"):
            binding.pa_error_check()
        assert (out[4:10] == 7.0).all()
        _tree.assert_attention(out[:4], want[:4], tol[:4])
        _tree.assert_attention(out[10:], want[10:], tol[10:])
    # Parents that are no earlier node: such a node has no parent.
    up, plain = list(c.up), list(c.up)
    up[4 + 3], up[10 + 2] = 3, -7
    plain[4 + 3] = plain[10 + 2] = -1
    out = c.run(parents=ints(up))
    with pytest.raises(binding.PaError, match="OOB"):
        binding.pa_error_check()
    _tree.assert_attention(out, *c.reference(plain))
    # A block id outside the pool: flagged, the other sequences unharmed.
    c.b.block_tables[1, 0] = 10 ** 6
    out = c.run()
    with pytest.raises(binding.PaError, match="OOB"):
        binding.pa_error_check()
    _tree.assert_attention(out[:4], want[:4], tol[:4])
    _tree.assert_attention(out[10:], want[10:], tol[10:])
    # Offsets that are none: a tree larger than max_tree_len, decreasing, beyond the rows.
    c = Case([30, 40, 50], T, 4, 2, 64, 16, seed=13)
    for cu in ([0, 4, 3, 15], [0, 4, 10, 99], [0, 15, 15, 15]):
        c.b.cu_q_lens = ints(cu)
        c.run()
        with pytest.raises(binding.PaError, match="OOB"):
            binding.pa_error_check()


def test_attention_in_a_pool_beyond_32_bit_offsets():
    """Blocks at the far end of a pool of more than 2^32 bytes and 2^31 elements."""
    nb = (1 << 32) // (2 * 8 * 16 * 128 * 2) + 2000  # 4.1 GB and some
    c = Case([300, 90], [12, 30], 8, 8, 128, 16, seed=14)
    b = c.b
    big = torch.zeros((nb, 2, 8, 16, 128), dtype=torch.bfloat16, device=DEV)
    n = c.pool.shape[0]
    big[nb - n:] = c.pool
    want = c.run()
    c.pool = big
    b.block_tables = torch.where(b.block_tables >= 0, b.block_tables + (nb - n), -1)
    assert torch.equal(c.run().view(torch.int16), want.view(torch.int16))


def test_attention_on_a_side_stream_and_in_two_graphs():
    """A captured call replays on new queries and lengths; two graphs with workspaces
    of their own replay one after the other, and a call on another stream agrees."""
    a = Case([500, 30], [8, 21], 8, 2, 128, 16, seed=15)
    b = Case([60, 2000], [33, 5], 8, 2, 128, 16, seed=16)
    want = [a.run(), b.run()]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        other = a.run()
        ws = a.workspace()
    explicit = a.run(out=torch.empty_like(other), ws=ws, stream=side)
    torch.cuda.synchronize()
    assert torch.equal(other.view(torch.int16), want[0].view(torch.int16))
    assert torch.equal(explicit.view(torch.int16), want[0].view(torch.int16))
    graphs, outs = [], []
    for c in (a, b):
        out, ws = torch.empty_like(c.b.q), c.workspace()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            c.run(out=out, ws=ws)
        graphs.append((g, ws))
        outs.append(out)
    for _ in range(2):
        for (g, _), out, w in zip(graphs, outs, want):
            out.fill_(float("nan"))
            g.replay()
            torch.cuda.synchronize()
            assert torch.equal(out.view(torch.int16), w.view(torch.int16))
    # New data under the same graph: queries, and a shorter context.
    a.b.q.mul_(0.5)
    a.b.seq_lens.sub_(ints([16, 3]))
    graphs[0][0].replay()
    torch.cuda.synchronize()
    _tree.assert_attention(outs[0], *a.reference())


def test_attention_of_sequences_that_share_their_prefix_blocks():
    """The same blocks in every table, split contexts and tiles of the trees' own."""
    Case([1024 + c for c in (0, 5, 64, 700)], [3, 64, 17, 1], 8, 2, 128, 16, seed=17,
         shared_prefix_blocks=64).check()


@pytest.mark.parametrize("ctx_max,fp8", [(40, False), (40, True), (900, False)])
def test_attention_of_thousands_of_small_trees(ctx_max, fp8):
    """Batches of more sequences than workers, a fifth of them empty and padded."""
    rng = np.random.default_rng(18)
    B = 2500 if ctx_max == 40 else 600
    T = (rng.integers(0, 5, B)).tolist()
    ctx = [int(rng.integers(0, ctx_max + 1)) if t else 0 for t in T]
    Case(ctx, T, 2, 1, 128, 16, seed=18, fp8=fp8).check()


def test_tree_calls_beside_others_on_two_streams():
    """Calls that overlap on the GPU, with workspaces of their own, and the chunked prefill
    beside them: the same bits as one after the other."""
    a = Case([3000, 40, 900], [40, 64, 16], 8, 2, 128, 16, seed=19)
    b = Case([2000, 2100], [9, 12], 4, 4, 64, 16, seed=20)
    p = make_batch(name="chunks", seq_lens=[900, 300], q_lens=[600, 300], num_heads=8,
                   num_kv_heads=2, head_size=64, block_size=16, scale=0.125, seed=22, device=DEV)
    gpu_write(p)
    max_q = int(p.q_lens.max())
    d = _tree.random_drafts(23, [20, 3], 40000, True)
    args = [x.to(DEV) for x in (d.target, d.draft, d.tokens, d.cu, d.parents, d.accept_u,
                                d.sample_u)]
    acc = torch.empty(2, 20, dtype=I32, device=DEV)
    num, nxt = (torch.empty(2, dtype=I32, device=DEV) for _ in range(2))
    pre = torch.empty_like(p.q)

    def first(out, ws):
        a.run(out=out, ws=ws)
        binding.pa_tree_verify(acc, num, nxt, *args)
        a.run(out=out, ws=ws)

    def second(out, ws):
        b.run(out=out, ws=ws)
        binding.pa_prefill_chunk(pre, p.q, p.cu_q_lens, max_q, p.kv_cache, p.block_tables,
                                 p.seq_lens, p.scale)
        b.run(out=out, ws=ws)

    work = [(first, a), (second, b)]
    bufs = [(torch.empty_like(c.b.q), c.workspace()) for _, c in work]
    for (f, _), x in zip(work, bufs):
        f(*x)
    torch.cuda.synchronize()
    want = [x[0].clone() for x in bufs] + [pre.clone(), acc.clone(), num.clone(), nxt.clone()]
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(5):
        for t in (bufs[0][0], bufs[1][0], pre):
            t.fill_(float("nan"))
        acc.zero_()
        for s in streams:
            s.wait_stream(torch.cuda.current_stream())
        for _ in range(4):
            for s, (f, _), x in zip(streams, work, bufs):
                with torch.cuda.stream(s):
                    f(*x)
        torch.cuda.synchronize()
        got = [bufs[0][0], bufs[1][0], pre, acc, num, nxt]
        for g, w in zip(got, want):
            assert torch.equal(g.view(torch.int16), w.view(torch.int16))
    assert nxt.tolist() == d.reference[1]


@pytest.mark.parametrize("fp8", [False, True])
def test_attention_does_not_depend_on_what_ran_before(fp8):
    """The same bits whatever the calls before left in the chip's memories (rows without
    a query, places not yet written), for few rows in ranges of a few tiles."""
    others = [Case([700, 1500, 64, 900], [64, 40, 33, 20], 16, 2, 128, 16, seed=24, fp8=f,
                   q_mult=m) for f in (True, False) for m in (1.0, 30.0)]
    c = Case([2500] * 5, [3] * 5, 8, 8, 128, 16, seed=7, fp8=fp8, q_mult=2.0)
    ws, out = c.workspace(), torch.empty_like(c.b.q)
    work = [(o, o.workspace(), torch.empty_like(o.b.q)) for o in others]
    want = c.run(ws=ws)
    _tree.assert_attention(want, *c.reference())
    for i in range(80):
        o, ws_o, out_o = work[i % 4]
        o.run(out=out_o, ws=ws_o)
        out.fill_(float("nan"))
        c.run(out=out, ws=ws)
        assert torch.equal(out.view(torch.int16), want.view(torch.int16)), i


# ---------------------------------------------------------------- verification
def run_verify(d, stream=None, max_tree=None, pad=0):
    """The call's (paths, next tokens), checked for its padding."""
    B = len(d.tree_lens)
    mt = max(1, max(d.tree_lens)) if max_tree is None else max_tree
    acc = torch.full((B, mt), -9, dtype=I32, device=DEV)
    num, nxt = torch.full((B,), -9, dtype=I32, device=DEV), torch.full((B,), -9, dtype=I32,
                                                                      device=DEV)

    def rows(t):
        if t is None:
            return None
        wide = torch.full((t.shape[0], t.shape[1] + pad), float("nan"), device=DEV)
        wide[:, :t.shape[1]] = t.to(DEV)
        return wide[:, :t.shape[1]]
    binding.pa_tree_verify(acc, num, nxt, rows(d.target), rows(d.draft), d.tokens.to(DEV),
                           d.cu.to(DEV), d.parents.to(DEV), d.accept_u.to(DEV),
                           d.sample_u.to(DEV), stream=stream)
    acc, num = acc.cpu(), num.tolist()
    for s, n in enumerate(num):
        if n >= 0:
            assert (acc[s, n:] == -1).all() and (acc[s, :n] >= 0).all()
    return [acc[s, :max(n, 0)].tolist() for s, n in enumerate(num)], nxt.tolist()


@pytest.mark.parametrize("with_draft", [True, False])
@pytest.mark.parametrize("shape", ["chain", "star", "tree", "forest"])
@pytest.mark.parametrize("vocab", [1, 2, 31, 32, 33, 1000, 4099])
def test_verify_is_the_walk_in_64_bits(with_draft, shape, vocab):
    T = [1, 2, 64, 0, 7, 33, 16, 5, 0, 64, 3]
    for seed in range(3):
        d = _tree.random_drafts(100 * vocab + seed, T, vocab, with_draft, shape)
        assert run_verify(d) == d.reference


@pytest.mark.parametrize("with_draft", [True, False])
@pytest.mark.parametrize("B,T,vocab,pad", [(1, 6, 32000, 0), (1, 12, 160001, 3), (3, 4, 131072, 8),
                                           (40, 9, 50021, 1), (300, 5, 2000, 0)])
def test_verify_of_large_vocabularies_and_batches(with_draft, B, T, vocab, pad):
    d = _tree.random_drafts(B + vocab, [T] * B, vocab, with_draft, sharp=3.0)
    assert run_verify(d, pad=pad) == d.reference


def test_verify_rejections_down_to_nothing():
    """Equal distributions accept every draft; a draft with all its weight where the
    target has none is always rejected; nothing left to draw from falls back to the
    target's most likely token, the lowest of equals."""
    V = 70
    p = torch.full((4, V), 1.0 / V)
    q = p.clone()
    cu = torch.tensor([0, 4], dtype=I32)
    chain = torch.tensor([-1, 0, 1, 2], dtype=I32)
    star = torch.tensor([-1, 0, 0, 0], dtype=I32)
    u = torch.tensor([0.0, 0.999, 0.999, 0.999])
    d = _tree.Drafts(p, q, torch.tensor([0, 3, 4, 5], dtype=I32), chain, cu, u,
                     torch.tensor([0.5]), [4])
    paths, nxt = run_verify(d)
    assert paths == [[0, 1, 2, 3]] and nxt == d.reference[1]
    # All of the draft's weight on a token that the target never gives.
    p2, q2 = torch.zeros(4, V), torch.zeros(4, V)
    p2[:, 9], q2[:, 3] = 1.0, 1.0
    d = _tree.Drafts(p2, q2, torch.tensor([0, 3, 3, 3], dtype=I32), star, cu, u * 0,
                     torch.tensor([0.0]), [4])
    assert run_verify(d) == d.reference == ([[0]], [9])
    # Rejected although equal (u = 1 is outside its range): the residual is nothing.
    p3 = torch.zeros(4, V)
    p3[:, 20], p3[:, 40] = 0.5, 0.5
    d = _tree.Drafts(p3, p3.clone(), torch.tensor([0, 40, 40, 20], dtype=I32), star, cu,
                     torch.ones(4), torch.tensor([0.7]), [4])
    assert run_verify(d) == d.reference == ([[0]], [20])
    # Without probabilities: every token with weight was proposed and rejected.
    d = _tree.Drafts(p3, None, torch.tensor([0, 40, 20, 20], dtype=I32), star, cu,
                     torch.ones(4), torch.tensor([0.7]), [4])
    assert run_verify(d) == d.reference == ([[0]], [20])


@pytest.mark.parametrize("u", [0.0, 1.0, 0.99999994])
def test_verify_draws_at_the_ends_of_the_distribution(u):
    V = 999
    g = torch.Generator().manual_seed(4)
    p = torch.softmax(torch.randn(2, V, generator=g), 1)
    p[:, :5] = 0.0
    p[:, -7:] = 0.0
    d = _tree.Drafts(p, None, torch.zeros(2, dtype=I32), torch.tensor([-1, -1], dtype=I32),
                     torch.tensor([0, 1, 2], dtype=I32), torch.zeros(2), torch.full((2,), u),
                     [1, 1])
    got = run_verify(d)
    assert got == d.reference
    assert got[1] == ([5, 5] if u == 0.0 else [V - 8, V - 8])


def test_verify_flags_bad_data():
    T = [5, 4, 6]
    for what in ("token", "parent", "offsets"):
        d = _tree.random_drafts(3, T, 50, True, "star")
        if what == "token":
            d.tokens[7], d.tokens[11] = 50, -1
            assert run_verify(d) == d.reference
        elif what == "parent":
            d.parents[6], d.parents[12] = 2, -5
            got = run_verify(d)
            d.parents[6] = d.parents[12] = -1
            assert got == d.reference
        else:
            want = d.reference
            d.cu = torch.tensor([0, 5, 4, 15], dtype=I32)
            got = run_verify(d, max_tree=8)
            assert got[0][0] == want[0][0] and got[1][1] == got[1][2] == -9
        with pytest.raises(binding.PaError, match="OOB"):
            binding.pa_error_check()


def test_verify_takes_apart_rows_and_refuses_other_layouts():
    d = _tree.random_drafts(31, [4, 1], 40, True)
    args = [x.to(DEV) for x in (d.tokens, d.cu, d.parents, d.accept_u, d.sample_u)]
    acc = torch.empty(2, 4, dtype=I32, device=DEV)
    num, nxt = (torch.empty(2, dtype=I32, device=DEV) for _ in range(2))
    p, q = d.target.to(DEV), d.draft.to(DEV)

    def call(p, q):
        binding.pa_tree_verify(acc, num, nxt, p, q, *args)
        return nxt.tolist()
    wide = torch.zeros(5, 97, device=DEV)
    wide[:, 20:60] = q
    assert call(p, wide[:, 20:60]) == call(p, q) == d.reference[1]
    one = _tree.random_drafts(32, [1], 40, True)  # a single row's stride says nothing
    binding.pa_tree_verify(acc[:1], num[:1], nxt[:1], one.target.to(DEV).expand(1, 40), None,
                           *(x.to(DEV) for x in (one.tokens, one.cu, one.parents, one.accept_u,
                                                 one.sample_u)))
    assert nxt.tolist()[0] == one.reference[1][0]
    for bad in (q[:1].expand(5, 40), q.t().contiguous().t(), q.double(), q[:, :39], q[:4],
                q.cpu(), q.flatten(), q.half()):
        for pair in ((p, bad), (bad, q)):
            with pytest.raises(ValueError):
                call(*pair)


def test_verify_replays_in_a_graph_and_on_a_side_stream():
    T = [7, 30, 2]
    d = _tree.random_drafts(21, T, 5000, True)
    t, q, tok, cu, up = (x.to(DEV) for x in (d.target, d.draft, d.tokens, d.cu, d.parents))
    au, su = d.accept_u.to(DEV), d.sample_u.to(DEV)
    acc = torch.empty(3, 30, dtype=I32, device=DEV)
    num, nxt = torch.empty(3, dtype=I32, device=DEV), torch.empty(3, dtype=I32, device=DEV)
    run = lambda: binding.pa_tree_verify(acc, num, nxt, t, q, tok, cu, up, au, su)  # noqa: E731
    run()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for seed in range(3):
        e = _tree.random_drafts(30 + seed, T, 5000, True)
        for dst, src in ((t, e.target), (q, e.draft), (tok, e.tokens), (up, e.parents),
                         (au, e.accept_u), (su, e.sample_u)):
            dst.copy_(src)
        g.replay()
        torch.cuda.synchronize()
        paths, nexts = e.reference
        assert nxt.tolist() == nexts
        assert [acc[i, :n].tolist() for i, n in enumerate(num.tolist())] == paths
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        assert run_verify(d) == d.reference


# ---------------------------------------------------------------- acceptance
def paths_of(rng, T):
    return [sorted({0, *rng.integers(0, n, rng.integers(0, n + 1)).tolist()}) if n else []
            for n in T]


def run_accept(pool, paths, T, b, new=True, max_tree=64):
    acc = torch.full((len(T), max_tree), -1, dtype=I32)
    for s, p in enumerate(paths):
        acc[s, :len(p)] = torch.tensor(p, dtype=I32)
    lens = torch.full((len(T),), -9, dtype=I32, device=DEV) if new else None
    binding.pa_tree_accept(pool, acc.to(DEV), ints([len(p) for p in paths]), b.cu_q_lens,
                           b.block_tables, b.seq_lens, lens)
    return lens


def raw(pool):
    return pool.cpu().numpy() if pool.dtype == torch.uint8 else \
        pool.cpu().view(torch.int16).numpy()


@pytest.mark.parametrize("kv_heads,D,bs", [(1, 64, 8), (2, 128, 16), (5, 64, 32), (8, 128, 8)])
@pytest.mark.parametrize("fp8", [False, True])
def test_accept_moves_the_rows_and_nothing_else(kv_heads, D, bs, fp8):
    T = [5, 1, 64, 0, 17, 33, 64, 64]
    ctx = [20, 7, 0, 9, 130, 31, 100, 5]
    rng = np.random.default_rng(kv_heads * D)
    b = make_batch(name="acc", seq_lens=[c + t for c, t in zip(ctx, T)], q_lens=T,
                   num_heads=kv_heads, num_kv_heads=kv_heads, head_size=D, block_size=bs,
                   scale=1.0, seed=2, device=DEV)
    pool = fp8_pool_of(b) if fp8 else b.kv_cache
    if not fp8:
        gpu_write(b)
    paths = paths_of(rng, T)
    paths[6], paths[7] = list(range(64)), list(range(1, 64))  # nothing moves; everything does
    want, lens = _tree.accept(raw(pool), paths, b.block_tables.cpu().numpy(),
                              b.seq_lens.tolist(), T)
    got = run_accept(pool, paths, T, b)
    assert np.array_equal(raw(pool), want)
    assert np.array_equal(got.cpu().numpy(), lens)
    before = raw(pool).copy()
    run_accept(pool, [[0] if n else [] for n in T], T, b, new=False)
    assert np.array_equal(raw(pool), before)


def test_accept_skips_and_flags_lists_that_are_no_path():
    T = [6, 6, 6, 6, 6]
    b = make_batch(name="acc", seq_lens=[30] * 5, q_lens=T, num_heads=2, num_kv_heads=2,
                   head_size=64, block_size=16, scale=1.0, seed=3, device=DEV)
    gpu_write(b)
    paths = [[0, 2, 5], [0, 3, 3], [0, 6], [4, 2], [1, 3]]
    good = [paths[0], [], [], [], paths[4]]
    want, lens = _tree.accept(raw(b.kv_cache), good, b.block_tables.cpu().numpy(), [30] * 5, T)
    got = run_accept(b.kv_cache, paths, T, b)
    with pytest.raises(binding.PaError, match="OOB"):
        binding.pa_error_check()
    assert np.array_equal(raw(b.kv_cache), want)
    assert got.tolist() == [27, 30, 30, 30, 26]
    b.block_tables[0, 1] = -1  # the block that holds positions 16 .. 31
    before = raw(b.kv_cache).copy()
    run_accept(b.kv_cache, [paths[0], [], [], [], []], T, b)
    with pytest.raises(binding.PaError, match="OOB"):
        binding.pa_error_check()
    assert np.array_equal(raw(b.kv_cache), before)


# ---------------------------------------------------------------- a speculative step
@pytest.mark.parametrize("fp8", [False, True])
@pytest.mark.parametrize("graph", [False, True])
def test_a_speculative_step_leaves_the_cache_of_the_accepted_tokens(fp8, graph):
    """Write the trees' K/V, attend, verify, accept, all on the device (eager or
    captured): the attention is that of the plain implementation, and the cache then
    equals one into which only the accepted tokens were written, so that the decode
    of the next token gives the same bits over both."""
    T, V, D = [9, 1, 20, 64], 300, 128
    ctx = [100, 15, 0, 700]
    d = _tree.random_drafts(77, T, V, True, sharp=3.0)
    b = make_batch(name="step", seq_lens=[c + t for c, t in zip(ctx, T)], q_lens=T, num_heads=8,
                   num_kv_heads=2, head_size=D, block_size=16, scale=D ** -0.5, seed=41,
                   device=DEV)
    start = fp8_pool_of(b) if fp8 else b.kv_cache.clone()
    pool = start.clone()
    sc = _tree.FP8_SCALES if fp8 else None
    up = d.parents.to(DEV)
    ws = torch.empty(binding.pa_tree_attention_workspace_bytes(4, 64, 8, 2, D),
                     dtype=torch.uint8, device=DEV)
    out = torch.empty_like(b.q)
    acc = torch.empty(4, 64, dtype=I32, device=DEV)
    num, nxt, lens = (torch.empty(4, dtype=I32, device=DEV) for _ in range(3))
    t, q, tok, cu = (x.to(DEV) for x in (d.target, d.draft, d.tokens, d.cu))
    au, su = d.accept_u.to(DEV), d.sample_u.to(DEV)
    max_len = b.max_seq_len

    def write(to, slots):
        if fp8:
            binding.pa_cache_write_fp8(to, b.k_new, b.v_new, slots, *sc)
        else:
            binding.pa_cache_write(to, b.k_new, b.v_new, slots)

    def step():
        write(pool, b.slot_mapping)
        binding.pa_tree_attention(out, b.q, cu, up, 64, pool, b.block_tables, b.seq_lens,
                                  max_len, b.scale, ws, kv_scales=sc)
        binding.pa_tree_verify(acc, num, nxt, t, q, tok, cu, up, au, su)
        binding.pa_tree_accept(pool, acc, num, cu, b.block_tables, b.seq_lens, lens)

    step()
    if graph:
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        pool.copy_(start)
        out.fill_(float("nan"))
        num.zero_()
        g.replay()
    binding.pa_error_check()
    paths, nexts = d.reference
    assert nxt.tolist() == nexts
    assert [acc[i, :n].tolist() for i, n in enumerate(num.tolist())] == paths
    assert max(len(p) for p in paths) > 2
    written = start.clone()
    write(written, b.slot_mapping)
    _tree.assert_attention(out, *_tree.tree_attention(
        b.q, written, b.block_tables, b.seq_lens.tolist(), T, d.parents.tolist(), b.scale, sc))
    # Only the accepted tokens, written where they belong.
    slots, rows = torch.full_like(b.slot_mapping, -1), d.cu.tolist()
    for s, path in enumerate(paths):
        for i, p in enumerate(path):
            slots[rows[s] + p] = b.slot_mapping[rows[s] + i]
    alone = start.clone()
    write(alone, slots)
    qn = b.q[:4].contiguous()
    res = []
    for where in (pool, alone):
        o, w = torch.empty_like(qn), workspace_for(b)
        a = (o, qn, where, b.block_tables, lens, max_len, b.scale)
        binding.pa_decode_fp8(*a, *sc, w) if fp8 else binding.pa_decode(*a, w)
        res.append(bits(o))
    assert np.array_equal(res[0], res[1])
    assert lens.tolist() == [c + len(p) for c, p in zip(ctx, paths)]
