"""Draft trees without a GPU: the plain implementations are pinned (attention by
the oracle, verification by the distribution it must give, acceptance by the cache
write), and the calls refuse bad arguments before anything is enqueued."""

from __future__ import annotations

import ctypes
import os

import numpy as np
import pytest
import torch

import oracle
from paged_kv_cache_287_gb300 import binding
from paged_kv_cache_287_gb300.workloads import make_batch
from tests import _tree

FAKE = 1 << 20  # 16-byte aligned, never dereferenced: every call below fails host checks


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        from paged_kv_cache_287_gb300 import build
        build.build()
    return binding.lib()


# ---------------------------------------------------------------- the plain implementations
def test_chain_attention_is_the_oracles_causal_attention():
    T = [1, 5, 3]
    b = make_batch(name="chain", seq_lens=[9, 40, 3], q_lens=T, num_heads=4, num_kv_heads=2,
                   head_size=64, block_size=8, scale=0.125, seed=5)
    pool = oracle.cache_write(b.kv_cache, b.k_new, b.v_new, b.slot_mapping)
    want = oracle.attention(b.q, b.cu_q_lens, pool, b.block_tables, b.seq_lens, 4, 0.125)
    bf16 = torch.from_numpy(pool.view(np.int16)).view(torch.bfloat16).view(b.kv_cache.shape)
    up = sum((_tree.random_parents(None, n, "chain") for n in T), [])
    got, tol = _tree.tree_attention(b.q, bf16, b.block_tables, b.seq_lens, T, up, 0.125)
    np.testing.assert_allclose(got, want, rtol=0, atol=1e-12)
    assert (tol > 0).all()


def test_a_nodes_result_is_that_of_its_own_path():
    """Attention of node i of a tree equals that of the last row of the chain made
    of its path: siblings have no part in it."""
    rng = np.random.default_rng(3)
    n, ctx = 9, 13
    up = _tree.random_parents(rng, n)
    b = make_batch(name="tree", seq_lens=[ctx + n], q_lens=[n], num_heads=2, num_kv_heads=1,
                   head_size=64, block_size=8, scale=0.125, seed=6)
    pool = oracle.cache_write(b.kv_cache, b.k_new, b.v_new, b.slot_mapping)
    bf16 = torch.from_numpy(pool.view(np.int16)).view(torch.bfloat16).view(b.kv_cache.shape)
    got, _ = _tree.tree_attention(b.q, bf16, b.block_tables, b.seq_lens, [n], up, 0.125)
    tables = b.block_tables.numpy()
    for i in range(n):
        path = _tree.path_to(up, i)[::-1]
        bits, lens = _tree.accept(pool, [path], tables, [ctx + n], [n])
        row = oracle.attention(b.q[i:i + 1], np.array([0, 1], np.int32), bits, b.block_tables,
                               torch.from_numpy(lens), 2, 0.125)
        np.testing.assert_allclose(got[i], row[0], rtol=0, atol=1e-12)


@pytest.mark.parametrize("shape,with_draft", [("chain", True), ("star", True), ("star", False),
                                              ("tree", True), ("chain", False)])
def test_verified_tokens_follow_the_targets_distribution(shape, with_draft):
    """The token after the root (an accepted child's, or the next one) is distributed
    as p_root: counted over many draws of tokens and uniform numbers, within five
    standard deviations of a binomial count.  Without draft probabilities any fixed
    proposal must do."""
    V, N, T = 5, 20000, 4
    rng = np.random.default_rng(11 + 7 * with_draft + len(shape))
    up = _tree.random_parents(rng, T, shape)
    target = rng.dirichlet(np.ones(V), size=T)
    draft = rng.dirichlet(np.ones(V), size=T) if with_draft else None
    fixed = rng.integers(0, V, size=T)
    counts = np.zeros(V)
    for _ in range(N):
        tokens = [int(rng.choice(V, p=draft[max(u, 0)])) if with_draft else int(f)
                  for u, f in zip(up, fixed)]
        paths, nexts = _tree.verify(target, draft, tokens, [T], up, rng.random(T),
                                    rng.random(1))
        counts[tokens[paths[0][1]] if len(paths[0]) > 1 else nexts[0]] += 1
    p = target[0]
    assert (np.abs(counts - N * p) <= 5 * np.sqrt(N * p * (1 - p)) + 1).all(), (counts / N, p)


def test_accept_leaves_what_writing_the_accepted_rows_alone_would():
    rng = np.random.default_rng(8)
    T = [6, 1, 9]
    b = make_batch(name="acc", seq_lens=[20, 7, 9], q_lens=T, num_heads=2, num_kv_heads=2,
                   head_size=64, block_size=8, scale=1.0, seed=9)
    pool = oracle.cache_write(b.kv_cache, b.k_new, b.v_new, b.slot_mapping)
    paths = [sorted({0, *rng.integers(0, n, 3).tolist()}) for n in T]
    got, lens = _tree.accept(pool, paths, b.block_tables.numpy(), b.seq_lens.tolist(), T)
    cu, slots = b.cu_q_lens.tolist(), b.slot_mapping.clone()
    for s, path in enumerate(paths):
        for i, p in enumerate(path):
            slots[cu[s] + p] = int(b.slot_mapping[cu[s] + i])
        for j in set(range(T[s])) - set(path):
            slots[cu[s] + j] = -1
    want = oracle.cache_write(b.kv_cache, b.k_new, b.v_new, slots)
    for s, path in enumerate(paths):
        for pos in range(int(lens[s])):
            blk, off = int(b.block_tables[s, pos // 8]), pos % 8
            assert np.array_equal(got[blk, :, :, off], want[blk, :, :, off])
    assert lens.tolist() == [20 - 6 + len(paths[0]), 7, len(paths[2])]


# ---------------------------------------------------------------- refusals
def _attn(**kw):
    a = dict(out=FAKE, q=FAKE, cu=FAKE, parents=FAKE, num_seqs=3, total=9, max_tree=8, kv=FAKE,
             num_blocks=10, block_size=16, num_heads=32, num_kv_heads=8, head_size=128, bt=FAKE,
             max_blocks=4, seq_lens=FAKE, max_seq=64, scale=0.1, ws=FAKE, ws_bytes=1 << 40,
             stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("status,kw", [
    (1, dict(kv=None)), (1, dict(kv=FAKE + 2)), (1, dict(out=None)), (1, dict(out=FAKE + 8)),
    (1, dict(q=None)), (1, dict(q=FAKE + 8)), (1, dict(cu=None)), (1, dict(cu=FAKE + 2)),
    (1, dict(parents=None)), (1, dict(parents=FAKE + 1)), (1, dict(bt=None)),
    (1, dict(seq_lens=None)), (1, dict(seq_lens=FAKE + 2)), (1, dict(num_seqs=-1)),
    (1, dict(total=-1)), (1, dict(max_tree=0)), (2, dict(max_tree=65)),
    (1, dict(max_blocks=0)), (1, dict(max_seq=65)), (1, dict(max_seq=-1)),
    (1, dict(scale=float("nan"))), (1, dict(scale=float("inf"))), (1, dict(num_kv_heads=5)),
    (2, dict(num_heads=64, num_kv_heads=4)), (2, dict(head_size=96)), (2, dict(block_size=12)),
    (6, dict(ws=None)), (6, dict(ws=FAKE + 64)), (6, dict(ws_bytes=1)),
    (2, dict(num_seqs=1 << 20, max_blocks=1 << 16)),
    (0, dict(num_seqs=0)), (0, dict(total=0))])
def test_tree_attention_host_checks(lib, status, kw):
    assert lib.pa_tree_attention(*_attn(**kw)) == status
    a8 = _attn(**kw)
    assert lib.pa_tree_attention_fp8(*a8[:18], 0.5, 0.25, *a8[18:]) == status


def test_tree_attention_fp8_host_checks(lib):
    for ks, vs in ((0.0, 1.0), (1.0, -1.0), (float("inf"), 1.0), (1.0, float("nan"))):
        a = _attn()
        assert lib.pa_tree_attention_fp8(*a[:18], ks, vs, *a[18:]) == 1
    a = _attn(head_size=64)
    assert lib.pa_tree_attention_fp8(*a[:18], 0.5, 0.5, *a[18:]) == 2
    w = lib.pa_tree_attention_workspace_bytes
    assert w(4, 16, 32, 8, 128) > 0
    assert w(4, 65, 32, 8, 128) == w(4, 0, 32, 8, 128) == w(-1, 4, 32, 8, 128) == 0
    assert w(4, 16, 30, 8, 128) == w(4, 16, 32, 8, 96) == w(4, 16, 128, 8, 128) == 0


def _verify(**kw):
    a = dict(accepted=FAKE, num=FAKE, next=FAKE, target=FAKE, ts=100, draft=FAKE, ds=100,
             tokens=FAKE, cu=FAKE, parents=FAKE, num_seqs=3, total=9, max_tree=8, vocab=100,
             accept_u=FAKE, sample_u=FAKE, stream=None)
    a.update(kw)
    return list(a.values())


@pytest.mark.parametrize("status,kw", [
    (1, dict(accepted=None)), (1, dict(num=None)), (1, dict(next=None)), (1, dict(target=None)),
    (1, dict(target=FAKE + 2)), (1, dict(draft=FAKE + 2)), (1, dict(ts=99)), (1, dict(ds=99)),
    (1, dict(tokens=None)), (1, dict(cu=None)), (1, dict(parents=None)),
    (1, dict(accept_u=None)), (1, dict(sample_u=None)), (1, dict(vocab=0)),
    (2, dict(vocab=(1 << 20) + 1, ts=1 << 21, ds=1 << 21)), (1, dict(num_seqs=-1)),
    (1, dict(total=-1)), (1, dict(max_tree=0)), (2, dict(max_tree=65)), (0, dict(num_seqs=0))])
def test_tree_verify_host_checks(lib, status, kw):
    assert lib.pa_tree_verify(*_verify(**kw)) == status


@pytest.mark.parametrize("status,kw", [
    (1, dict(kv=None)), (1, dict(kv=FAKE + 8)), (1, dict(accepted=None)), (1, dict(num=None)),
    (1, dict(cu=None)), (1, dict(bt=None)), (1, dict(seq_lens=None)), (1, dict(new=FAKE)),
    (1, dict(new=FAKE + 2)), (1, dict(num_seqs=-1)), (1, dict(max_blocks=0)),
    (1, dict(max_tree=0)), (2, dict(max_tree=65)), (2, dict(head_size=32)),
    (0, dict(num_seqs=0))])
def test_tree_accept_host_checks(lib, status, kw):
    a = dict(kv=FAKE, num_blocks=10, block_size=16, num_kv_heads=8, head_size=128, accepted=FAKE,
             num=FAKE, cu=FAKE, num_seqs=3, max_tree=8, bt=FAKE, max_blocks=4, seq_lens=FAKE,
             new=None, stream=None)
    a.update(kw)
    assert lib.pa_tree_accept(*a.values()) == status
    assert lib.pa_tree_accept_fp8(*a.values()) == status


def test_tree_bindings_name_the_tensor_at_fault(lib):
    """Host tensors: no call reaches the library."""
    d = _tree.random_drafts(1, [3, 2], 7, True)
    i32 = torch.int32
    acc, num, nxt = (torch.empty(2, 3, dtype=i32), torch.empty(2, dtype=i32),
                     torch.empty(2, dtype=i32))
    with pytest.raises(ValueError, match="accepted must be a CUDA tensor"):
        binding.pa_tree_verify(acc, num, nxt, d.target, d.draft, d.tokens, d.cu, d.parents,
                               d.accept_u, d.sample_u)
    pool = torch.zeros(4, 2, 1, 8, 64, dtype=torch.bfloat16)
    bt, sl = torch.zeros(2, 2, dtype=i32), torch.ones(2, dtype=i32)
    with pytest.raises(ValueError, match="kv_cache must be a CUDA tensor"):
        binding.pa_tree_accept(pool, acc, num, d.cu, bt, sl)
    q = torch.zeros(5, 4, 64, dtype=torch.bfloat16)
    ws = torch.empty(256, dtype=torch.uint8)
    with pytest.raises(ValueError, match="kv_cache must be a CUDA tensor"):
        binding.pa_tree_attention(q, q, d.cu, d.parents, 3, pool, bt, sl, 8, 0.1, ws)
    with pytest.raises(ValueError, match="kv_scales"):
        binding.pa_tree_attention(q, q, d.cu, d.parents, 3, pool.to(torch.uint8), bt, sl, 8, 0.1,
                                  ws)


def _packed(lib, call, values):
    """The packed call of these members (pointers None or int)."""
    buf = ctypes.create_string_buffer(lib.pa_tree_args_bytes(call))
    binding.TREE_ARGS[call].pack_into(buf, 0, *(0 if v is None else v for v in values))
    f = (lib.pa_tree_attention_packed, lib.pa_tree_verify_packed, lib.pa_tree_accept_packed)[call]
    return f(ctypes.addressof(buf))


def test_packed_structs_have_the_headers_layout(lib):
    assert [lib.pa_tree_args_bytes(i) for i in (0, 1, 2, 3, -1)] == [136, 120, 96, 0, 0]
    for f in (lib.pa_tree_attention_packed, lib.pa_tree_verify_packed, lib.pa_tree_accept_packed):
        assert f(None) == 1


@pytest.mark.parametrize("kw", [
    dict(kv=None), dict(out=None), dict(q=FAKE + 8), dict(cu=None), dict(parents=None),
    dict(bt=None), dict(seq_lens=None), dict(num_seqs=-1), dict(total=-1), dict(max_tree=0),
    dict(max_tree=65), dict(max_blocks=0), dict(max_seq=65), dict(scale=float("nan")),
    dict(num_kv_heads=5), dict(num_heads=64, num_kv_heads=4), dict(head_size=96),
    dict(block_size=12), dict(ws=None), dict(ws_bytes=1), dict(num_seqs=0), dict(total=0),
    dict(num_blocks=0)])
def test_packed_tree_attention_decides_as_the_plain_call(lib, kw):
    """Each case is decided by another member."""
    a = dict(zip(("out", "q", "cu", "parents", "num_seqs", "total", "max_tree", "kv", "num_blocks",
                  "block_size", "num_heads", "num_kv_heads", "head_size", "bt", "max_blocks",
                  "seq_lens", "max_seq", "scale", "ws", "ws_bytes", "stream"), _attn(**kw)))
    names = ("out q cu parents kv bt seq_lens ws ws_bytes stream num_seqs total max_tree "
             "num_blocks block_size num_heads num_kv_heads head_size max_blocks max_seq").split()
    members = [a[n] for n in names]
    b = _attn(**kw)
    assert _packed(lib, 0, members + [0, a["scale"], 1.0, 1.0]) == lib.pa_tree_attention(*b)
    assert _packed(lib, 0, members + [1, a["scale"], 0.5, 0.25]) == \
        lib.pa_tree_attention_fp8(*b[:18], 0.5, 0.25, *b[18:])


@pytest.mark.parametrize("kw", [
    dict(num_seqs=0), dict(accepted=None), dict(num=None), dict(next=None), dict(target=FAKE + 2),
    dict(draft=FAKE + 2), dict(ts=99), dict(ds=99), dict(tokens=None), dict(cu=None),
    dict(parents=None), dict(accept_u=None), dict(sample_u=None), dict(max_tree=65),
    dict(vocab=0), dict(total=-1), dict(num_seqs=-1)])
def test_packed_tree_verify_decides_as_the_plain_call(lib, kw):
    a = dict(zip(("accepted num next target ts draft ds tokens cu parents num_seqs total max_tree "
                  "vocab accept_u sample_u stream").split(), _verify(**kw)))
    names = ("accepted num next target draft tokens cu parents accept_u sample_u stream ts ds "
             "num_seqs total max_tree vocab").split()
    assert _packed(lib, 1, [a[n] for n in names]) == lib.pa_tree_verify(*_verify(**kw))


@pytest.mark.parametrize("kw", [
    dict(num_seqs=0), dict(kv=FAKE + 8), dict(accepted=None), dict(num=None), dict(cu=None),
    dict(bt=None), dict(seq_lens=None), dict(new=FAKE), dict(num_seqs=-1), dict(max_blocks=0),
    dict(max_tree=65), dict(head_size=32), dict(block_size=12), dict(num_kv_heads=0),
    dict(num_blocks=0)])
def test_packed_tree_accept_decides_as_the_plain_call(lib, kw):
    a = dict(kv=FAKE, num_blocks=10, block_size=16, num_kv_heads=8, head_size=128, accepted=FAKE,
             num=FAKE, cu=FAKE, num_seqs=3, max_tree=8, bt=FAKE, max_blocks=4, seq_lens=FAKE,
             new=None, stream=None)
    a.update(kw)
    names = ("kv accepted num cu bt seq_lens new stream num_blocks block_size num_kv_heads "
             "head_size num_seqs max_tree max_blocks").split()
    for kv8 in (0, 1):
        want = (lib.pa_tree_accept_fp8 if kv8 else lib.pa_tree_accept)(*a.values())
        assert _packed(lib, 2, [a[n] for n in names] + [kv8]) == want
