"""The 4-bit decode where numbers come to the ends of their ranges: tensor scales next to the
smallest, weights far below the largest, scores and factors beyond binary32."""

from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from paged_kv_cache_287_gb300 import binding
from tests import _fp4
from tests.test_gpu_fp4 import DEV, Batch, bf16, ints, np64

pytestmark = pytest.mark.gpu

# Lengths, query and KV heads, head size, block size: a segment's pieces in a warp of its own,
# merged in one CTA (a CTA per segment), and merged by the second kernel.
WARP = ([500] * 310, 16, 8, 64, 16)
CTA = ([3900, 4000], 8, 2, 128, 16)
SPLIT = ([20000], 16, 4, 128, 32)
SHAPES = pytest.mark.parametrize("shape", [WARP, CTA, SPLIT], ids=["warp", "cta", "split"])


def parts(b: Batch):
    """Views of a batch's pool: codes [blocks, heads, 2, bs, D / 2] and scales [.., D / 16]."""
    n = b.bs * b.d // 2
    return (b.pool[..., :n].unflatten(-1, (b.bs, b.d // 2)),
            b.pool[..., n:].unflatten(-1, (b.bs, b.d // 16)))


@SHAPES
@pytest.mark.parametrize("v_scale", [2.0 ** -126, 1e-40])
def test_v_scales_next_to_the_smallest(shape, v_scale):
    """The output is a normal number although v_scale over the sum of the weights is not."""
    b = Batch(*shape, seed=3)
    codes, sc = parts(b)
    codes[:, :, 1] &= 0x77  # V: no signs, the largest scales
    sc[:, :, 1].clamp_(min=0x7e)
    b.q *= 0.01  # nearly the same weight for all
    scales = (0.01, v_scale)
    out = b.run(scales=scales)
    assert (np64(out) > 100 * v_scale).all()
    b.check(out, scales=scales, seqs=range(0, len(b.lens), 37))


def tail_bound(p, v, out, n):
    """How far a kernel's row may be off whose scores are exact: the output's rounding to bf16
    (2^-8); P's rounding to f16, 2^-11 of a weight, or half a step of f16's smallest numbers,
    2^-25, where the largest weight is 2^11 or more; n tokens' sums, each of n / 8 (the weights
    of a lane) and n / 16 (a product's) additions rounded by 2^-24 and 2^-23 at most; 2^-17 for the
    exponential, its argument (up to 32, four roundings of 2^-24) and the merges."""
    mass = p @ np.abs(v)
    return (2.0 ** -8 * np.abs(out) + (2.0 ** -11 + n * 2.0 ** -26 + 2.0 ** -17) * mass
            + 2.0 ** -36 * p.max() * np.abs(v).sum(0) + 2.0 ** -133)


def peaked(shape, peak, level):
    """One key `level` powers of two above the others, whose V alone is not zero (and positive):
    the output is what the tail brings."""
    b = Batch(*shape, seed=5)
    codes, sc = parts(b)
    codes[:, :, 0], sc[:, :, 0] = 0, 0x38
    codes[:, :, 1] &= 0x77
    for s, n in enumerate(b.lens):
        at = peak % n
        blk, o = int(b.tables[s, at // b.bs]), at % b.bs
        codes[blk, :, 0, o], codes[blk, :, 1, o] = 0x77, 0
    b.q.fill_(1.0)
    return b, level * math.log(2.0) / (6 * b.d)


@SHAPES
@pytest.mark.parametrize("peak", [0, 77, -1])
@pytest.mark.parametrize("level", [12.3, 25.1, 27.6, 31.0])
def test_weights_far_below_the_largest(shape, peak, level):
    b, scale = peaked(shape, peak, level)
    scales = (1.0, 0.37)
    out = np64(b.run(scales=scales, scale=scale))
    binding.pa_error_check()
    for s in range(0, len(b.lens), 103):
        k, v = b.rows(s, scales)
        x = k[:, 0].sum(-1) * scale
        p = np.exp(x - x.max())
        p /= p.sum()
        for h in range(b.hq):
            vh = v[:, h * b.hkv // b.hq]
            want = p @ vh
            assert want.max() > 0
            off = np.abs(out[s, h] - want)
            assert (off <= tail_bound(p, vh, want, b.lens[s])).all(), (s, h, (off / want).max())


@pytest.mark.parametrize("level, near", [(25.1, False), (25.1, True), (0.0, True)])
def test_a_long_tail_in_one_warp(level, near):
    """131072 tokens to each warp of the GPU (the sequences share their blocks), one key far above
    the others, its V zero or beside theirs; and no key above the others."""
    n, hkv, d, bs = 131072, 8, 64, 32
    b, scale = peaked(([n], hkv, hkv, d, bs), 1000, level)
    codes, _ = parts(b)
    if near:
        blk, o = int(b.tables[0, 1000 // bs]), 1000 % bs
        codes[blk, :, 1, o] = 0x21
    warps = 16 * torch.cuda.get_device_properties(0).multi_processor_count
    count = -(-warps // hkv)
    q = torch.ones(count, hkv, d, dtype=torch.bfloat16, device=DEV)
    out = torch.empty_like(q)
    ws = torch.empty(binding.pa_decode_fp4_workspace_bytes(count, hkv, hkv, d),
                     dtype=torch.uint8, device=DEV)
    tables = b.tables.to(DEV).expand(count, -1).contiguous()
    binding.pa_decode_fp4(out, q, b.pool.to(DEV), tables, ints([n] * count), n, scale, 1.0, 0.37,
                          ws)
    binding.pa_error_check()
    k, v = b.rows(0, (1.0, 0.37))
    x = k[:, 0].sum(-1) * scale
    p = np.exp(x - x.max())
    p /= p.sum()
    got = np64(out)
    for h in range(hkv):
        want = p @ v[:, h]
        off = np.abs(got[:, h] - want)
        assert (off <= tail_bound(p, v[:, h], want, n)).all(), (h, (off / want).max())


def test_a_long_context_of_any_numbers():
    b = Batch([131072, 5], 4, 1, 128, 16, seed=6, q_mult=2.0)
    b.check(b.run())


@pytest.mark.parametrize("odd", [0, 1])
def test_no_weight_leaves_f16_where_scores_step_far(odd):
    """Scores so large that their own steps are `u` powers of two of weight: whatever the steps
    above the reference, the weights stay finite and the output between the values."""
    b = Batch(*WARP, seed=7)
    codes, sc = parts(b)
    codes[:, :, 0], sc[:, :, 0, :, 1:] = 0x77, 0x7e
    codes[:, :, 0, :, :8], sc[:, :, 0, :, :1] = 0, 0x08  # the first 16: steps of 2^-7
    for s, n in enumerate(b.lens):
        for blk, first in zip(b.tables[s].tolist(), range(0, n, b.bs)):
            step = odd + min(first // 96, 4)
            codes[blk, :, 0, :, 0] = step
    codes[:, :, 1] &= 0x77
    b.q.fill_(1.0)
    seqs = range(0, len(b.lens), 103)
    most = {s: np.abs(b.rows(s, (1.0, 1.0))[1]).max(0) for s in seqs}
    for u in (1.0, 2.0, 4.0, 7.5, 8.0, 12.0, 14.9, 15.0, 15.9, 15.9999, 16.0, 16.1, 24.0, 32.0, 64.0):
        out = np64(b.run(scales=(1.0, 1.0), scale=u * 128 * math.log(2.0)))
        for s in seqs:
            top = most[s].repeat(b.hq // b.hkv, 0)
            assert np.isfinite(out[s]).all(), (u, s)
            assert (out[s] >= 0).all() and (out[s] <= top * (1 + 2.0 ** -7)).all(), (u, s)


@SHAPES
@pytest.mark.parametrize("sign", [1, -1])
def test_scores_beyond_binary32(shape, sign):
    """The factor of a score is finite, the scores times it are not: the largest key takes all,
    whichever pieces its segment is merged from; also where every score is negative."""
    b = Batch(*shape, seed=11)
    b.q[:] = b.q[:, :1].abs() * 1e6
    codes, _ = parts(b)
    codes[:, :, 0] &= 0x77
    if sign < 0:
        codes[:, :, 0] |= 0x88
    out = np64(b.run(scales=(1.0, 0.37), scale=2e31))
    binding.pa_error_check()
    checked = 0
    for s in range(0, len(b.lens), 53):
        k, v = b.rows(s, (1.0, 0.37))
        for h in range(b.hq):
            kv = h * b.hkv // b.hq
            x = k[:, kv] @ np64(b.q[s])[h]
            top = np.sort(np.abs(x))
            top = top[:2] if sign < 0 else top[::-1][:2]
            if abs(top[0] - top[1]) < 1e-4 * top[1]:  # nearer than the fp32 sums tell apart
                continue
            want = v[x.argmax(), kv]
            assert (np.abs(out[s, h] - want) <= 2.0 ** -8 * np.abs(want)).all(), (s, h)
            checked += 1
    assert checked


@SHAPES
def test_a_small_factor_of_large_queries(shape):
    """scale * k_scale below binary32's normal numbers, the scores not."""
    b = Batch(*shape, seed=12)
    codes, sc = parts(b)
    codes[:] = codes[:, :, :1, :, :1] & 0x0f  # a row's elements are alike, K's and V's too
    codes |= codes << 4
    sc.clamp_(min=0x7e)
    b.q.fill_(2.0 ** 126)
    scales, scale = (1.34375 * 2.0 ** -73, 0.37), 1.3125 * 2.0 ** -73  # 20.4 steps of the smallest
    b.check(b.run(scales=scales, scale=scale), scales=scales, scale=scale,
            seqs=range(0, len(b.lens), 37))


@SHAPES
def test_a_large_factor_of_small_queries(shape):
    """scale * k_scale beyond binary32, the scores around one: queries of 2^-126 on keys of a
    single element of the smallest code and scale."""
    b = Batch(*shape, seed=13)
    codes, sc = parts(b)
    codes[:, :, 0, :, 1:], sc[:, :, 0] = 0, 0x01
    codes[:, :, 0, :, 0] &= 0x09  # element 0: 0, 0.5 and their negatives
    b.q.fill_(2.0 ** -126)
    scales, scale = (2.0 ** 30 / 3, 0.37), 2.0 ** 106 * 1.1
    b.check(b.run(scales=scales, scale=scale), scales=scales, scale=scale,
            seqs=range(0, len(b.lens), 37))


def test_every_attention_over_a_context_read_back_is_the_formula():
    """pa_decode and pa_prefill_chunk over the rows read back, pa_decode_fp4 over the pool itself:
    each against the formula over the numbers that it reads.  The bf16 kernels' P is rounded to
    bf16, 2^-8 of a weight."""
    gen = torch.Generator().manual_seed(23)
    n, hq, hkv, d, bs, nb = 333, 8, 2, 128, 16, 30
    sc = (0.0017, 0.0021)
    k, v = bf16((n, hkv, d), gen), bf16((n, hkv, d), gen)
    perm = torch.randperm(nb, generator=gen)[:21]
    slots = (perm[:, None] * bs + torch.arange(bs)).reshape(-1)[:n]
    pool = torch.zeros(binding.fp4_pool_shape(nb, hkv, bs, d), dtype=torch.uint8, device=DEV)
    binding.pa_cache_write_fp4(pool, k.to(DEV), v.to(DEV), ints(slots), *sc)
    kb, vb = (torch.empty(n, hkv, d, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    binding.pa_cache_read_fp4(kb, vb, pool, ints(slots), *sc)
    wide = torch.zeros(nb, 2, hkv, bs, d, dtype=torch.bfloat16, device=DEV)
    binding.pa_cache_write(wide, kb, vb, ints(slots))
    tables, lens = ints(perm)[None].contiguous(), ints([n])
    q = bf16((1, hq, d), gen, 2.0).to(DEV)
    out4, out16, chunk = (torch.empty_like(q) for _ in range(3))
    ws = torch.empty(max(binding.pa_decode_fp4_workspace_bytes(1, hq, hkv, d),
                         binding.pa_decode_workspace_bytes(1, hq, hkv, d)), dtype=torch.uint8,
                     device=DEV)
    scale = d ** -0.5
    binding.pa_decode_fp4(out4, q, pool, tables, lens, n, scale, *sc, ws)
    binding.pa_decode(out16, q, wide, tables, lens, n, scale, ws)
    binding.pa_prefill_chunk(chunk, q, ints([0, 1]), 1, wide, tables, lens, scale)
    binding.pa_error_check()
    q = np64(q[0])
    want, tol = _fp4.attend(q, *_fp4.read_rows(pool.cpu().numpy(), slots, bs, d, sc), scale, n)
    assert (np.abs(np64(out4[0]) - want) <= tol).all()
    assert tol.max() < np.abs(want).max() / 20
    k64, v64 = np64(kb), np64(vb)
    want, tol = _fp4.attend(q, k64, v64, scale, n)
    for h in range(hq):
        x = k64[:, h * hkv // hq] @ q[h] * scale
        p = np.exp(x - x.max())
        tol[h] += 2.0 ** -8 * (p / p.sum()) @ np.abs(v64[:, h * hkv // hq])
    assert tol.max() < np.abs(want).max() / 20
    for out in (out16, chunk):
        assert (np.abs(np64(out[0]) - want) <= tol).all()


@pytest.mark.parametrize("d, segs, tokens", [
    (128, 4, 1408), (128, 8, 1056), (128, 16, 768), (128, 32, 832), (128, 72, 2304),
    (128, 144, 4096), (64, 1, 4032), (64, 2, 3456), (64, 4, 2304), (64, 8, 1600), (64, 24, 1280),
    (64, 72, 4000)])
def test_both_sides_of_a_cta_per_segment(d, segs, tokens):
    """At the rule's border for 152 SMs and one token beyond: the tile more moves the batch to
    the other side, whose sums have another order, but not the result."""
    hkv = math.gcd(segs, 8)
    for n in (tokens, tokens + 1):
        b = Batch([n - (i % 3) * 7 for i in range(segs // hkv)], 2 * hkv, hkv, d, 16, seed=tokens)
        out = b.run()
        binding.pa_error_check()
        b.check(out, seqs=range(0, segs // hkv, 5))
