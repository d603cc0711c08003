"""The 4-bit pool's calls and the rotation on a GB300 against the plain definitions (64 bits;
the quantiser's binary32 steps bit for bit)."""

from __future__ import annotations

import math

import numpy as np
import pytest
import torch

from paged_kv_cache_287_gb300 import binding
from tests import _fp4

pytestmark = pytest.mark.gpu
DEV = "cuda"
SCALES = (0.0023, 1 / 3)  # k_scale, v_scale: neither a power of two


def bf16(shape, gen, mult=1.0):
    return (torch.randn(shape, generator=gen) * mult).to(torch.bfloat16)


def ints(x):
    return torch.as_tensor(x, dtype=torch.int32, device=DEV)


def np64(t):
    return t.float().cpu().numpy().astype(np.float64)


def random_pool(nb, hkv, bs, d, gen, nan_share=0.0):
    """A pool of any codes and moderate scales, on the CPU."""
    pool = torch.randint(0, 256, binding.fp4_pool_shape(nb, hkv, bs, d), dtype=torch.uint8,
                         generator=gen)
    n = bs * d // 2
    sc = torch.randint(0x20, 0x60, pool[..., n:].shape, dtype=torch.uint8, generator=gen)
    if nan_share:
        sc[torch.rand(sc.shape, generator=gen) < nan_share] = 0x7f
    pool[..., n:] = sc
    return pool


# ------------------------------------------------------------------ rows in and out
@pytest.mark.parametrize("d, bs, hkv, n", [(128, 16, 8, 37), (64, 8, 4, 1), (128, 32, 1, 129),
                                           (64, 16, 3, 64), (128, 8, 2, 2048), (64, 32, 5, 7)])
def test_write_is_the_definition_bit_for_bit(d, bs, hkv, n):
    gen = torch.Generator().manual_seed(n)
    nb = -(-n // bs) + 3
    pool = random_pool(nb, hkv, bs, d, gen)
    k, v = bf16((n, hkv, d), gen), bf16((n, hkv, d), gen, 300.0)
    slots = torch.randperm(nb * bs, generator=gen)[:n].to(torch.int32)
    slots[::5] = -1  # padding
    want = pool.numpy().copy()
    _fp4.write_rows(want, k, v, slots.tolist(), bs, SCALES)
    got = pool.to(DEV)
    binding.pa_cache_write_fp4(got, k.to(DEV), v.to(DEV), slots.to(DEV), *SCALES)
    binding.pa_error_check()
    assert np.array_equal(got.cpu().numpy(), want)


@pytest.mark.parametrize("g", [1.0, 1 / 64, 0.0019, 1e-40, 2.0 ** -126, 2.0 ** 120, 7e30])
def test_write_of_every_kind_of_number(g):
    """Every bf16 number as the largest of its group, ties, zeros, infinities and NaNs beside
    others, at ordinary, tiny and huge tensor scales."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16)
    first = bits.view(torch.bfloat16)
    # A group: the number, fractions of it (steps and ties of the code), and others.
    f = torch.tensor([1, 1 / 24, 1 / 12, 1 / 8, 1 / 6, 5 / 24, 0.25, 7 / 24, 1 / 3, 5 / 12, 0.5,
                      7 / 12, 2 / 3, 5 / 6, -0.125, -1.0])
    group = (first.float()[:, None] * f).to(torch.bfloat16)
    other = group[torch.randperm(65536, generator=torch.Generator().manual_seed(1))]
    k = torch.cat([group, other], 1).reshape(-1, 1, 128)
    v = torch.cat([group[:, :8], other[:, :8]], 1).reshape(-1, 1, 128)
    v = torch.cat([v, v])[:k.shape[0]]
    n, bs = k.shape[0], 32
    pool = torch.zeros(binding.fp4_pool_shape(n // bs, 1, bs, 128), dtype=torch.uint8)
    want = pool.numpy().copy()
    slots = torch.arange(n, dtype=torch.int32)
    _fp4.write_rows(want, k, v, slots.tolist(), bs, (g, 1.0))
    got = pool.to(DEV)
    if g == 2.0 ** 120:  # its largest element, 2688 g, is no finite fp32 number: refused
        with pytest.raises(binding.PaError, match="INVALID"):
            binding.pa_cache_write_fp4(got, k.to(DEV), v.to(DEV), slots.to(DEV), g, 1.0)
        return
    binding.pa_cache_write_fp4(got, k.to(DEV), v.to(DEV), slots.to(DEV), g, 1.0)
    assert np.array_equal(got.cpu().numpy(), want)


def test_write_at_many_tensor_scales():
    """Scales of few bits and of many, values whose quotients meet ties again and again."""
    gen = torch.Generator().manual_seed(30)
    scales = [2.0 ** e for e in (-30, -9, 0, 7)] + [3.0, 0.75, 1 / 3, 0.1, 5 / 2688, 0.7, 1.1e-3]
    n, bs = 256, 32
    k = bf16((n, 2, 128), gen)
    k[::2] = (k[::2].float() * 8).round().to(torch.bfloat16) / 8
    for a, b in zip(scales, scales[1:] + scales[:1]):
        kk = (k.float() * a * 200).to(torch.bfloat16)
        v = (k.float() * b).to(torch.bfloat16)
        pool = torch.zeros(binding.fp4_pool_shape(n // bs, 2, bs, 128), dtype=torch.uint8)
        want = pool.numpy().copy()
        _fp4.write_rows(want, kk, v, range(n), bs, (a, b))
        got = pool.to(DEV)
        binding.pa_cache_write_fp4(got, kk.to(DEV), v.to(DEV), ints(range(n)), a, b)
        assert np.array_equal(got.cpu().numpy(), want), (a, b)


@pytest.mark.parametrize("scales", [(1.0, 2.0 ** -6), (1 / 3, 0.0123), (1e-35, 1e35),
                                    (2.0 ** 100, 2.0 ** -126), (1e-40, 3.3)])
def test_rope_into_an_fp8_pool_at_many_scales(scales):
    t = Turn(40, 4, 2, 128, 16, 64, norm=(False, False), seed=9)
    t.wide[1] *= 1e30
    t.wide[2] *= 1e-30
    t.wide[4, 3] = math.inf
    t.wide[5, 7] = math.nan
    _, pool16 = t.run()
    t.bits = 8
    start = torch.zeros(pool16.shape, dtype=torch.uint8, device=DEV)
    _, pool = t.run(pool=start.clone(), scales=scales)
    slot = t.slots.clamp(min=0).long()
    k, v = (pool16[slot // 16, side, :, slot % 16].contiguous() for side in (0, 1))
    binding.pa_cache_write_fp8(start, k, v, t.slots.to(DEV), *scales)
    assert torch.equal(pool, start)


def test_write_of_strided_rows_leaves_the_rest():
    gen = torch.Generator().manual_seed(8)
    n, hkv, d, bs = 21, 2, 64, 8
    qkv = bf16((n, (6 + 2 * hkv) * d + 24), gen).to(DEV)
    k = qkv[:, 6 * d:8 * d].unflatten(1, (hkv, d))
    v = qkv[:, 8 * d:10 * d].unflatten(1, (hkv, d))
    pool = random_pool(9, hkv, bs, d, gen)
    slots = torch.randperm(72, generator=gen)[:n].to(torch.int32)
    want = pool.numpy().copy()
    _fp4.write_rows(want, k.cpu(), v.cpu(), slots.tolist(), bs, SCALES)
    got = pool.to(DEV)
    binding.pa_cache_write_fp4(got, k, v, slots.to(DEV), *SCALES)
    assert np.array_equal(got.cpu().numpy(), want)


def test_slots_beyond_the_pool_are_flagged_and_skipped():
    gen = torch.Generator().manual_seed(9)
    pool = random_pool(3, 2, 16, 128, gen)
    k, v = bf16((4, 2, 128), gen), bf16((4, 2, 128), gen)
    slots = [5, 48, 2 ** 31 - 1, 47]
    want = pool.numpy().copy()
    _fp4.write_rows(want, k, v, slots, 16, SCALES)
    got = pool.to(DEV)
    binding.pa_cache_write_fp4(got, k.to(DEV), v.to(DEV), ints(slots), *SCALES)
    with pytest.raises(binding.PaError, match="OOB"):
        binding.pa_error_check()
    assert np.array_equal(got.cpu().numpy(), want)
    ko, vo = (torch.full((4, 2, 128), 7.0, dtype=torch.bfloat16, device=DEV) for _ in range(2))
    binding.pa_cache_read_fp4(ko, vo, got, ints(slots), *SCALES)
    with pytest.raises(binding.PaError, match="OOB"):
        binding.pa_error_check()
    assert (ko[1:3] == 7).all() and (vo[1:3] == 7).all() and not (ko[[0, 3]] == 7).all()
    binding.pa_error_check()


@pytest.mark.parametrize("d, bs, hkv, n", [(128, 16, 8, 517), (64, 8, 4, 1), (128, 32, 2, 33),
                                           (64, 32, 3, 1000)])
def test_read_gives_the_values(d, bs, hkv, n):
    gen = torch.Generator().manual_seed(n)
    pool = random_pool(40, hkv, bs, d, gen, nan_share=0.01)
    slots = torch.randint(0, 40 * bs, (n,), generator=gen)  # some slots several times
    slots[1::7] = -3
    ko, vo = (torch.full((n, hkv + 1, d), 7.0, dtype=torch.bfloat16, device=DEV)[:, :hkv]
              for _ in range(2))
    binding.pa_cache_read_fp4(ko, vo, pool.to(DEV), ints(slots), *SCALES)
    binding.pa_error_check()
    for got, want in zip((ko, vo), _fp4.read_rows(pool.numpy(), slots.clamp(min=0), bs, d,
                                                  SCALES)):
        want = _fp4.bf16_of_product(want)
        want[1::7] = 7.0
        assert torch.equal(got.cpu().nan_to_num(nan=1e30), want.nan_to_num(nan=1e30))
        assert (got._base[:, hkv:] == 7).all()


@pytest.mark.parametrize("hkv, d, shift", [(40, 128, 8), (255, 64, 0), (40, 128, 16), (3, 64, 24)])
def test_many_heads_and_rows_off_the_wide_boundary(hkv, d, shift):
    """More columns than a block has threads; rows 16 bytes off a 32-byte boundary."""
    gen = torch.Generator().manual_seed(hkv)
    n, bs = 11, 16
    wide = bf16((2, n, hkv * d + 32), gen)
    k, v = (x[:, shift:shift + hkv * d].unflatten(1, (hkv, d)) for x in wide)
    kd, vd = (x[:, shift:shift + hkv * d].unflatten(1, (hkv, d)) for x in wide.to(DEV))
    pool = random_pool(4, hkv, bs, d, gen)
    slots = torch.randperm(64, generator=gen)[:n]
    want = pool.numpy().copy()
    _fp4.write_rows(want, k, v, slots.tolist(), bs, SCALES)
    got = pool.to(DEV)
    binding.pa_cache_write_fp4(got, kd, vd, ints(slots), *SCALES)
    assert np.array_equal(got.cpu().numpy(), want)
    back = torch.full(wide.shape, 7.0, dtype=torch.bfloat16, device=DEV)
    kb, vb = (x[:, shift:shift + hkv * d].unflatten(1, (hkv, d)) for x in back)
    binding.pa_cache_read_fp4(kb, vb, got, ints(slots), *SCALES)
    for x, y in zip((kb, vb), _fp4.read_rows(want, slots.numpy(), bs, d, SCALES)):
        assert torch.equal(x.cpu(), _fp4.bf16_of_product(y))
    assert (back[:, :, :shift] == 7).all() and (back[:, :, shift + hkv * d:] == 7).all()
    binding.pa_error_check()


def test_no_rows_are_a_no_op():
    pool = random_pool(2, 1, 16, 64, torch.Generator().manual_seed(1)).to(DEV)
    rows = torch.empty(0, 1, 64, dtype=torch.bfloat16, device=DEV)
    before = pool.clone()
    binding.pa_cache_write_fp4(pool, rows, rows, ints([]), *SCALES)
    binding.pa_cache_read_fp4(rows, rows, pool, ints([]), *SCALES)
    assert torch.equal(pool, before)


def test_every_code_and_scale_reads_back():
    pool = torch.zeros(binding.fp4_pool_shape(32, 1, 8, 64), dtype=torch.uint8)
    row = torch.arange(512).view(32, 1, 2, 8, 1)
    pool[..., :256].unflatten(3, (8, 32))[:] = (row + torch.arange(32) * 7).to(torch.uint8)
    pool[..., 256:].unflatten(3, (8, 4))[:] = (row * 3 + torch.arange(4)).to(torch.uint8)
    slots = torch.arange(256)
    for scales_ in ((1.0, 2.0 ** -120), (3e38 / 448 / 6, 1e-40)):
        out = [torch.empty(256, 1, 64, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
        binding.pa_cache_read_fp4(*out, pool.to(DEV), ints(slots), *scales_)
        for got, want in zip(out, _fp4.read_rows(pool.numpy(), slots, 8, 64, scales_)):
            want = _fp4.bf16_of_product(want)
            assert torch.equal(got.cpu().nan_to_num(nan=1e30), want.nan_to_num(nan=1e30))


# ------------------------------------------------------------------ attention
class Batch:
    """A decoding batch over a random pool whose free slots hold NaN."""

    def __init__(self, lens, hq, hkv, d, bs, seed=0, q_mult=1.0, extra_blocks=3, table_pad=1,
                 shared=0):
        gen = torch.Generator().manual_seed(seed)
        need = [-(-n // bs) for n in lens]
        self.nb = sum(need) + extra_blocks
        pool = random_pool(self.nb, hkv, bs, d, gen)
        perm = torch.randperm(self.nb, generator=gen).to(torch.int32)
        tables = torch.full((len(lens), max(need + [1]) + table_pad), -1, dtype=torch.int32)
        at = 0
        n_codes = bs * d // 2
        sc = pool[..., n_codes:].view(self.nb, hkv, 2, bs, d // 16)
        free = torch.ones(self.nb, bs, dtype=torch.bool)
        for s, n in enumerate(lens):
            tables[s, :need[s]] = perm[at:at + need[s]]
            if shared and s:
                tables[s, :min(shared, need[s])] = tables[0, :min(shared, need[s])]
            at += need[s]
            for b in range(need[s]):
                free[tables[s, b], :max(0, min(bs, n - b * bs))] = False
        sc.masked_fill_(free[:, None, None, :, None], 0x7f)
        self.lens, self.hq, self.hkv, self.d, self.bs = lens, hq, hkv, d, bs
        self.pool, self.tables = pool, tables
        self.q = bf16((len(lens), hq, d), gen, q_mult)
        self.scale = 1 / math.sqrt(d)

    def workspace(self, fill=None):
        n = binding.pa_decode_fp4_workspace_bytes(len(self.lens), self.hq, self.hkv, self.d)
        w = torch.empty(n, dtype=torch.uint8, device=DEV)
        return w if fill is None else w.fill_(fill)

    def run(self, max_len=None, scales=SCALES, scale=None, fill=0xff):
        out = torch.full(self.q.shape, math.nan, dtype=torch.bfloat16, device=DEV)
        binding.pa_decode_fp4(out, self.q.to(DEV), self.pool.to(DEV), self.tables.to(DEV),
                              ints(self.lens), max(self.lens) if max_len is None else max_len,
                              self.scale if scale is None else scale, *scales,
                              self.workspace(fill))
        return out

    def rows(self, s, scales=SCALES):
        pos = np.arange(max(0, self.lens[s]))
        slots = self.tables[s].numpy()[pos // self.bs] * self.bs + pos % self.bs
        return _fp4.read_rows(self.pool.numpy(), slots, self.bs, self.d, scales)

    def check(self, out, scales=SCALES, scale=None, seqs=None):
        got = np64(out)
        for s in range(len(self.lens)) if seqs is None else seqs:
            want, tol = _fp4.attend(np64(self.q[s]), *self.rows(s, scales),
                                    self.scale if scale is None else scale, self.lens[s])
            off = np.abs(got[s] - want)
            assert (off <= tol).all(), (s, self.lens[s], off.max(), (off / tol).max())


LENGTHS = [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 63, 64, 65, 100, 127, 128, 129, 300]


@pytest.mark.parametrize("d, bs", [(128, 16), (128, 8), (128, 32), (64, 16), (64, 8), (64, 32)])
@pytest.mark.parametrize("hq, hkv", [(8, 2), (8, 1), (3, 3)])
def test_decode_ragged(d, bs, hq, hkv):
    b = Batch(LENGTHS, hq, hkv, d, bs, seed=d + bs + hq)
    out = b.run()
    binding.pa_error_check()
    b.check(out)
    assert (out[0] == 0).all()


@pytest.mark.parametrize("group", [1, 2, 3, 4, 5, 6, 7, 8])
def test_decode_every_group(group):
    for d in (64, 128):
        b = Batch([77, 1, 40, 205], group * 2, 2, d, 16, seed=group)
        b.check(b.run())


@pytest.mark.parametrize("lens, hq, hkv, d, bs", [
    ([1], 4, 1, 128, 16), ([0], 4, 1, 128, 16), ([0, 0, 0], 8, 2, 64, 8), ([5000], 8, 1, 128, 16),
    ([20000], 32, 8, 128, 16), ([9001, 1, 0, 12], 8, 4, 64, 32), ([4097] * 3, 16, 2, 128, 8),
    ([640] * 40, 8, 8, 128, 16), ([50] * 700, 4, 1, 64, 16), ([513, 0] * 60, 32, 4, 128, 32),
    (list(range(0, 400)), 8, 2, 128, 16), ([2048] * 19, 8, 8, 128, 16), ([33] * 38, 4, 4, 64, 8),
])
def test_decode_shapes(lens, hq, hkv, d, bs):
    """One piece and many: few long sequences, many short ones, empty ones among them."""
    b = Batch(lens, hq, hkv, d, bs, seed=len(lens))
    out = b.run()
    binding.pa_error_check()
    b.check(out, seqs=range(0, len(lens), max(1, len(lens) // 40)))
    again = b.run(fill=0x3c)
    assert torch.equal(out.view(torch.int16), again.view(torch.int16))


@pytest.mark.parametrize("max_len", [300, 301, 512, 4096])
def test_decode_with_a_looser_bound(max_len):
    """max_seq_len only sizes the launch."""
    b = Batch([300, 17, 0, 256], 8, 2, 128, 16, seed=4, table_pad=300)
    b.check(b.run(max_len=max_len))
    binding.pa_error_check()


@pytest.mark.parametrize("scale", [0.0, -0.3, 3.0, 1e-30, 1e30])
def test_decode_scales(scale):
    b = Batch([200, 3, 65], 8, 2, 128, 16, seed=6)
    if scale == 1e30:  # one key takes all: ties aside, P is 0 or 1
        b.q[:] = b.q[:, :1]
    out = b.run(scale=scale)
    if scale != 1e30:
        b.check(out, scale=scale)
        return
    got = np64(out)
    for s in range(3):
        k, v = b.rows(s)
        for h in range(8):
            x = k[:, h // 4] @ np64(b.q[s])[h]
            top = np.sort(x)
            if len(x) > 1 and top[-1] - top[-2] < 1e-3:
                continue
            want = v[x.argmax(), h // 4]
            assert (np.abs(got[s, h] - want) <= 2.0 ** -8 * np.abs(want) + 1e-30).all()


@pytest.mark.parametrize("scales", [(1.0, 1.0), (2.0 ** -60, 2.0 ** 60), (2.0 ** 30, 2.0 ** -100),
                                    (2.0 ** -130, 1.0), (2.0 ** 110, 1.0)])
def test_decode_tensor_scales(scales):
    b = Batch([150, 40], 8, 2, 128, 16, seed=7)
    scale = 0.02 / scales[0]
    out = b.run(scales=scales, scale=scale)
    b.check(out, scales=scales, scale=scale)


def test_decode_of_large_and_small_queries():
    for mult in (2.0 ** -100, 2.0 ** -20, 50.0, 2.0 ** 60):
        b = Batch([70, 130], 8, 2, 128, 16, seed=8, q_mult=mult)
        b.check(b.run(scale=0.1 / mult), scale=0.1 / mult)


def test_decode_sharp_rises():
    """Keys that grow along the sequence move the softmax's reference again and again."""
    b = Batch([700], 8, 1, 128, 16, seed=9)
    n = b.bs * b.d // 2
    sc = b.pool[..., n:].view(b.nb, 1, 2, 16, 8)
    for t in range(700):
        blk, o = int(b.tables[0, t // 16]), t % 16
        sc[blk, 0, 0, o] = min(0x7e, 8 + t // 6)  # up to the largest scale
    b.check(b.run(scale=0.05), scale=0.05)


def test_decode_special_values():
    """A NaN scale of a live token makes its sequence's heads NaN (K) or their 16 elements (V),
    and nothing else; infinite queries as the formula."""
    b = Batch([90, 45, 33], 8, 2, 128, 16, seed=10)
    n = b.bs * b.d // 2
    sc = b.pool[..., n:].view(b.nb, 2, 2, 16, 8)
    sc[int(b.tables[0, 2]), 1, 0, 5, 3] = 0x7f  # K of sequence 0, KV head 1
    sc[int(b.tables[1, 1]), 0, 1, 9, 2] = 0x7f  # V of sequence 1, KV head 0, elements 32..47
    out = b.run().float().cpu()
    assert out[0, 4:].isnan().all() and not out[0, :4].isnan().any()
    assert out[1, :4, 32:48].isnan().all()
    assert not out[1, :4, :32].isnan().any() and not out[1, :4, 48:].isnan().any()
    assert not out[1, 4:].isnan().any()
    b.check(b.run(), seqs=[2])
    b.q[2, 3, 7] = math.inf
    out = b.run().float().cpu()
    assert out[2, 3].isnan().all() and not out[2, :3].isnan().any()


def test_decode_bad_tables_and_lengths_are_flagged():
    b = Batch([64, 64, 64], 8, 2, 128, 16, seed=11, table_pad=4)
    good = b.run()
    binding.pa_error_check()
    b.tables[1, 2] = b.nb + 5
    out = b.run()
    with pytest.raises(binding.PaError, match="OOB"):
        binding.pa_error_check()
    assert torch.equal(out[[0, 2]], good[[0, 2]])
    # Its tokens read as zeros.
    pos = np.arange(64)
    tab = b.tables[1].numpy().copy()
    tab[2] = 0
    k, v = _fp4.read_rows(b.pool.numpy(), tab[pos // 16] * 16 + pos % 16, 16, 128, SCALES)
    k[32:48], v[32:48] = 0, 0
    want, tol = _fp4.attend(np64(b.q[1]), k, v, b.scale, 64)
    assert (np.abs(np64(out[1]) - want) <= tol).all()
    b.tables[1, 2] = -7
    assert torch.equal(b.run(), out)
    with pytest.raises(binding.PaError, match="OOB"):
        binding.pa_error_check()
    for bad in (-4, 65, 2 ** 31 - 1):
        b = Batch([64, 64, 64], 8, 2, 128, 16, seed=11, table_pad=4)
        b.lens = [64, bad, 64]
        out = b.run(max_len=64)
        with pytest.raises(binding.PaError, match="OOB"):
            binding.pa_error_check()
        assert torch.equal(out[[0, 2]], good[[0, 2]])
        assert torch.equal(out[1], good[1]) if bad > 0 else (out[1] == 0).all()


def test_decode_of_the_most_heads():
    """255 KV heads of 8 query heads, whole segments to a CTA and split."""
    for lens in ([40, 0, 200], [900, 33, 1]):
        b = Batch(lens, 2040, 255, 64, 16, seed=sum(lens))
        out = b.run()
        binding.pa_error_check()
        b.check(out)


def test_decode_sharing_blocks():
    b = Batch([200, 210, 220, 64], 8, 2, 128, 16, seed=12, shared=3)
    b.check(b.run())


def test_decode_of_many_sequences():
    """More sequences than one CTA's tables hold at full depth."""
    lens = [(i * 7) % 41 for i in range(9000)]
    b = Batch(lens, 2, 1, 64, 8, seed=13)
    out = b.run()
    binding.pa_error_check()
    b.check(out, seqs=range(0, 9000, 311))
    assert (out[0] == 0).all() and (out[41] == 0).all()


def test_decode_far_in_a_large_pool():
    """Byte offsets beyond 32 bits."""
    b = Batch([100, 200], 8, 8, 128, 32, seed=14)
    far = (1 << 32) // (8 * 2 * 32 * 72) + 1000
    big = torch.zeros(binding.fp4_pool_shape(far + b.nb, 8, 32, 128), dtype=torch.uint8,
                      device=DEV)
    big[far:] = b.pool.to(DEV)
    tables = torch.where(b.tables >= 0, b.tables + far, b.tables).to(DEV)
    out = torch.empty(b.q.shape, dtype=torch.bfloat16, device=DEV)
    binding.pa_decode_fp4(out, b.q.to(DEV), big, tables, ints(b.lens), 200, b.scale, *SCALES,
                          b.workspace())
    b.check(out)
    # Writes and reads there, too.
    gen = torch.Generator().manual_seed(1)
    rows = bf16((3, 8, 128), gen)
    slots = ints([far * 32 + 5, (far + 2) * 32 + 31, 7])
    binding.pa_cache_write_fp4(big, rows.to(DEV), rows.to(DEV), slots, *SCALES)
    out = [torch.empty(3, 8, 128, dtype=torch.bfloat16, device=DEV) for _ in range(2)]
    binding.pa_cache_read_fp4(*out, big, slots, *SCALES)
    for got, g in zip(out, SCALES):
        want = _fp4.dequantise(*_fp4.quantise(rows.float().numpy(), g), g)
        assert torch.equal(got.cpu(), _fp4.bf16_of_product(want))
    binding.pa_error_check()


@pytest.mark.parametrize("n", [1, 40, 700])
def test_decode_of_nothing_but_empty_sequences(n):
    b = Batch([0] * n, 4, 2, 128, 16)
    assert (b.run(max_len=0) == 0).all()
    assert (b.run(max_len=16) == 0).all()
    binding.pa_error_check()


def test_decode_batches_beyond_the_tables_are_refused():
    for d, n in ((128, 30000), (64, 40000)):
        b = Batch([1], 1, 1, d, 16)
        out = torch.empty(n, 1, d, dtype=torch.bfloat16, device=DEV)
        with pytest.raises(binding.PaError, match="UNSUPPORTED"):
            binding.pa_decode_fp4(out, out, b.pool.to(DEV),
                                  torch.zeros(n, 2, dtype=torch.int32, device=DEV),
                                  torch.ones(n, dtype=torch.int32, device=DEV), 1, 1.0, 1.0, 1.0,
                                  b.workspace())


def test_decode_of_the_largest_batches():
    """The ring shrinks as the tables grow."""
    for d, n in ((128, 10000), (64, 18000)):
        lens = [(i * 5) % 34 for i in range(n)]
        b = Batch(lens, 1, 1, d, 32, seed=n)
        out = b.run()
        binding.pa_error_check()
        b.check(out, seqs=range(0, n, n // 50))


@pytest.mark.parametrize("d, bs, n, lens", [
    (128, 8, 128, [4577, 3001, 4096, 4200]), (128, 16, 128, [4577, 3001, 4096, 4200]),
    (128, 32, 128, [4577, 3001, 4096, 4200]), (64, 8, 128, [4577, 3001, 4096, 4200]),
    (64, 32, 128, [4577, 3001, 4096, 4200]), (64, 16, 61, [9001, 40, 8999]),
    (128, 8, 1300, [577, 449, 500, 33]), (128, 32, 1300, [577, 449, 500, 33]),
    (64, 8, 5400, [133, 90, 128, 60, 0])])
def test_decode_of_many_tiles_a_warp(d, bs, n, lens):
    """Some 50 tiles a warp and more, of few sequences that come again and again."""
    b = Batch(lens, 32, 8, d, bs, seed=n + d + bs)
    which = [(i * 7 + i // 5) % len(lens) for i in range(n)]
    out = torch.full((n, 32, d), math.nan, dtype=torch.bfloat16, device=DEV)
    binding.pa_decode_fp4(out, b.q[which].to(DEV), b.pool.to(DEV), b.tables[which].to(DEV),
                          ints([lens[i] for i in which]), max(lens), b.scale, *SCALES,
                          b.workspace(0xff))
    binding.pa_error_check()
    got, which = np64(out), np.array(which)
    for s in range(len(lens)):
        want, tol = _fp4.attend(np64(b.q[s]), *b.rows(s), b.scale, lens[s])
        off = np.abs(got[which == s] - want)
        assert (off <= tol).all(), (s, off.max(), (off / tol).max())


def test_decode_where_every_boundary_falls():
    """Segments of every number of tiles, so that ranges begin and end anywhere in them."""
    for n, hkv, length in ((20, 8, 97), (8, 20, 1000), (160, 1, 65), (3, 60, 321), (152, 1, 33),
                           (153, 1, 32), (77, 2, 640), (1, 200, 2049)):
        b = Batch([length] * n, hkv * 2, hkv, 64, 16, seed=n, table_pad=256)
        out = b.run(max_len=4096)
        binding.pa_error_check()
        b.check(out, seqs=range(0, n, max(1, n // 10)))


# ------------------------------------------------------------------ rotation
class Turn:
    def __init__(self, n, hq, hkv, d, bs, rot, axes=1, interleaved=False, norm=(True, True),
                 seed=0, stride_pad=0, bits=16):
        gen = torch.Generator().manual_seed(seed)
        self.n, self.hq, self.hkv, self.d, self.bs, self.rot = n, hq, hkv, d, bs, rot
        self.axes, self.interleaved, self.bits = axes, interleaved, bits
        width = (hq + 2 * hkv) * d
        self.wide = bf16((n, width + stride_pad), gen)
        self.qkv = self.wide[:, :width]
        self.weights = [(torch.rand(d, generator=gen) + 0.5).to(torch.bfloat16) if w else None
                        for w in norm]
        ang = torch.arange(777, dtype=torch.float64)[:, None] * 50.0 ** (
            -torch.arange(rot // 2) / (rot // 2))
        self.cs = torch.cat([ang.cos(), ang.sin()], 1).float()
        self.positions = torch.randint(0, 777, (axes, n), generator=gen).to(torch.int32)
        self.pair_axis = (torch.randint(0, axes, (rot // 2,), generator=gen).to(torch.int32)
                          if axes > 1 else None)
        nb = -(-n // bs) + 2
        self.slots = torch.randperm(nb * bs, generator=gen)[:n].to(torch.int32)
        if n > 4:
            self.slots[3] = -1
        self.eps = 1e-5
        shape = binding.fp4_pool_shape(nb, hkv, bs, d) if bits == 4 else (nb, 2, hkv, bs, d)
        self.pool = (bf16(shape, gen) if bits == 16 else
                     torch.randint(0, 120, shape, dtype=torch.uint8, generator=gen))

    def run(self, pool=None, qkv=None, scales=SCALES):
        pool = self.pool.to(DEV) if pool is None else pool
        q = torch.full((self.n, self.hq, self.d), math.nan, dtype=torch.bfloat16, device=DEV)
        qkv = self.wide.to(DEV)[:, :self.qkv.shape[1]] if qkv is None else qkv
        qw, kw = (None if w is None else w.to(DEV) for w in self.weights)
        pos = self.positions.to(DEV)
        binding.pa_qkv_rope_write(
            q, qkv, pool, self.slots.to(DEV), pos if self.axes > 1 else pos[0], self.cs.to(DEV),
            q_weight=qw, k_weight=kw, eps=self.eps,
            pair_axis=None if self.pair_axis is None else self.pair_axis.to(DEV),
            interleaved=self.interleaved, kv_scales=None if self.bits == 16 else scales)
        return q, pool

    def want(self):
        w = [None if x is None else x.float().numpy() for x in self.weights]
        return _fp4.rotate(self.qkv.float().numpy(), self.hq, self.hkv, self.positions.numpy(),
                           self.cs.numpy(), None if self.pair_axis is None else
                           self.pair_axis.numpy(), self.interleaved, *w, self.eps)

    def v(self):
        return self.qkv.view(self.n, -1, self.d)[:, self.hq + self.hkv:]


def close(got, want, size):
    """bf16's rounding, and in fp32 a norm (at most 8 + log2 D roundings of its sum, halved by
    the root, and five more), its weight and three of the rotation: 20 of 2^-24 of the
    products' magnitudes."""
    tol = 2.0 ** -8 * np.abs(want) + 20 * 2.0 ** -24 * size
    off = np.abs(np64(got) - want)
    assert (off <= tol).all(), (off.max(), (off / tol).max())


TURNS = [
    dict(n=1, hq=32, hkv=4, d=64, bs=16, rot=64),
    dict(n=37, hq=8, hkv=2, d=128, bs=16, rot=128, axes=3),
    dict(n=130, hq=5, hkv=1, d=128, bs=32, rot=48, interleaved=True, stride_pad=40),
    dict(n=65, hq=6, hkv=3, d=64, bs=8, rot=16, axes=2, interleaved=True),
    dict(n=9, hq=7, hkv=7, d=64, bs=8, rot=48, norm=(False, True)),
    dict(n=12, hq=16, hkv=2, d=128, bs=16, rot=96, norm=(True, False), axes=8, stride_pad=8),
    dict(n=2500, hq=4, hkv=2, d=64, bs=16, rot=32, norm=(False, False)),
    dict(n=700, hq=32, hkv=8, d=128, bs=16, rot=128),
    dict(n=6000, hq=3, hkv=1, d=128, bs=16, rot=80),
    dict(n=5, hq=40, hkv=40, d=64, bs=8, rot=64, interleaved=True, axes=3),
    dict(n=3, hq=9, hkv=3, d=128, bs=32, rot=112, interleaved=True, norm=(True, False)),
    dict(n=1, hq=1, hkv=1, d=128, bs=16, rot=16, axes=4),
]


@pytest.mark.parametrize("case", TURNS, ids=str)
def test_rope_into_a_bf16_pool(case):
    t = Turn(**case, seed=case["n"])
    q, pool = t.run()
    binding.pa_error_check()
    wq, wk, sq, sk = t.want()
    close(q, wq, sq)
    want = t.pool.clone()
    live = (t.slots >= 0).nonzero()[:, 0]
    b, o = t.slots[live].long() // t.bs, t.slots[live].long() % t.bs
    close(pool.cpu()[b, 0, :, o], wk[live], sk[live])
    got = pool.cpu()
    want[b, 0, :, o] = got[b, 0, :, o]
    want[b, 1, :, o] = t.v()[live]
    assert torch.equal(got.view(torch.int16), want.view(torch.int16))  # V and the rest, bits


@pytest.mark.parametrize("bits", [8, 4])
@pytest.mark.parametrize("case", TURNS, ids=str)
def test_rope_into_quantised_pools_is_the_write_of_its_bf16_rows(case, bits):
    t = Turn(**case, seed=case["n"])
    q16, pool16 = t.run()
    t.bits = bits
    nb = pool16.shape[0]
    shape = (binding.fp4_pool_shape(nb, t.hkv, t.bs, t.d) if bits == 4
             else (nb, 2, t.hkv, t.bs, t.d))
    start = torch.randint(0, 120, shape, dtype=torch.uint8,
                          generator=torch.Generator().manual_seed(3)).to(DEV)
    q, pool = t.run(pool=start.clone())
    assert torch.equal(q.view(torch.int16), q16.view(torch.int16))
    slot = t.slots.clamp(min=0).long()
    k, v = (pool16[slot // t.bs, side, :, slot % t.bs].contiguous() for side in (0, 1))
    want = start.clone()
    write = binding.pa_cache_write_fp4 if bits == 4 else binding.pa_cache_write_fp8
    write(want, k, v, t.slots.to(DEV), *SCALES)
    assert torch.equal(pool, want)
    binding.pa_error_check()


def test_rope_of_the_most_heads():
    t = Turn(2, 2040, 255, 64, 16, 32, axes=8, seed=6)
    q, pool = t.run()
    binding.pa_error_check()
    wq, wk, sq, sk = t.want()
    close(q, wq, sq)
    b, o = t.slots.long() // 16, t.slots.long() % 16
    close(pool.cpu()[b, 0, :, o], wk, sk)
    assert torch.equal(pool.cpu()[b, 1, :, o], t.v())


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_without_a_norm_rounds_its_steps_apart(interleaved):
    """The formula's products and sums each rounded to fp32, then to bf16: the same bits."""
    t = Turn(60, 4, 2, 128, 16, 64, norm=(False, False), interleaved=interleaved)
    q, _ = t.run()
    x = t.qkv.view(60, -1, 128)[:, :4].float()
    row = t.cs[t.positions[0].long()][:, None]
    c, s = row[..., :32], row[..., 32:]
    at = (slice(0, 64, 2), slice(1, 64, 2)) if interleaved else (slice(0, 32), slice(32, 64))
    want = x.clone()
    want[..., at[0]] = x[..., at[0]] * c - x[..., at[1]] * s
    want[..., at[1]] = x[..., at[1]] * c + x[..., at[0]] * s
    assert torch.equal(q.cpu(), want.to(torch.bfloat16))


def test_rope_of_bad_positions_axes_and_slots():
    for bad in (-1, 777, 2 ** 31 - 1):
        t = Turn(20, 4, 2, 64, 16, 64, axes=2, seed=5)
        good_q, good_pool = t.run()
        t.positions[1, 7] = bad
        q, pool = t.run()
        with pytest.raises(binding.PaError, match="OOB"):
            binding.pa_error_check()
        assert q[7].isnan().all()  # left as it was
        keep = [i for i in range(20) if i != 7]
        assert torch.equal(q[keep], good_q[keep])
        want = good_pool.clone()
        b, o = divmod(int(t.slots[7]), 16)
        want[b, :, :, o] = t.pool[b, :, :, o].to(DEV)
        assert torch.equal(pool.view(torch.int16), want.view(torch.int16))
    # An axis that no pair uses may hold anything.
    t = Turn(20, 4, 2, 64, 16, 64, axes=2, seed=5)
    t.pair_axis[:] = 0
    t.positions[1] = -5
    t.run()
    binding.pa_error_check()
    # An axis beyond the axes is the first, flagged.
    good_q, _ = t.run()
    t.pair_axis[3] = 2
    q, _ = t.run()
    with pytest.raises(binding.PaError, match="OOB"):
        binding.pa_error_check()
    assert torch.equal(q, good_q)
    # A slot beyond the pool: q is there, the pool as it was.
    t = Turn(6, 4, 2, 64, 16, 64, seed=6)
    good_q, good_pool = t.run()
    keep = t.slots.clone()
    t.slots[:] = -1
    t.slots[2] = 10 ** 6
    q, pool = t.run()
    with pytest.raises(binding.PaError, match="OOB"):
        binding.pa_error_check()
    assert torch.equal(q, good_q)
    assert torch.equal(pool.cpu().view(torch.int16), t.pool.view(torch.int16))
    assert not torch.equal(keep, t.slots)


def test_rope_of_special_numbers():
    """Zero rows stay zero under a norm; a NaN or an infinity spoils its head alone."""
    t = Turn(4, 4, 2, 128, 16, 128, seed=7)
    t.wide[0] = 0
    t.wide[1, 5] = math.nan
    t.wide[2, 128 + 9] = math.inf
    q, pool = t.run()
    assert (q[0] == 0).all()
    assert q[1, 0].isnan().all() and not q[1, 1:].isnan().any()
    assert q[2, 1].isnan().any() and not q[2, [0, 2, 3]].isnan().any()
    assert not q[3].isnan().any()
    binding.pa_error_check()


def test_rope_refusals_of_the_binding():
    t = Turn(4, 4, 2, 64, 16, 64)
    cases = [dict(qkv=t.qkv.to(DEV)[:, 1:]), dict(qkv=t.qkv.to(DEV).T), dict(qkv=t.qkv)]
    for kw in cases:
        with pytest.raises(ValueError):
            t.run(**kw)
    t.bits = 8
    with pytest.raises(ValueError, match="kv_scales"):
        t.run(pool=torch.zeros(3, 2, 2, 16, 64, dtype=torch.uint8, device=DEV), scales=None)
    t.bits, t.axes = 16, 2
    t.positions = t.positions.repeat(2, 1)
    with pytest.raises(ValueError, match="pair_axis"):
        t.run()


# ------------------------------------------------------------------ together
class Step:
    """Steps of a decoding batch: rotation and write, then the attention."""

    def __init__(self, lens, hq, hkv, d, bs, rot, seed=0):
        self.b = Batch(lens, hq, hkv, d, bs, seed=seed)
        gen = torch.Generator().manual_seed(seed + 1)
        n = len(lens)
        self.qkv = bf16((n, (hq + 2 * hkv) * d), gen).to(DEV)
        ang = torch.arange(4096, dtype=torch.float64)[:, None] * 1e4 ** (
            -torch.arange(rot // 2) / (rot // 2))
        self.cs = torch.cat([ang.cos(), ang.sin()], 1).float().to(DEV)
        self.kw = bf16((d,), gen, 0.1).add_(1).to(DEV)
        last = [x - 1 for x in lens]
        self.positions = ints(last)
        self.slots = ints([int(self.b.tables[s, x // bs]) * bs + x % bs
                           for s, x in enumerate(last)])
        self.pool, self.tables = self.b.pool.to(DEV), self.b.tables.to(DEV)
        self.lens = ints(lens)
        self.q = torch.empty(n, hq, d, dtype=torch.bfloat16, device=DEV)
        self.out = torch.empty_like(self.q)
        self.ws = self.b.workspace()

    def run(self):
        binding.pa_qkv_rope_write(self.q, self.qkv, self.pool, self.slots, self.positions, self.cs,
                                  k_weight=self.kw, kv_scales=SCALES)
        binding.pa_decode_fp4(self.out, self.q, self.pool, self.tables, self.lens,
                              max(self.b.lens), self.b.scale, *SCALES, self.ws)

    def check(self):
        self.b.pool = self.pool.cpu()
        self.b.q = self.q.cpu()
        self.b.check(self.out)


@pytest.mark.parametrize("lens, d, bs", [([77, 1, 300, 33], 128, 16), ([12, 400, 64], 64, 8),
                                         ([500] * 30, 128, 32)])
def test_a_step_captured_and_replayed(lens, d, bs):
    s = Step(lens, 8, 2, d, bs, d, seed=d)
    s.run()
    s.check()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=stream):
        s.run()
        s.run()
    for seed in (1, 2):
        s.qkv.copy_(bf16(s.qkv.shape, torch.Generator().manual_seed(seed)))
        s.out.fill_(math.nan)
        graph.replay()
        torch.cuda.synchronize()
        first = s.out.clone()
        s.check()
        s.run()
        assert torch.equal(first.view(torch.int16), s.out.view(torch.int16))
    binding.pa_error_check()


def test_two_graphs_and_eager_calls_take_turns_with_one_workspace():
    a, b = Step([700, 30, 1500], 8, 2, 128, 16, 128, seed=3), Step([900] * 40, 8, 2, 128, 16, 64, 4)
    a.ws = b.ws = a.ws if a.ws.numel() >= b.ws.numel() else b.ws
    a.run()
    b.run()
    torch.cuda.synchronize()
    want = a.out.clone(), b.out.clone()
    graphs = []
    for step in (a, b):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step.run()
        graphs.append(g)
    for order in ("ab", "ba", "aabb"):
        a.ws.copy_(torch.randint(0, 256, a.ws.shape, dtype=torch.uint8, device=DEV))
        for x in order:
            step = a if x == "a" else b
            step.out.fill_(math.nan)
            graphs[x == "b"].replay()
            torch.cuda.synchronize()
            assert torch.equal(step.out.view(torch.int16), want[x == "b"].view(torch.int16))
            step.run()
    binding.pa_error_check()


def test_calls_on_another_stream():
    """The stream argument, and PyTorch's current one; work behind a long kernel waits for it."""
    s = Step([300, 77], 8, 2, 128, 16, 128, seed=5)
    s.run()
    torch.cuda.synchronize()
    want = s.out.clone()
    side = torch.cuda.Stream()
    fresh = s.qkv.clone()
    s.qkv.zero_()
    torch.cuda.synchronize()
    big = torch.randn(4096, 4096, device=DEV)
    with torch.cuda.stream(side):
        for _ in range(8):
            big = big @ big * 1e-3
        s.qkv.copy_(fresh)
        s.run()
    side.synchronize()
    assert torch.equal(s.out.view(torch.int16), want.view(torch.int16))
    s.out.fill_(0)
    torch.cuda.synchronize()
    binding.pa_decode_fp4(s.out, s.q, s.pool, s.tables, s.lens, 300, s.b.scale, *SCALES, s.ws,
                          stream=side)
    side.synchronize()
    assert torch.equal(s.out.view(torch.int16), want.view(torch.int16))


def test_two_steps_at_once_on_their_own_streams():
    a, b = Step([900, 30, 2000], 8, 2, 128, 16, 128, seed=1), Step([1500] * 5, 16, 2, 64, 8, 64, 2)
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for _ in range(20):
        for step, stream in zip((a, b), streams):
            with torch.cuda.stream(stream):
                step.run()
    torch.cuda.synchronize()
    a.check()
    b.check()
    binding.pa_error_check()


def test_a_context_read_back_is_what_the_attention_sees():
    """Written in 4 bits, read back, put into a bf16 pool: pa_decode there and pa_decode_fp4 here
    differ by their own roundings alone, and a prompt chunk attends to the context."""
    gen = torch.Generator().manual_seed(21)
    n, hq, hkv, d, bs = 333, 8, 2, 128, 16
    nb = 30
    k, v = bf16((n, hkv, d), gen).to(DEV), bf16((n, hkv, d), gen).to(DEV)
    perm = torch.randperm(nb, generator=gen)[:21]
    slots = ints((perm[:, None] * bs + torch.arange(bs)).reshape(-1)[:n])
    pool = torch.zeros(binding.fp4_pool_shape(nb, hkv, bs, d), dtype=torch.uint8, device=DEV)
    sc = (0.0017, 0.0021)
    binding.pa_cache_write_fp4(pool, k, v, slots, *sc)
    kb, vb = torch.empty_like(k), torch.empty_like(v)
    binding.pa_cache_read_fp4(kb, vb, pool, slots, *sc)
    wide = torch.zeros(nb, 2, hkv, bs, d, dtype=torch.bfloat16, device=DEV)
    binding.pa_cache_write(wide, kb, vb, slots)
    tables, lens = ints(perm)[None].contiguous(), ints([n])
    q = bf16((1, hq, d), gen).to(DEV)
    out4, out16 = torch.empty_like(q), torch.empty_like(q)
    ws = torch.empty(max(binding.pa_decode_fp4_workspace_bytes(1, hq, hkv, d),
                         binding.pa_decode_workspace_bytes(1, hq, hkv, d)), dtype=torch.uint8,
                     device=DEV)
    scale = d ** -0.5
    binding.pa_decode_fp4(out4, q, pool, tables, lens, n, scale, *sc, ws)
    binding.pa_decode(out16, q, wide, tables, lens, n, scale, ws)
    chunk = torch.empty_like(q)
    binding.pa_prefill_chunk(chunk, q, ints([0, 1]), 1, wide, tables, lens, scale)
    binding.pa_error_check()
    # The read-back rounds each value to bf16 (2^-8 of it at most): scores move by 2^-8 of
    # their magnitudes, weights by twice that.
    k64, v64 = np64(kb), np64(vb)
    want, tol = _fp4.attend(np64(q[0]), k64, v64, scale, n)
    p = np.abs(k64).max() * np.abs(np64(q)).sum(-1).max() * scale
    loose = tol + np.abs(v64).max() * (2 * p + 1) * 2.0 ** -8
    assert (np.abs(np64(out16[0]) - want) <= loose).all()
    assert (np.abs(np64(chunk[0]) - want) <= loose).all()
    assert (np.abs(np64(out4[0]) - want) <= loose).all()


def test_bindings_refuse_wrong_tensors():
    gen = torch.Generator().manual_seed(2)
    b = Batch([20, 30], 4, 2, 64, 16)
    pool, q, tables, lens = b.pool.to(DEV), b.q.to(DEV), b.tables.to(DEV), ints(b.lens)
    ws, out = b.workspace(), torch.empty_like(b.q, device=DEV)

    def decode(**kw):
        a = dict(out=out, q=q, kv_cache=pool, block_tables=tables, seq_lens=lens, max_seq_len=30,
                 scale=0.1, k_scale=1.0, v_scale=1.0, workspace=ws)
        a.update(kw)
        binding.pa_decode_fp4(**a)

    for kw in (dict(q=q[:1]), dict(out=out.float()), dict(kv_cache=pool[:, :, :1]),
               dict(kv_cache=pool[..., :-16].contiguous()), dict(kv_cache=pool.transpose(1, 2)),
               dict(block_tables=tables[:1]), dict(block_tables=tables.long()),
               dict(seq_lens=lens[:1]), dict(q=q.transpose(0, 1)), dict(workspace=ws[None])):
        with pytest.raises(ValueError):
            decode(**kw)
    with pytest.raises(binding.PaError, match="WORKSPACE"):
        decode(workspace=ws[:256])
    with pytest.raises(binding.PaError, match="INVALID"):
        decode(max_seq_len=10 ** 6)
    with pytest.raises(binding.PaError, match="INVALID"):
        decode(k_scale=-1.0)
    rows = bf16((3, 2, 64), gen).to(DEV)
    slots = ints([1, 2, 3])
    for kw in (dict(k_new=rows[:2]), dict(v_new=rows.float()), dict(slot_mapping=slots[:2]),
               dict(k_new=rows.transpose(1, 2)), dict(k_new=rows[..., :48], v_new=rows[..., :48]),
               dict(k_new=torch.cat([rows, rows], 1)[:, :2]), dict(kv_cache=pool[0])):
        a = dict(kv_cache=pool, k_new=rows, v_new=rows, slot_mapping=slots, k_scale=1.0,
                 v_scale=1.0)
        a.update(kw)
        with pytest.raises(ValueError):
            binding.pa_cache_write_fp4(**a)
    decode()
    binding.pa_error_check()
