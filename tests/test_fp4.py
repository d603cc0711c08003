"""The 4-bit pool without a GPU: its format, its definition's quantiser, and every refusal of
the calls over it (before anything is launched)."""

from __future__ import annotations

import ctypes
import os

import numpy as np
import pytest
import torch

from paged_kv_cache_287_gb300 import binding
from tests import _fp4

FAKE = 1 << 20  # 256-byte aligned, never dereferenced: every call below fails host checks


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(binding.LIB_PATH):
        from paged_kv_cache_287_gb300 import build
        build.build()
    return binding.lib()


def test_block_bytes(lib):
    assert lib.pa_kv_block_bytes_fp4(16, 8, 128) == 2 * 16 * 8 * (128 // 2 + 128 // 16)
    assert lib.pa_kv_block_bytes_fp4(8, 4, 64) * 32 == lib.pa_kv_block_bytes(8, 4, 64) * 9
    for bad in ((0, 8, 128), (16, -1, 128), (16, 8, 0), (16, 8, 72)):
        assert lib.pa_kv_block_bytes_fp4(*bad) == 0
    nb, heads, two, tile = binding.fp4_pool_shape(5, 8, 16, 128)
    assert (nb, heads, two) == (5, 8, 2)
    assert heads * two * tile == lib.pa_kv_block_bytes_fp4(16, 8, 128)


def test_formats_against_torch():
    """e4m3 codes, and the nearest of them, as PyTorch's own type has them."""
    codes = torch.arange(256, dtype=torch.uint8)
    want = codes.view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(_fp4.E4M3, want, equal_nan=True)
    x = torch.rand(20000, generator=torch.Generator().manual_seed(1)) * 500
    x = torch.cat([x, x / 1000, torch.tensor([0.0, 447.9, 448.0])]).clamp(max=448.0)
    got = _fp4.nearest_even(x.double().numpy(), _fp4.E4M3[:127])
    assert np.array_equal(got, x.to(torch.float8_e4m3fn).view(torch.uint8).numpy())


def test_quantiser_by_hand():
    """Scale and codes of a group written out: the largest element 12 of scale 2, each tie."""
    x = np.array([12, -12, 0.5, 1.5, 2.5, 3.5, 5, 7, 10, -0.0, 0.0, 0.51, -1.5, -5, 9.9, 1],
                 np.float32)
    codes, s = _fp4.quantise(x[None], 1.0)
    assert _fp4.E4M3[s[0, 0]] == 2.0
    want = [6, -6, 0, 1, 1, 2, 2, 4, 4, -0.0, 0, 0.5, -1, -2, 4, 0.5]  # of x / 2, ties to even
    got = _fp4.dequantise(codes, s, 0.5)[0]
    assert got.tolist() == want
    assert np.signbit(got[9]) and not np.signbit(got[10])


def test_quantiser_error_bound():
    """No element is off by more than a half step of its scale where it did not saturate, the
    scale by 2^-4 of itself: |x - x'| <= s (1 at most) and the largest within 1/6 of itself."""
    gen = torch.Generator().manual_seed(3)
    x = torch.randn(200, 128, generator=gen).to(torch.bfloat16).float().numpy()
    for g in (1.0, 0.002, 1 / 3):
        codes, s = _fp4.quantise(x, g)
        y = _fp4.dequantise(codes, s, g)
        d = _fp4.E4M3[s].repeat(16, -1) * float(np.float32(g))
        assert (np.abs(x - y) <= d * (1 + 2.0 ** -20)).all()
        assert (d.max() * 6 <= np.abs(x).max() * (1 + 2.0 ** -4) * (1 + 2.0 ** -20))


def test_quantiser_special_groups():
    x = np.zeros((6, 16), np.float32)
    x[1, 3] = np.nan
    x[1, 4] = 5
    x[2, 0], x[2, 1], x[2, 2] = np.inf, 1344.0, -np.inf
    x[3, :] = 2.0 ** -130
    x[4, 5] = 2.0 ** 120
    x[5, 7] = -2.0 ** -9
    codes, s = _fp4.quantise(x, 1.0)
    y = _fp4.dequantise(codes, s, 1.0)
    assert (y[0] == 0).all() and s[0, 0] == 0
    assert np.isnan(y[1]).all() and (codes[1] == 0).all()
    assert y[2, 0] == 2688 and y[2, 1] == 1344 and y[2, 2] == -2688
    assert (codes[3] == 0).all() and s[3, 0] == 0
    assert y[4, 5] == 2688
    assert s[5, 0] == 0 and (codes[5] == 0).all()  # 2^-9 / 6 rounds to no scale


def test_codes_without_a_division():
    """The kernels' shortcuts give the quotient's code for every bf16 x: two products around it
    that agree, and, where the divisor has at most 12 bits, one rounded to 18 bits; with a
    reciprocal off by up to 2^-23 either way."""
    x = (np.arange(65536, dtype=np.uint32) << 16).view(np.float32)
    x = x[np.isfinite(x)]
    rng = np.random.default_rng(0)

    def code(v):
        v = np.minimum(np.abs(v), np.float32(6)).astype(np.float64)
        return _fp4.nearest_even(v, _fp4.E2M1[:8])

    for n in range(300):
        if n % 2:
            d = np.float32(rng.integers(1, 4096) * 2.0 ** rng.integers(-90, 80))
        else:
            d = np.float32(_fp4.E4M3[rng.integers(1, 127)] * rng.random() * 10.0 ** rng.integers(
                -20, 20))
        if not 1e-30 < d < 1e30:
            continue
        near = x[(np.abs(x) <= d * 8) & (np.abs(x) >= d * 0.1)]
        want = code(near / d)
        for off in (-1, 0, 1):
            r = np.float32((1 + off * 2.0 ** -23) / np.float64(d))
            lo = code(near * np.float32(r * np.float32(1 - 2.0 ** -20)))
            hi = code(near * np.float32(r * np.float32(1 + 2.0 ** -20)))
            assert (lo[lo == hi] == want[lo == hi]).all()
            if d.view(np.uint32) & 0xfff == 0:
                q = (near * r).view(np.uint32) + np.uint32(0x20) & np.uint32(0xffffffc0)
                assert (code(q.view(np.float32)) == want).all()


# ------------------------------------------------------------------ refusals
def _cache(**kw):
    a = dict(kv=FAKE, k=FAKE, v=FAKE, slots=FAKE, stream=0, stride=8 * 128, nb=10, bs=16, hkv=8,
             d=128, n=4, ks=1.0, vs=1.0)
    a.update(kw)
    buf = ctypes.create_string_buffer(binding.FP4_ARGS[0].size)
    binding.FP4_ARGS[0].pack_into(buf, 0, *a.values())
    return buf


def _decode(**kw):
    a = dict(out=FAKE, q=FAKE, kv=FAKE, tables=FAKE, lens=FAKE, ws=FAKE, ws_bytes=1 << 30, stream=0,
             b=3, nb=10, bs=16, hq=32, hkv=8, d=128, mb=4, max_len=64, scale=0.1, ks=1.0, vs=1.0)
    a.update(kw)
    buf = ctypes.create_string_buffer(binding.FP4_ARGS[1].size)
    binding.FP4_ARGS[1].pack_into(buf, 0, *a.values())
    return buf


def _rope(**kw):
    a = dict(q_out=FAKE, kv=FAKE, qkv=FAKE, qw=FAKE, kw=FAKE, cs=FAKE, pos=FAKE, axis=0,
             slots=FAKE, stream=0, stride=48 * 128, n=4, nb=10, bs=16, hq=32, hkv=8, d=128,
             rot=128, max_pos=100, axes=1, inter=0, bits=16, eps=1e-6, ks=1.0, vs=1.0)
    a.update(kw)
    buf = ctypes.create_string_buffer(binding.FP4_ARGS[2].size)
    binding.FP4_ARGS[2].pack_into(buf, 0, *a.values())
    return buf


NAN, INF = float("nan"), float("inf")


@pytest.mark.parametrize("status, kw", [
    (1, dict(kv=0)), (1, dict(kv=FAKE + 8)), (1, dict(k=0)), (1, dict(v=FAKE + 2)),
    (1, dict(slots=0)), (1, dict(slots=FAKE + 2)), (1, dict(nb=0)), (1, dict(n=-1)),
    (2, dict(d=96)), (2, dict(bs=12)), (2, dict(hkv=256, stride=1 << 20)),
    (2, dict(nb=1 << 27)), (1, dict(stride=8 * 128 - 8)), (1, dict(stride=8 * 128 + 4)),
    (1, dict(ks=0.0)), (1, dict(vs=-1.0)), (1, dict(ks=NAN)), (1, dict(vs=INF)),
    (1, dict(ks=1.3e35)), (0, dict(n=0, vs=1.2e35)),
    (0, dict(n=0)), (0, dict(n=0, k=0, v=0, slots=0)),
])
def test_cache_refusals(lib, status, kw):
    assert lib.pa_cache_write_fp4(_cache(**kw)) == status
    assert lib.pa_cache_read_fp4(_cache(**kw)) == status
    assert lib.pa_cache_write_fp4(None) == lib.pa_cache_read_fp4(None) == 1


@pytest.mark.parametrize("status, kw", [
    (1, dict(out=0)), (1, dict(q=FAKE + 8)), (1, dict(kv=0)), (1, dict(tables=0)),
    (1, dict(lens=FAKE + 2)), (1, dict(b=-1)), (1, dict(hkv=5)), (2, dict(hq=72)),
    (2, dict(d=256)), (2, dict(bs=64)), (1, dict(mb=0)), (1, dict(max_len=65)),
    (1, dict(max_len=-1)), (1, dict(scale=NAN)), (1, dict(scale=INF)), (1, dict(ks=0.0)),
    (1, dict(vs=NAN)), (1, dict(ks=1e36)), (2, dict(b=1 << 20, mb=1 << 16, max_len=1 << 20)),
    (2, dict(b=1, mb=1 << 28, max_len=(1 << 31) - 1)), (2, dict(b=10456)),
    (2, dict(b=19160, d=64)), (2, dict(b=9944, bs=8, max_len=9)),
    (2, dict(b=18648, bs=8, d=64, max_len=9)), (6, dict(ws=0)),
    (6, dict(ws=FAKE + 128)), (6, dict(ws_bytes=100)), (0, dict(b=0)),
])
def test_decode_refusals(lib, status, kw):
    assert lib.pa_decode_fp4(_decode(**kw)) == status
    assert lib.pa_decode_fp4(None) == 1


@pytest.mark.parametrize("status, kw", [
    (1, dict(q_out=0)), (1, dict(kv=0)), (1, dict(qkv=FAKE + 8)), (1, dict(qw=FAKE + 8)),
    (1, dict(kw=FAKE + 2)), (1, dict(cs=0)), (1, dict(pos=0)), (1, dict(slots=0)),
    (1, dict(stride=48 * 128 - 8)), (1, dict(stride=48 * 128 + 4)), (1, dict(n=-1)),
    (1, dict(rot=0)), (2, dict(rot=120)), (2, dict(rot=144)), (1, dict(max_pos=0)),
    (1, dict(axes=0)), (2, dict(axes=9, axis=FAKE)), (1, dict(axes=2)),
    (1, dict(axis=FAKE + 2)), (1, dict(bits=6)), (1, dict(bits=4, ks=0.0)),
    (1, dict(bits=8, vs=NAN)), (1, dict(bits=4, vs=1e36)),
    (0, dict(n=0, bits=8, vs=1e36)), (1, dict(eps=NAN)), (1, dict(eps=-1.0)), (1, dict(eps=INF)),
    (1, dict(hq=30)), (2, dict(hq=72)), (2, dict(d=96)), (0, dict(n=0)),
    (0, dict(n=0, eps=NAN, qw=0, kw=0)),
])
def test_rope_refusals(lib, status, kw):
    assert lib.pa_qkv_rope_write(_rope(**kw)) == status
    assert lib.pa_qkv_rope_write(None) == 1


def test_struct_and_workspace_sizes(lib):
    for call, layout in enumerate(binding.FP4_ARGS):
        assert lib.pa_fp4_args_bytes(call) == layout.size
    assert lib.pa_fp4_args_bytes(3) == lib.pa_fp4_args_bytes(-1) == 0
    assert lib.pa_decode_fp4_workspace_bytes(3, 32, 8, 128) > 0
    for bad in ((-1, 32, 8, 128), (3, 32, 0, 128), (3, 30, 8, 128), (3, 72, 8, 128),
                (3, 32, 8, 96)):
        assert lib.pa_decode_fp4_workspace_bytes(*bad) == 0


def test_binding_refuses_cpu_tensors(lib):
    kv = torch.zeros(binding.fp4_pool_shape(4, 2, 16, 64), dtype=torch.uint8)
    rows = torch.zeros(3, 2, 64, dtype=torch.bfloat16)
    slots = torch.zeros(3, dtype=torch.int32)
    for call in (lambda: binding.pa_cache_write_fp4(kv, rows, rows, slots, 1.0, 1.0),
                 lambda: binding.pa_cache_read_fp4(rows, rows, kv, slots, 1.0, 1.0),
                 lambda: binding.pa_decode_fp4(rows, rows, kv, slots[None], slots, 4, 1.0, 1.0,
                                               1.0, kv.flatten()),
                 lambda: binding.pa_qkv_rope_write(rows, rows.view(3, -1), kv, slots, slots,
                                                   torch.zeros(4, 64), kv_scales=(1.0, 1.0))):
        with pytest.raises(ValueError):
            call()


# ------------------------------------------------------------------ the plain forms themselves
def test_plain_attention_against_torch():
    gen = torch.Generator().manual_seed(5)
    q, k, v = (torch.randn(n, h, 64, generator=gen, dtype=torch.float64)
               for n, h in ((1, 6), (50, 2), (50, 2)))
    out, tol = _fp4.attend(q[0].numpy(), k.numpy(), v.numpy(), 0.125, 37)
    for h in range(6):
        p = torch.softmax(k[:37, h // 3] @ q[0, h] * 0.125, 0)
        assert np.allclose(out[h], (p @ v[:37, h // 3]).numpy(), rtol=1e-12)
    assert (tol < 0.02).all()


@pytest.mark.parametrize("interleaved", [False, True])
def test_plain_rotation_keeps_lengths_and_differences(interleaved):
    """A rotation keeps norms, and products of rows go by the difference of their positions."""
    rng = np.random.default_rng(2)
    d, rot = 64, 32
    freq = 100.0 ** (-np.arange(rot // 2) / (rot // 2))
    ang = np.arange(50)[:, None] * freq
    cs = np.concatenate([np.cos(ang), np.sin(ang)], 1)
    x = rng.standard_normal((1, 3 * d)).repeat(4, 0)
    pos = np.array([[3, 11, 13, 21]])
    q, k, _, _ = _fp4.rotate(x, 1, 1, pos, cs, None, interleaved, None, None, 0.0)
    assert np.allclose((q ** 2).sum(-1), (x[:, None, :d] ** 2).sum(-1))
    dots = np.einsum("nhd,mhd->nm", q, k)
    assert np.isclose(dots[0, 1], dots[2, 3]) and not np.isclose(dots[0, 1], dots[0, 2])
