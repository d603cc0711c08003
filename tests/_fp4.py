"""Plain CPU implementations for the 4-bit pool and the rotation, from their definitions.

Quantisation follows the binary32 steps of its definition (numpy float32); everything else is
in 64 bits.
"""

from __future__ import annotations

import numpy as np
import torch

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E2M1 = np.concatenate([E2M1, -E2M1])


def _e4m3_table() -> np.ndarray:
    v = np.empty(256)
    for b in range(256):
        e, m = b >> 3 & 15, b & 7
        x = m * 2.0 ** -9 if e == 0 else (8 + m) * 2.0 ** (e - 10)
        if b & 127 == 127:
            x = np.nan
        v[b] = -x if b & 128 else x
    return v


E4M3 = _e4m3_table()


def nearest_even(x: np.ndarray, grid: np.ndarray) -> np.ndarray:
    """Index of the nearest of an increasing grid, ties to the even index, ends saturating."""
    up = np.clip(np.searchsorted(grid, x), 1, len(grid) - 1)
    low, high = x - grid[up - 1], grid[up] - x
    return np.where((high < low) | ((high == low) & (up % 2 == 0)), up, up - 1)


def quantise(x: np.ndarray, g: float):
    """float32 rows [..., D] (bf16 values) to code bytes [..., D / 2] and scales [..., D / 16]."""
    x = x.astype(np.float32).reshape(*x.shape[:-1], -1, 16)
    g = np.float32(g)
    with np.errstate(all="ignore"):
        amax = np.abs(x).max(-1)  # NaN where one is
        t = amax / (np.float32(6) * g)
        s = nearest_even(np.minimum(np.nan_to_num(t, nan=0.0, posinf=448.0), 448.0)
                         .astype(np.float64), E4M3[:127])
        s = np.where(np.isnan(amax), 127, s).astype(np.uint8)
        d = (E4M3[s].astype(np.float32) * g)[..., None]
        a = np.abs(x) / d
        fine = np.broadcast_to(d > 0, x.shape)
        c = nearest_even(np.where(fine, np.minimum(a, np.float32(6)), 0).astype(np.float64),
                         E2M1[:8])
        c = np.where(fine, c + 8 * np.signbit(x), 0).astype(np.uint8)
    c = c.reshape(*c.shape[:-2], -1)
    return c[..., 0::2] | c[..., 1::2] << 4, s


def dequantise(codes: np.ndarray, s: np.ndarray, g: float) -> np.ndarray:
    """Code bytes and scales to values, in 64 bits (code * scale * binary32 g, unrounded)."""
    c = np.stack([codes & 15, codes >> 4], -1).reshape(*s.shape, 16)
    x = E2M1[c] * E4M3[s][..., None] * float(np.float32(g))
    return x.reshape(*s.shape[:-1], 16 * s.shape[-1])


def split_pool(pool: np.ndarray, bs: int, d: int):
    """Views of a pool [NB, H, 2, tile]: codes [NB, H, 2, bs, D/2], scales [NB, H, 2, bs, D/16]."""
    nb, h = pool.shape[:2]
    n = bs * d // 2
    return (pool[..., :n].reshape(nb, h, 2, bs, d // 2),
            pool[..., n:].reshape(nb, h, 2, bs, d // 16))


def write_rows(pool: np.ndarray, k, v, slots, bs: int, scales) -> None:
    """The pool's bytes after the write, in place (slots outside the pool are skipped)."""
    d = k.shape[-1]
    n = bs * d // 2
    for side, (x, g) in enumerate(zip((k, v), scales)):
        codes, s = quantise(x.float().numpy(), g)
        for i, slot in enumerate(slots):
            if 0 <= slot < pool.shape[0] * bs:
                b, o = divmod(int(slot), bs)
                pool[b, :, side, o * d // 2:(o + 1) * d // 2] = codes[i]
                pool[b, :, side, n + o * d // 16:n + (o + 1) * d // 16] = s[i]


def read_rows(pool: np.ndarray, slots, bs: int, d: int, scales):
    """K and V rows [N, H, D] of the slots, in 64 bits."""
    codes, s = split_pool(pool, bs, d)
    slots = np.asarray(slots)
    return [dequantise(codes[slots // bs, :, side, slots % bs], s[slots // bs, :, side, slots % bs],
                       g) for side, g in enumerate(scales)]


def bf16_of_product(x: np.ndarray) -> torch.Tensor:
    """What a read-back stores: rounded to binary32, then to bf16."""
    return torch.from_numpy(x.astype(np.float32)).to(torch.bfloat16)


def attend(q, k, v, scale: float, length: int):
    """softmax(scale q.K^T) V of one sequence in 64 bits, and the bound of a kernel's error.

    q [Hq, D] (bf16 values), k, v [tokens, Hkv, D].  The bound counts: the output's rounding to
    bf16 (2^-8 of it); P's rounding to f16, 2^-11 of each weight, or 2^-25 of the largest where
    a weight is below 2^-14 of it; the scores' fp32 sums (D roundings of at most the sum of
    magnitudes, 2^-24 each, and four for the factors), and q's f16 form, which is exact down to
    2^-14 of a head's largest element and off by 2^-25 of that below; 2^-21 for the
    exponential and its argument's rounding, 2^-20 for the sums over tokens and pieces (their
    roundings do not add up: at most 2^-24 sqrt(tokens) to 131072 tokens, and four times that).
    """
    hq, d = q.shape
    hkv = k.shape[1]
    g = hq // hkv
    if length == 0:
        return np.zeros((hq, d)), np.zeros((hq, d))
    q, k, v = q.astype(np.float64), k[:length], v[:length]
    out, tol = np.empty((hq, d)), np.empty((hq, d))
    for h in range(hq):
        kh, vh = k[:, h // g], v[:, h // g]
        x = kh @ q[h] * scale
        p = np.exp(x - x.max())
        p /= p.sum()
        out[h] = p @ vh
        size = (np.abs(kh) @ np.abs(q[h])).max() * abs(scale)
        small = np.abs(kh).sum(1).max() * np.abs(q[h]).max() * 2.0 ** -24 * abs(scale)
        dx = (d + 4) * 2.0 ** -24 * size + small + 2.0 ** -23 * np.abs(x).max()
        weight = 2.0 ** -11 + 2 * dx + 2.0 ** -20
        tol[h] = (2.0 ** -8 * np.abs(out[h]) + weight * (p @ np.abs(vh))
                  + 2.0 ** -24 * np.abs(vh).sum(0) * p.max())
        tol[h] += 2.0 ** -133  # the output's own underflow
    return out, tol


def rotate(qkv, hq: int, hkv: int, positions, cos_sin, pair_axis, interleaved: bool, q_weight,
           k_weight, eps: float):
    """q [N, Hq, D] and K [N, Hkv, D] in 64 bits, and the magnitude their rounding errors go by:
    of a rotated pair's element the sum of its two products' magnitudes."""
    n = qkv.shape[0]
    x = qkv.reshape(n, hq + 2 * hkv, -1)[:, :hq + hkv].astype(np.float64).copy()
    d = x.shape[-1]
    for w, lo, hi in ((q_weight, 0, hq), (k_weight, hq, hq + hkv)):
        if w is not None:
            r = np.sqrt((x[:, lo:hi] ** 2).mean(-1, keepdims=True) + eps)
            x[:, lo:hi] = x[:, lo:hi] / r * w.astype(np.float64)
    rot = cos_sin.shape[1]
    size = np.abs(x)
    y = x.copy()
    for i in range(rot // 2):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + rot // 2)
        axis = 0 if pair_axis is None else int(pair_axis[i])
        row = cos_sin[positions[axis]].astype(np.float64)
        c, s = row[:, i][:, None], row[:, i + rot // 2][:, None]
        y[..., a] = x[..., a] * c - x[..., b] * s
        y[..., b] = x[..., b] * c + x[..., a] * s
        size[..., a] = np.abs(x[..., a] * c) + np.abs(x[..., b] * s)
        size[..., b] = np.abs(x[..., b] * c) + np.abs(x[..., a] * s)
    return y[:, :hq], y[:, hq:], size[:, :hq], size[:, hq:]
