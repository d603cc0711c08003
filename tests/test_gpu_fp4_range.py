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
