"""Draft-tree kernels without a GPU: the order of what their sources synchronise.

What these hand-overs prevent shows on a GPU only now and then, or not at all, so the
sources themselves are read: each rule names a statement and what has to stand before it.
"""

from __future__ import annotations

import os
import re

from paged_kv_cache_287_gb300 import build


def source(name: str) -> str:
    """A kernel source without its comments."""
    with open(os.path.join(build.CSRC, name)) as f:
        return re.sub(r"//[^\n]*", "", f.read())


def kernel(text: str, name: str) -> str:
    """The body of __global__ function `name`."""
    at = text.index("{", text.index(")", re.search(rf"\b{name}\(", text).start()))
    depth = 0
    for i in range(at, len(text)):
        depth += {"{": 1, "}": -1}.get(text[i], 0)
        if depth == 0:
            return text[at:i + 1]
    raise AssertionError(f"{name} has no end")


def test_a_peers_shared_memory_is_written_once_its_cta_has_started():
    """A CTA of a cluster may be stored to only when it is known to run: the cluster's
    first barrier is waited for before the first remote store."""
    body = kernel(source("pa_tree_verify.cu"), "tree_verify_kernel")
    stores = [m.start() for m in re.finditer(r"st\.shared::cluster", body)]
    assert stores
    arrive, wait = body.find("cluster_arrive()"), body.find("cluster_wait()")
    assert 0 <= arrive < wait < min(stores)
    # Sequences without work leave before they arrive.
    assert body.index("if (span.n <= 0)") < arrive


def test_shared_memory_written_by_a_warp_is_handed_over_by_a_warp_barrier():
    """Stores of several lanes that a product reads (or that lane 0 announces): the fence to
    the asynchronous side, by every lane, then a barrier of the warp."""
    text = source("pa_tree_attention.cu")
    fences = [m.end() for m in re.finditer(r"fence_proxy_async_smem\(\);", text)]
    assert len(fences) >= 3
    for at in fences:
        assert re.match(r"\s*__syncwarp\(\);", text[at:]), text[at:at + 80]
