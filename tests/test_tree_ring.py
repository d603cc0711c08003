"""The places of K and V tiles in the tree attention's shared memory, without a GPU.

The kernel's rules (``csrc/pa_tree_ring.h``) are compiled for the host and run under
random orders of its threads: the warps that copy K and V, the threads that issue the two
products, the products themselves, the softmax.  Barriers show a phase's parity alone, as
the GPU's do.  No order may stall, and no product may read a place that holds another
tile.
"""

from __future__ import annotations

import ctypes
import os
import random
import shutil
import subprocess

import pytest

from paged_kv_cache_287_gb300 import build

CONFIGS = [(64, False), (128, False), (128, True)]  # head size, FP8 pool
NONE, SCORES, OUTPUT = range(3)

DRIVER = """
#include "pa_tree_ring.h"
using namespace pa;
template <class R> void rule(int what, int i, int *o) {
    if (what == 0) { o[0] = R::k(i).slot; o[1] = R::k(i).use; }
    if (what == 1) { o[0] = R::v(i).slot; o[1] = R::v(i).use; }
    if (what == 2) { o[0] = (int)R::k_after(i).what; o[1] = R::k_after(i).tile; }
    if (what == 3) { o[0] = (int)R::v_after(i).what; o[1] = R::v_after(i).tile; }
    if (what == 4) { o[0] = R::kSlots; o[1] = R::kInFlight; o[2] = R::kKLandsByScores; }
}
extern "C" void ring_rule(int d, int kv8, int what, int i, int *o) {
    if (kv8) rule<TreeRing<128, true>>(what, i, o);
    else if (d == 64) rule<TreeRing<64, false>>(what, i, o);
    else rule<TreeRing<128, false>>(what, i, o);
}
"""


@pytest.fixture(scope="module")
def rules(tmp_path_factory):
    cxx = shutil.which("g++")
    if cxx is None:
        pytest.skip("no host compiler")
    where = tmp_path_factory.mktemp("ring")
    src, so = where / "ring.cpp", where / "ring.so"
    src.write_text(DRIVER)
    subprocess.run([cxx, "-std=c++17", "-shared", "-fPIC", "-I", build.CSRC, str(src), "-o",
                    str(so)], check=True)
    lib = ctypes.CDLL(os.fspath(so))

    def table(d, kv8, n):
        o = (ctypes.c_int * 3)()

        def get(what, i):
            o[:] = [0, 0, 0]
            lib.ring_rule(d, int(kv8), what, i, o)
            return o[0], o[1], o[2]
        return {"k": [get(0, i)[:2] for i in range(n)], "v": [get(1, i)[:2] for i in range(n)],
                "k_after": [get(2, i)[:2] for i in range(n)],
                "v_after": [get(3, i)[:2] for i in range(n)],
                "slots": get(4, 0)[0], "in_flight": get(4, 0)[1], "by_scores": get(4, 0)[2]}
    return table


class Barrier:
    """Completed phases; a wait for parity p passes while the current phase's is not p."""

    def __init__(self):
        self.done = 0

    def passes(self, parity):
        return (self.done & 1) != parity


def simulate(r, n, rng, one_warp, kv8):
    """Threads as generators that yield what they wait for (a function) before each step.
    One whose weight is small runs only now and then.  Of an FP8 pool the warps that convert
    V fill its places (and wait for nothing at their end)."""
    full = [Barrier() for _ in range(r["slots"])]
    s_done, pv_done = [Barrier() for _ in range(4)], [Barrier() for _ in range(4)]
    p_full, pv_issued = [Barrier(), Barrier()], [Barrier(), Barrier()]
    holds = [None] * r["slots"]   # what a slot holds (from the copy's issue on)
    landing, s_queue, pv_queue = [], [], []

    def tile_wait(bars, i):
        return lambda: bars[i & 3].passes((i >> 2) & 1)

    def after(rule):
        what, t = rule
        return (lambda: True) if what == NONE else tile_wait(s_done if what == SCORES else
                                                             pv_done, t)

    def load(kind, i):
        yield after(r[kind + "_after"][i])
        slot = r[kind][i][0]
        before = holds[slot]
        # The product that reads what lay there is done.
        assert before is None or before in finished, f"{kind}{i} over {before}"
        holds[slot] = (kind, i)
        landing.append(slot)

    finished = set()

    def land(kind):
        for i in range(max(0, n - r["in_flight"]), n):
            if kind == "k" and r["by_scores"]:
                yield tile_wait(s_done, i)
            else:
                slot, use = r[kind][i]
                yield (lambda slot=slot, use=use: full[slot].passes(use & 1))

    def k_warp():
        for i in range(n):
            yield from load("k", i)
            if one_warp and i > 0:
                yield from load("v", i - 1)
        if one_warp:
            yield from load("v", n - 1)
        yield from land("k")
        if one_warp:
            yield from land("v")

    def v_warp():
        for i in range(n):
            yield from load("v", i)
        if not kv8:
            yield from land("v")

    def copies():
        for _ in range(2 * n):
            yield lambda: bool(landing)
            full[landing.pop(rng.randrange(len(landing)))].done += 1

    def scores():
        for i in range(n):
            if i >= 2:
                yield lambda i=i: pv_issued[i & 1].passes((i // 2 - 1) & 1)
            slot, use = r["k"][i]
            yield lambda slot=slot, use=use: full[slot].passes(use & 1)
            assert holds[slot] == ("k", i), f"scores {i} read {holds[slot]}"
            s_queue.append(i)

    def s_product():
        for _ in range(n):
            yield lambda: bool(s_queue)
            i = s_queue.pop(0)
            assert holds[r["k"][i][0]] == ("k", i), f"scores {i}: overwritten"
            finished.add(("k", i))
            s_done[i & 3].done += 1

    def softmax():
        for i in range(n):
            yield tile_wait(s_done, i)
            p_full[i & 1].done += 1

    def output():
        for i in range(n):
            yield lambda i=i: p_full[i & 1].passes((i // 2) & 1)
            slot, use = r["v"][i]
            yield lambda slot=slot, use=use: full[slot].passes(use & 1)
            assert holds[slot] == ("v", i), f"output {i} read {holds[slot]}"
            pv_queue.append(i)
            pv_issued[i & 1].done += 1

    def pv_product():
        for _ in range(n):
            yield lambda: bool(pv_queue)
            i = pv_queue.pop(0)
            assert holds[r["v"][i][0]] == ("v", i), f"output {i}: overwritten"
            finished.add(("v", i))
            pv_done[i & 3].done += 1

    names = [k_warp, copies, scores, s_product, softmax, output, pv_product]
    if not one_warp:
        names.append(v_warp)
    run = [(g.__name__, g()) for g in names]
    weight = {name: rng.choice([1.0, 1.0, 0.1, 0.003]) for name, _ in run}
    wants = {name: next(g, None) for name, g in run}
    while any(w is not None for w in wants.values()):
        ready = [(name, g) for name, g in run if wants[name] is not None and wants[name]()]
        assert ready, "stalled: " + ", ".join(k for k, w in wants.items() if w is not None)
        name, g = rng.choices(ready, [weight[x] for x, _ in ready])[0]
        wants[name] = next(g, None)
    assert len(finished) == 2 * n


@pytest.mark.parametrize("d,kv8,one_warp", [(64, False, True), (64, False, False),
                                            (128, False, True), (128, False, False),
                                            (128, True, False)])
def test_no_order_of_the_threads_stalls_or_overwrites_a_tile(rules, d, kv8, one_warp):
    r = rules(d, kv8, 64)
    rng = random.Random(d + kv8)
    for n in [*range(1, 12), 17, 24, 40]:
        for _ in range(60):
            simulate(r, n, rng, one_warp, kv8)


@pytest.mark.parametrize("d,kv8", CONFIGS)
def test_a_load_waits_for_what_its_place_held_before(rules, d, kv8):
    """For every place: the tile in it before (none at first), as often as it was filled."""
    r = rules(d, kv8, 64)
    order = [("k", 0)]
    for i in range(1, 64):
        order += [("k", i), ("v", i - 1)]
    held, fills = {}, {}
    for kind, i in order:
        slot, use = r[kind][i]
        assert 0 <= slot < r["slots"] and use == fills.get(slot, 0)
        what, tile = r[kind + "_after"][i]
        assert (what, tile)[:1 if what == NONE else 2] == (
            (NONE,) if slot not in held else
            (SCORES if held[slot][0] == "k" else OUTPUT, held[slot][1]))
        held[slot], fills[slot] = (kind, i), use + 1
