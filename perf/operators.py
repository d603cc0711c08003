"""The operators of a speculative step over a paged KV cache, as cases to be timed.

A draft tree of at most 64 nodes per sequence (node 0: the last committed token;
``parents[i] < i``) is checked by the target model in one pass:

* ``attention``: every node attends to its sequence's cached context, its
  ancestors and itself, through the block table (bf16 or FP8 e4m3 pool);
* ``verify``: the drafted tokens are accepted or rejected against the target's
  probabilities with given random numbers, and the next token is drawn;
* ``accept``: the accepted nodes' K/V rows move up behind the context, in place.

``own`` false: the plain forms below.  ``own`` true: the library's entry points.
"""

import math

import torch

own = False

DEV = "cuda"
MAX_NODES = 64


def listed():
    """The cases, each with what it stands for."""
    return [
        # One user's chat with a chain of four drafted tokens behind the last one:
        # latency of a single sequence of the small model's heads.
        dict(name="attention chain b1", op="attention", b=1, heads=32, kv_heads=4, dim=64,
             block=16, t_lo=5, t_hi=5, shape="chain", ctx_lo=100, ctx_hi=100, log=False,
             q_mult=1.0, pool="bf16"),
        # A serving batch with a 16-node tree per sequence, ordinary contexts.
        dict(name="attention tree b32", op="attention", b=32, heads=32, kv_heads=8, dim=128,
             block=16, t_lo=12, t_hi=16, shape="tree", ctx_lo=512, ctx_hi=4096, log=False,
             q_mult=1.0, pool="bf16"),
        # The same from an FP8 pool, twice the sequences and short chains.
        dict(name="attention chain b64 fp8", op="attention", b=64, heads=32, kv_heads=8, dim=128,
             block=16, t_lo=3, t_hi=8, shape="chain", ctx_lo=512, ctx_hi=4096, log=False,
             q_mult=1.0, pool="fp8"),
        # The widest trees under the widest groups: 64 nodes x 8 query heads per KV
        # head, ragged, where the products weigh as much as the cache's bytes.
        dict(name="attention wide b16", op="attention", b=16, heads=64, kv_heads=8, dim=128,
             block=16, t_lo=33, t_hi=64, shape="tree", ctx_lo=1024, ctx_hi=8192, log=False,
             q_mult=1.0, pool="bf16"),
        # Long skewed contexts, sharp softmax, odd tree sizes, small blocks.
        dict(name="attention long b8", op="attention", b=8, heads=32, kv_heads=8, dim=128,
             block=8, t_lo=7, t_hi=23, shape="tree", ctx_lo=1024, ctx_hi=131072, log=True,
             q_mult=2.0, pool="bf16"),
        # One sequence's chain of five against its draft distribution: latency.
        dict(name="verify chain b1", op="verify", b=1, vocab=32000, t_lo=6, t_hi=6,
             shape="chain", draft=True),
        # Trees whose siblings were drawn from the draft distribution, odd
        # vocabulary: several rounds of residuals per node.
        dict(name="verify tree b48", op="verify", b=48, vocab=50021, t_lo=9, t_hi=31,
             shape="tree", draft=True),
        # Wide trees proposed without probabilities, large vocabulary.
        dict(name="verify wide b64", op="verify", b=64, vocab=131072, t_lo=33, t_hi=64,
             shape="tree", draft=False),
        # A large serving batch of chains against large-vocabulary distributions.
        dict(name="verify chain b256", op="verify", b=256, vocab=131072, t_lo=6, t_hi=6,
             shape="chain", draft=True),
        # One sequence's accepted rows: latency.
        dict(name="accept b1", op="accept", b=1, kv_heads=4, dim=64, block=16, t_lo=5, t_hi=5,
             acc_lo=3, acc_hi=3, ctx_lo=100, ctx_hi=100, pool="bf16"),
        # A large batch of wide trees.
        dict(name="accept b256", op="accept", b=256, kv_heads=8, dim=128, block=16, t_lo=33,
             t_hi=64, acc_lo=1, acc_hi=9, ctx_lo=512, ctx_hi=4096, pool="bf16"),
        # The same kind of batch in an FP8 pool with large blocks.
        dict(name="accept b128 fp8", op="accept", b=128, kv_heads=8, dim=128, block=32, t_lo=8,
             t_hi=16, acc_lo=1, acc_hi=6, ctx_lo=64, ctx_hi=2048, pool="fp8"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of these ranges."""
    op = rng.choice(["attention", "attention", "attention", "verify", "verify", "accept"])
    t_hi = _log_int(rng, 1, MAX_NODES)
    t_lo = rng.randint(max(1, t_hi // 2), t_hi)
    shape = rng.choice(["chain", "tree"])
    if op == "attention":
        fp8 = rng.random() < 0.3
        kv_heads = rng.choice([1, 2, 4, 8])
        group = rng.choice([1, 2, 3, 4, 5, 8])
        b = _log_int(rng, 1, 64)
        # Not more cache or products than the largest listed case.
        room = 16 * 4608 * 8 * 64 * 8 // (b * kv_heads * max(64, t_hi * group))
        ctx_hi = _log_int(rng, 1, max(2, min(65536, room)))
        return dict(op=op, b=b, heads=kv_heads * group, kv_heads=kv_heads,
                    dim=128 if fp8 else rng.choice([64, 128]), block=rng.choice([8, 16, 32]),
                    t_lo=t_lo, t_hi=t_hi, shape=shape, ctx_lo=rng.randint(0, ctx_hi),
                    ctx_hi=ctx_hi, log=False, q_mult=rng.choice([1.0, 2.0]),
                    pool="fp8" if fp8 else "bf16")
    if op == "verify":
        b, vocab = _log_int(rng, 1, 256), _log_int(rng, 1000, 160000)
        t_hi = max(1, min(t_hi, 256 * 131072 * 6 // (b * vocab)))
        return dict(op=op, b=b, vocab=vocab, t_lo=max(1, t_hi - rng.randint(0, 6)), t_hi=t_hi,
                    shape=shape, draft=rng.random() < 0.6)
    fp8 = rng.random() < 0.4
    ctx_hi = _log_int(rng, 1, 4096)
    acc_hi = rng.randint(1, min(12, t_lo))
    return dict(op=op, b=_log_int(rng, 1, 256), kv_heads=rng.choice([1, 2, 4, 8]),
                dim=rng.choice([64, 128]), block=rng.choice([8, 16, 32]), t_lo=t_lo, t_hi=t_hi,
                acc_lo=rng.randint(1, acc_hi), acc_hi=acc_hi, ctx_lo=rng.randint(0, ctx_hi),
                ctx_hi=ctx_hi, pool="fp8" if fp8 else "bf16")


# ------------------------------------------------------------------ inputs
def _spread(lo, hi, n, log=False):
    """n whole numbers spread over [lo, hi]: the same ones for every seed."""
    at = [(i + 0.5) / n for i in range(n)]
    if log:
        return [int(math.exp(math.log(lo) + (math.log(hi) - math.log(lo)) * x)) for x in at]
    return [lo + int((hi - lo + 1) * x) for x in at]


def _shuffled(values, gen):
    return [values[i] for i in torch.randperm(len(values), generator=gen).tolist()]


def _trees(case, gen):
    """Tree sizes, and every node's parent within its tree (-1: the root)."""
    lens = _shuffled(_spread(case["t_lo"], case["t_hi"], case["b"]), gen)
    parents = []
    for n in lens:
        if case.get("shape", "tree") == "chain":
            up = list(range(n - 1))
        else:  # a random recursive tree in breadth-first order
            r = torch.rand(max(0, n - 1), generator=gen).tolist()
            up = sorted(int(x * (i + 1)) for i, x in enumerate(r))
        parents += [-1] + up
    return lens, parents


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _offsets(lens):
    cu = [0]
    for n in lens:
        cu.append(cu[-1] + n)
    return _ints(cu)


def _placed(case, tree_lens, gen):
    """Sequence lengths (context and tree), block tables and the pool's blocks."""
    ctx = _shuffled(_spread(case["ctx_lo"], case["ctx_hi"], case["b"], case.get("log", False)), gen)
    lens = [c + t for c, t in zip(ctx, tree_lens)]
    need = [-(-n // case["block"]) for n in lens]
    # A pool of a size that goes by the case alone, about a tenth of it free.
    most = sum(-(-c // case["block"]) for c in ctx) + sum(-(-t // case["block"]) for t in tree_lens)
    blocks = math.ceil(most * 1.1)
    perm = torch.randperm(blocks, generator=gen).to(torch.int32)
    tables = torch.full((case["b"], max(need)), -1, dtype=torch.int32)
    at = 0
    for s, n in enumerate(need):
        tables[s, :n] = perm[at:at + n]
        at += n
    return lens, tables.to(DEV), blocks


def _pool(case, blocks, gen):
    shape = (blocks, 2, case["kv_heads"], case["block"], case["dim"])
    x = torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(generator=gen)
    if case["pool"] == "bf16":
        return x
    return (x.float() * 64.0).clamp_(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def prepare(case, seed):
    gen = torch.Generator().manual_seed(seed)
    dev = torch.Generator(device=DEV).manual_seed(seed + 1)
    lens, parents = _trees(case, gen)
    s = dict(case=case, cu=_offsets(lens), parents=_ints(parents), max_tree=max(lens),
             total=sum(lens))
    rows = s["total"]
    if case["op"] == "attention":
        seq, s["tables"], blocks = _placed(case, lens, gen)
        s["pool"] = _pool(case, blocks, dev)
        s["seq_lens"], s["max_seq"] = _ints(seq), max(seq)
        q = torch.empty(rows, case["heads"], case["dim"], dtype=torch.bfloat16, device=DEV)
        s["q"] = q.normal_(generator=dev).mul_(case["q_mult"])
        s["out"] = torch.empty_like(q)
        s["scale"] = 1.0 / math.sqrt(case["dim"])
        s["kv_scales"] = (1.0 / 64, 1.0 / 64) if case["pool"] == "fp8" else None
        if own:
            from paged_kv_cache_287_gb300 import binding
            need = binding.pa_tree_attention_workspace_bytes(
                case["b"], s["max_tree"], case["heads"], case["kv_heads"], case["dim"])
            s["workspace"] = torch.empty(need, dtype=torch.uint8, device=DEV)
    elif case["op"] == "verify":
        logits = torch.empty(rows, case["vocab"], device=DEV).normal_(generator=dev).mul_(2.5)
        s["target"] = torch.softmax(logits, dim=1)
        noise = torch.empty_like(logits).normal_(generator=dev)
        draft = torch.softmax(logits.add_(noise, alpha=0.7), dim=1)
        del logits, noise
        # A node's token is drawn from the draft's distribution after its parent.
        base = torch.repeat_interleave(s["cu"][:-1].long(),
                                       (s["cu"][1:] - s["cu"][:-1]).long())
        up = base + s["parents"].long().clamp(min=0)
        u = torch.rand(rows, 1, dtype=torch.float64, device=DEV, generator=dev)
        tokens = torch.empty(rows, dtype=torch.int32, device=DEV)
        for lo in range(0, rows, 256):
            cdf = draft[up[lo:lo + 256]].double().cumsum(1)
            hit = torch.searchsorted(cdf, u[lo:lo + 256] * cdf[:, -1:], right=True)
            tokens[lo:lo + 256] = hit[:, 0].clamp(max=case["vocab"] - 1).to(torch.int32)
        s["tokens"] = tokens
        s["draft"] = draft if case["draft"] else None
        s["accept_u"] = torch.rand(rows, device=DEV, generator=dev)
        s["sample_u"] = torch.rand(case["b"], device=DEV, generator=dev)
        s["accepted"] = torch.empty(case["b"], s["max_tree"], dtype=torch.int32, device=DEV)
        s["num_accepted"] = torch.empty(case["b"], dtype=torch.int32, device=DEV)
        s["next"] = torch.empty(case["b"], dtype=torch.int32, device=DEV)
    else:
        seq, s["tables"], blocks = _placed(case, lens, gen)
        s["pool"] = _pool(case, blocks, dev)
        s["seq_lens"] = _ints(seq)
        counts = _shuffled(_spread(case["acc_lo"], case["acc_hi"], case["b"]), gen)
        path = torch.full((case["b"], s["max_tree"]), -1, dtype=torch.int32)
        for i, (n, t) in enumerate(zip(counts, lens)):
            pick = torch.randperm(t - 1, generator=gen)[:n - 1] + 1
            path[i, :n] = torch.cat([torch.zeros(1, dtype=torch.int64), pick.sort().values])
        s["path"], s["num_accepted"] = path.to(DEV), _ints(counts)
        s["new_lens"] = torch.empty(case["b"], dtype=torch.int32, device=DEV)
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    op = state["case"]["op"]
    if own:
        from paged_kv_cache_287_gb300 import binding
        if op == "attention":
            binding.pa_tree_attention(
                state["out"], state["q"], state["cu"], state["parents"], state["max_tree"],
                state["pool"], state["tables"], state["seq_lens"], state["max_seq"],
                state["scale"], state["workspace"], kv_scales=state["kv_scales"])
            return state["out"]
        if op == "verify":
            binding.pa_tree_verify(
                state["accepted"], state["num_accepted"], state["next"], state["target"],
                state["draft"], state["tokens"], state["cu"], state["parents"],
                state["accept_u"], state["sample_u"])
            return state["accepted"], state["num_accepted"], state["next"]
        binding.pa_tree_accept(state["pool"], state["path"], state["num_accepted"], state["cu"],
                               state["tables"], state["seq_lens"], state["new_lens"])
        return _bits(state["pool"]), state["new_lens"]
    if op == "attention":
        return _plain_attention(state)
    if op == "verify":
        return _plain_verify(state)
    return _plain_accept(state)


def _bits(pool):
    return pool if pool.dtype == torch.uint8 else pool.view(torch.int16)


def _node_rows(state, width):
    """Row of node t of every tree, [b, width] (clamped), and which of them are real."""
    lens = (state["cu"][1:] - state["cu"][:-1]).long()
    t = torch.arange(width, device=DEV)
    real = t < lens[:, None]
    return (state["cu"][:-1].long()[:, None] + t).clamp(max=state["total"] - 1), real, lens


def _plain_attention(state):
    """softmax(scale * q.K^T) V over the context and the node's ancestors, in 32 bits."""
    case, width = state["case"], state["max_tree"]
    b, kvh, d = case["b"], case["kv_heads"], case["dim"]
    g = case["heads"] // kvh
    rows, real, lens = _node_rows(state, width)
    kv = state["pool"][state["tables"].clamp(min=0).long()]  # [b, blocks, 2, kv heads, bs, d]
    if case["pool"] == "fp8":
        kv = kv.view(torch.float8_e4m3fn)
    k = kv[:, :, 0].permute(0, 2, 1, 3, 4).reshape(b, kvh, -1, d).float()
    v = kv[:, :, 1].permute(0, 2, 1, 3, 4).reshape(b, kvh, -1, d).float()
    del kv
    if case["pool"] == "fp8":
        k, v = k * state["kv_scales"][0], v * state["kv_scales"][1]
    # Ancestors: (I + parent)^64 of the tree's graph, by squaring.
    up = state["parents"].long()[rows]
    reach = torch.eye(width, device=DEV).repeat(b, 1, 1)
    reach = reach + (up[:, :, None] == torch.arange(width, device=DEV)) * real[:, :, None]
    for _ in range(6):
        reach = (torch.bmm(reach, reach) > 0).float()
    ctx = (state["seq_lens"].long() - lens)[:, None, None]
    pos = torch.arange(k.shape[2], device=DEV)[None, None, :]
    node = (pos - ctx).clamp(0, width - 1).expand(b, width, -1)
    sees = (pos < ctx) | ((pos < ctx + lens[:, None, None]) & (reach.gather(2, node) > 0))
    q = state["q"][rows].float().view(b, width, kvh, g, d).permute(0, 2, 3, 1, 4)
    x = torch.matmul(q.reshape(b, kvh, g * width, d), k.transpose(2, 3)) * state["scale"]
    x = x.view(b, kvh, g, width, -1).masked_fill_(~sees[:, None, None], -math.inf)
    p = x.sub_(x.amax(-1, keepdim=True)).exp_()
    o = torch.matmul(p.view(b, kvh, g * width, -1), v).view(b, kvh, g, width, d)
    o = (o / p.sum(-1, keepdim=True)).permute(0, 3, 1, 2, 4).reshape(b, width, kvh * g, d)
    seq = torch.repeat_interleave(torch.arange(b, device=DEV), lens, output_size=state["total"])
    return o[seq, torch.arange(state["total"], device=DEV) - state["cu"].long()[seq]].to(
        torch.bfloat16)


def _plain_verify(state):
    """The walk down every tree at once, node by node, in 64 bits."""
    case, width = state["case"], state["max_tree"]
    b, draft = case["b"], state["draft"]
    rows, real, _ = _node_rows(state, width)
    up, tok = state["parents"].long()[rows], state["tokens"].long()[rows]
    u = state["accept_u"].double()[rows]
    seq = torch.arange(b, device=DEV)
    cur = torch.zeros(b, dtype=torch.int64, device=DEV)  # the last accepted node
    left = state["target"][rows[:, 0]].double()  # what may still be drawn after it
    mass = torch.ones(b, dtype=torch.float64, device=DEV)
    on_path = torch.zeros(b, width, dtype=torch.bool, device=DEV)
    on_path[:, 0] = True
    for i in range(1, width):
        t, asked = tok[:, i], real[:, i] & (up[:, i] == cur) & (mass > 0)
        have = left[seq, t]
        if draft is None:
            ok = asked & (u[:, i] * mass < have)
            no = asked & ~ok
            left[seq, t] = torch.where(no, 0.0, have)
            mass = torch.where(no, mass - have, mass)
        else:
            q = draft[rows[seq, cur]].double()
            ok = asked & (u[:, i] * q[seq, t] * mass < have)
            no = asked & ~ok
            left = torch.where(no[:, None], (left / mass[:, None] - q).clamp(min=0), left)
            mass = torch.where(no, left.sum(1), mass)
        cur = torch.where(ok, i, cur)
        left = torch.where(ok[:, None], state["target"][rows[:, i]].double(), left)
        mass = torch.where(ok, 1.0, mass)
        on_path[:, i] = ok
    # The next token: the first whose cumulated weight exceeds u times the whole.
    cdf = left.cumsum(1)
    goal = state["sample_u"].double()[:, None] * cdf[:, -1:]
    last = (torch.arange(case["vocab"], device=DEV) * (left > 0)).amax(1)
    nxt = torch.searchsorted(cdf, goal, right=True)[:, 0].minimum(last)
    best = state["target"][rows[seq, cur]].argmax(1)
    nxt = torch.where(cdf[:, -1] > 0, nxt, best)
    count = on_path.sum(1)
    path = torch.sort((~on_path).to(torch.int8), dim=1, stable=True).indices
    path = torch.where(torch.arange(width, device=DEV) < count[:, None], path, -1)
    return path.int(), count.int(), nxt.int()


def _plain_accept(state):
    """Row path[i] of the tree to place i behind the context; the rest as it was."""
    pool, path = state["pool"], state["path"].long()
    block = state["case"]["block"]
    lens = state["cu"][1:] - state["cu"][:-1]
    base = (state["seq_lens"] - lens).long()[:, None]
    i = torch.arange(path.shape[1], device=DEV)
    used = i < state["num_accepted"][:, None]
    # Unused places repeat the root's move onto itself.
    src = base + torch.where(used, path, path[:, :1])
    dst = base + torch.where(used, i, 0)
    tables = state["tables"].long()
    rows = pool[tables.gather(1, src // block), :, :, src % block]
    pool[tables.gather(1, dst // block), :, :, dst % block] = rows
    return _bits(pool), (base[:, 0] + state["num_accepted"]).int()


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    t = _spread(case["t_lo"], case["t_hi"], case["b"])
    rows = sum(t)
    if case["op"] == "verify":
        # One row of the target's (and the draft's) probabilities per sequence, and a
        # value of each per node.
        sides = 2 if case["draft"] else 1
        return {"bytes": 4 * case["b"] * case["vocab"] * sides + 4 * rows * (3 + sides),
                "flops": case["b"] * case["vocab"] * 2 * sides}
    byte = 1 if case["pool"] == "fp8" else 2
    row = 2 * case["kv_heads"] * case["dim"] * byte
    if case["op"] == "accept":
        moved = sum(_spread(case["acc_lo"], case["acc_hi"], case["b"])) - case["b"]
        return {"bytes": 2 * moved * row + 4 * rows, "flops": 0}
    ctx = _spread(case["ctx_lo"], case["ctx_hi"], case["b"], case["log"])
    mean_t = rows / case["b"]
    keys = sum(ctx) + rows
    return {"bytes": keys * row + 4 * rows * case["heads"] * case["dim"] + 4 * keys // case["block"],
            "flops": 4 * case["heads"] * case["dim"] * (sum(ctx) * mean_t + rows * mean_t / 2)}


# ------------------------------------------------------------------ the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "attention":
        return _exact_attention(s)
    if case["op"] == "verify":
        return _exact_verify(s)
    return None  # a copy of bits has no computed numbers


def _exact_attention(s):
    case = s["case"]
    g, d = case["heads"] // case["kv_heads"], case["dim"]
    cu, parents = s["cu"].tolist(), s["parents"].tolist()
    out = torch.empty(s["total"], case["heads"], d, dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["seq_lens"].tolist()):
        lo, hi = cu[b], cu[b + 1]
        ids = s["tables"][b, :-(-n // case["block"])].long()
        hidden = torch.ones(hi - lo, n, dtype=torch.bool)
        hidden[:, :n - (hi - lo)] = False
        for i in range(hi - lo):
            j = i
            while j >= 0:
                hidden[i, n - (hi - lo) + j] = False
                j = parents[lo + j]
        hidden = hidden.to(DEV)
        for h in range(case["kv_heads"]):
            kv = s["pool"][ids, :, h].transpose(0, 1).reshape(2, -1, d)[:, :n]
            if case["pool"] == "fp8":
                kv = kv.contiguous().view(torch.float8_e4m3fn).float().double()
                k, v = kv[0] * s["kv_scales"][0], kv[1] * s["kv_scales"][1]
            else:
                k, v = kv[0].double(), kv[1].double()
            for a in range(h * g, (h + 1) * g):
                x = (s["q"][lo:hi, a].double() @ k.T) * s["scale"]
                out[lo:hi, a] = torch.softmax(x.masked_fill(hidden, -math.inf), dim=1) @ v
    return out


def _exact_verify(s):
    case = s["case"]
    cu, parents, tokens = s["cu"].tolist(), s["parents"].tolist(), s["tokens"].tolist()
    accept_u, sample_u = s["accept_u"].tolist(), s["sample_u"].tolist()
    paths = torch.full((case["b"], s["max_tree"]), -1, dtype=torch.int32)
    counts, nexts = [], []
    for b in range(case["b"]):
        lo, n = cu[b], cu[b + 1] - cu[b]
        path, going = [0], True
        while going:
            at, going = path[-1], False
            r, z = s["target"][lo + at].double(), 1.0
            for c in range(at + 1, n):
                if parents[lo + c] != at or z <= 0:
                    continue
                x = tokens[lo + c]
                if s["draft"] is None:
                    if accept_u[lo + c] * z < r[x].item():
                        path.append(c)
                        going = True
                        break
                    z -= r[x].item()
                    r[x] = 0.0
                else:
                    q = s["draft"][lo + at].double()
                    if accept_u[lo + c] * q[x].item() * z < r[x].item():
                        path.append(c)
                        going = True
                        break
                    r = (r / z - q).clamp(min=0)
                    z = r.sum().item()
        paths[b, :len(path)] = torch.tensor(path)
        counts.append(len(path))
        whole = r.sum().item()
        if whole > 0:
            over = (r.cumsum(0) > sample_u[b] * whole).nonzero()
            nexts.append(over[0].item() if len(over) else r.nonzero()[-1].item())
        else:
            nexts.append(s["target"][lo + path[-1]].argmax().item())
    return paths, torch.tensor(counts, dtype=torch.int32), torch.tensor(nexts, dtype=torch.int32)
