"""The operators of a step over a paged KV cache held in 4 bits, as cases to be timed.

A 4-bit pool is uint8 ``[blocks, kv_heads, 2, block * (dim / 2 + dim / 16)]``: of every
(block, head) first K, then V, each ``block`` rows of ``dim / 2`` bytes (element 2i is the low
nibble of byte i, an e2m1 code) followed by ``block`` rows of ``dim / 16`` e4m3 scales, one per
16 elements.  An element is code * scale * (k_scale or v_scale).

* ``decode``: one query token per sequence attends to its cached tokens;
* ``store``: new rows are quantised into their slots and read back, as the attention sees them;
* ``load``: the rows of cached contexts are read back;
* ``rotate``: a projection's q, k, v rows: norms of q and k per head, rotary positions of one
  axis or of several, K and V into a bf16 or FP8 pool, all in one pass;
* ``step``: the rotation of a step's new tokens with the write into a 4-bit pool, then the
  attention over it.

``own`` false: the plain forms below.  ``own`` true: the library's entry points.
"""

import math

import torch

own = False

DEV = "cuda"
EPS = 1e-6


def listed():
    """The cases, each with what it stands for."""
    return [
        # Four short chats of a small model: latency of the smallest call.
        dict(name="decode b4 short", op="decode", b=4, heads=32, kv_heads=4, dim=64, block=16,
             ctx_lo=1, ctx_hi=128, log=False, q_mult=1.0),
        # A large serving batch of ordinary contexts.
        dict(name="decode b256", op="decode", b=256, heads=32, kv_heads=8, dim=128, block=16,
             ctx_lo=512, ctx_hi=4096, log=False, q_mult=1.0),
        # Long skewed contexts and a sharp softmax.
        dict(name="decode long b32", op="decode", b=32, heads=32, kv_heads=8, dim=128, block=16,
             ctx_lo=1024, ctx_hi=131072, log=True, q_mult=2.0),
        # The widest groups, blocks of 32 tokens, odd lengths that end inside a block.
        dict(name="decode wide b47", op="decode", b=47, heads=64, kv_heads=8, dim=128, block=32,
             ctx_lo=33, ctx_hi=2111, log=False, q_mult=1.0),
        # The new tokens of a serving batch's decoding step.
        dict(name="store b256", op="store", n=256, kv_heads=8, dim=128, block=16),
        # A mixed step's new tokens: prompt chunks and decoding sequences.
        dict(name="store 4344", op="store", n=4344, kv_heads=8, dim=128, block=16),
        # A short context of a small model read back.
        dict(name="load 517", op="load", n=517, kv_heads=4, dim=64, block=8),
        # Cached contexts read back before a prompt's next chunk.
        dict(name="load 32768", op="load", n=32768, kv_heads=8, dim=128, block=16),
        # One token of a small model: latency.
        dict(name="rotate b1", op="rotate", n=1, heads=32, kv_heads=4, dim=64, block=16, rot=64,
             axes=1, interleaved=False, norm=True, pool="bf16"),
        # A serving batch's tokens into an FP8 pool: norms, part of each head turned, in
        # neighbouring pairs.
        dict(name="rotate b256 fp8", op="rotate", n=256, heads=40, kv_heads=8, dim=128,
             block=16, rot=64, axes=1, interleaved=True, norm=True, pool="fp8"),
        # Prompt chunks with images: time, height and width positions, norms.
        dict(name="rotate 4344 axes", op="rotate", n=4344, heads=32, kv_heads=8, dim=128,
             block=16, rot=128, axes=3, interleaved=False, norm=True, pool="bf16"),
        # A whole step of a serving batch: rotation and 4-bit write, then the attention.
        dict(name="step b64", op="step", b=64, heads=32, kv_heads=8, dim=128, block=16,
             ctx_lo=512, ctx_hi=4096, log=False, q_mult=1.0, rot=128, axes=1, interleaved=False,
             norm=False, pool="fp4"),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    """One more case of these ranges."""
    op = rng.choice(["decode", "decode", "store", "load", "rotate", "rotate", "step"])
    kv_heads = rng.choice([1, 2, 4, 8])
    dim, block = rng.choice([64, 128]), rng.choice([8, 16, 32])
    if op in ("store", "load"):
        return dict(op=op, n=_log_int(rng, 1, 32768 if op == "load" else 8192),
                    kv_heads=kv_heads, dim=dim, block=block)
    heads = kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8])
    turn = dict(rot=rng.choice([16, 32, 48, 64] + [96, 128] * (dim == 128)),
                axes=rng.choice([1, 1, 2, 3]), interleaved=rng.random() < 0.4)
    if op == "rotate":
        return dict(op=op, n=_log_int(rng, 1, 4344), heads=heads, kv_heads=kv_heads, dim=dim,
                    block=block, norm=rng.random() < 0.6, pool=rng.choice(["bf16", "fp8"]),
                    **turn)
    b = _log_int(rng, 1, 256)
    # Not more cache than the largest listed case.
    ctx_hi = _log_int(rng, 1, max(2, min(131072, 256 * 2304 * 8 // (b * kv_heads))))
    case = dict(op=op, b=b, heads=heads, kv_heads=kv_heads, dim=dim, block=block,
                ctx_lo=rng.randint(1, ctx_hi), ctx_hi=ctx_hi, log=False,
                q_mult=rng.choice([1.0, 2.0]))
    # A 4-bit step is much coarser than the last bits of a norm: the step's rotation goes
    # without one here.
    return dict(case, norm=False, pool="fp4", **turn) if op == "step" else case


# ------------------------------------------------------------------ inputs
def _spread(lo, hi, n, log=False):
    """n whole numbers spread over [lo, hi]: the same ones for every seed."""
    at = [(i + 0.5) / n for i in range(n)]
    if log:
        return [int(math.exp(math.log(lo) + (math.log(hi) - math.log(lo)) * x)) for x in at]
    return [lo + int((hi - lo + 1) * x) for x in at]


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device=DEV)


def _tile(case):
    """Bytes of K (or V) of one (block, head) of a 4-bit pool, and of its codes."""
    codes = case["block"] * case["dim"] // 2
    return codes + case["block"] * case["dim"] // 16, codes


def _scales(gen):
    """Per-tensor scales as a calibration leaves them: its largest element over 6 * 448."""
    return tuple((5.0 + torch.rand((), generator=gen).item()) / 2688 for _ in range(2))


def _fp4_pool(case, blocks, gen, scales):
    """A pool of quantised normal numbers."""
    bs, d, heads = case["block"], case["dim"], case["kv_heads"]
    tile, split = _tile(case)
    pool = torch.empty(blocks, heads, 2, tile, dtype=torch.uint8, device=DEV)
    step = max(1, (1 << 25) // (heads * bs * d))
    for lo in range(0, blocks, step):
        n = min(step, blocks - lo)
        for side, g in enumerate(scales):
            x = torch.empty(n, heads, bs, d, dtype=torch.bfloat16, device=DEV)
            codes, sc = _quantise(x.normal_(generator=gen), g)
            pool[lo:lo + n, :, side, :split] = codes.view(n, heads, -1)
            pool[lo:lo + n, :, side, split:] = sc.view(n, heads, -1)
    return pool


def _context(case, s, gen, dev):
    """Lengths, tables and a 4-bit pool of a decoding batch."""
    b, bs = case["b"], case["block"]
    lens = _spread(case["ctx_lo"], case["ctx_hi"], b, case["log"])
    need = [-(-n // bs) for n in lens]
    # A pool of a size that goes by the case alone, about a tenth of it free.
    blocks = math.ceil(sum(need) * 1.1)
    order = torch.randperm(b, generator=gen).tolist()
    perm = torch.randperm(blocks, generator=gen).to(torch.int32)
    tables = torch.full((b, max(need)), -1, dtype=torch.int32)
    at, slots = 0, []
    for row, i in enumerate(order):
        tables[row, :need[i]] = perm[at:at + need[i]]
        at += need[i]
        last = lens[i] - 1
        slots.append(int(tables[row, last // bs]) * bs + last % bs)
    s["seq_lens"], s["max_seq"] = _ints([lens[i] for i in order]), max(lens)
    s["tables"], s["slots"] = tables.to(DEV), _ints(slots)
    s["positions"] = (s["seq_lens"] - 1).expand(case.get("axes", 1), b).contiguous()
    s["kv_scales"] = _scales(gen)
    s["pool"] = _fp4_pool(case, blocks, dev, s["kv_scales"])
    s["scale"] = 1.0 / math.sqrt(case["dim"])
    s["q"] = torch.empty(b, case["heads"], case["dim"], dtype=torch.bfloat16, device=DEV)
    s["q"].normal_(generator=dev).mul_(case["q_mult"])
    s["out"] = torch.empty_like(s["q"])
    if own:
        from paged_kv_cache_287_gb300 import binding
        need = binding.pa_decode_fp4_workspace_bytes(b, case["heads"], case["kv_heads"],
                                                     case["dim"])
        s["workspace"] = torch.empty(need, dtype=torch.uint8, device=DEV)


def _projected(case, s, n, gen, dev, positions):
    """A projection's rows and what turns them."""
    width = (case["heads"] + 2 * case["kv_heads"]) * case["dim"]
    s["qkv"] = torch.empty(n, width, dtype=torch.bfloat16, device=DEV).normal_(generator=dev)
    s["q_weight"] = s["k_weight"] = None
    if case["norm"]:
        for name in ("q_weight", "k_weight"):
            w = torch.empty(case["dim"], device=DEV).normal_(generator=dev).mul_(0.2).add_(1.0)
            s[name] = w.to(torch.bfloat16)
    pairs = case["rot"] // 2
    freq = 500000.0 ** (-torch.arange(pairs, dtype=torch.float64, device=DEV) / pairs)
    angle = torch.arange(positions, dtype=torch.float64, device=DEV)[:, None] * freq
    s["cos_sin"] = torch.cat([angle.cos(), angle.sin()], 1).float()
    s["pair_axis"] = None
    if case["axes"] > 1:  # the first pairs turn with the first axis, and so on
        s["pair_axis"] = _ints([i * case["axes"] // pairs for i in range(pairs)])


def _slots(case, n, gen):
    """Slots of n tokens in blocks of their own, in an order of their own, and the pool's blocks."""
    bs = case["block"]
    used = -(-n // bs)
    blocks = math.ceil(used * 1.1) + 1
    perm = torch.randperm(blocks, generator=gen)[:used]
    slots = (perm[:, None] * bs + torch.arange(bs)).reshape(-1)[:n]
    return slots.to(torch.int32).to(DEV), blocks


def prepare(case, seed):
    gen = torch.Generator().manual_seed(seed)
    dev = torch.Generator(device=DEV).manual_seed(seed + 1)
    s = dict(case=case)
    if case["op"] in ("decode", "step"):
        _context(case, s, gen, dev)
        if case["op"] == "step":
            _projected(case, s, case["b"], gen, dev, case["ctx_hi"])
        return s
    n = case["n"]
    s["slots"], blocks = _slots(case, n, gen)
    rows = (n, case["kv_heads"], case["dim"])
    if case["op"] == "rotate":
        _projected(case, s, n, gen, dev, 8192)
        # Text counts every axis up; an image's tokens share their time.
        at = torch.arange(n)
        side = max(1, math.isqrt(n // 2))
        axes = torch.stack([at // 7, at // side % side, at % side])[:case["axes"]]
        s["positions"] = ((axes if case["axes"] > 1 else at[None]) + 100).to(torch.int32).to(DEV)
        s["q"] = torch.empty(n, case["heads"], case["dim"], dtype=torch.bfloat16, device=DEV)
        shape = (blocks, 2, case["kv_heads"], case["block"], case["dim"])
        s["pool"] = torch.empty(shape, dtype=torch.bfloat16, device=DEV).normal_(generator=dev)
        s["kv_scales"] = None
        if case["pool"] == "fp8":
            s["kv_scales"] = (1.0 / 64, 1.0 / 32)
            s["pool"] = s["pool"].mul_(64.0).to(torch.float8_e4m3fn).view(torch.uint8)
        return s
    s["kv_scales"] = _scales(gen)
    s["pool"] = _fp4_pool(case, blocks, dev, s["kv_scales"])
    s["k_out"] = torch.empty(rows, dtype=torch.bfloat16, device=DEV)
    s["v_out"] = torch.empty_like(s["k_out"])
    if case["op"] == "store":
        s["k_new"] = torch.empty_like(s["k_out"]).normal_(generator=dev)
        s["v_new"] = torch.empty_like(s["k_out"]).normal_(generator=dev)
    return s


# ------------------------------------------------------------------ one pass
def run(state):
    s, op = state, state["case"]["op"]
    if own:
        from paged_kv_cache_287_gb300 import binding
        if op in ("rotate", "step"):
            binding.pa_qkv_rope_write(
                s["q"], s["qkv"], s["pool"], s["slots"], s["positions"], s["cos_sin"],
                q_weight=s["q_weight"], k_weight=s["k_weight"], eps=EPS,
                pair_axis=s["pair_axis"], interleaved=s["case"]["interleaved"],
                kv_scales=s["kv_scales"])
        if op == "rotate":
            return s["q"], _values(s)
        if op in ("decode", "step"):
            binding.pa_decode_fp4(s["out"], s["q"], s["pool"], s["tables"], s["seq_lens"],
                                  s["max_seq"], s["scale"], *s["kv_scales"], s["workspace"])
            return s["out"] if op == "decode" else (s["q"], s["out"])
        if op == "store":
            binding.pa_cache_write_fp4(s["pool"], s["k_new"], s["v_new"], s["slots"],
                                       *s["kv_scales"])
        binding.pa_cache_read_fp4(s["k_out"], s["v_out"], s["pool"], s["slots"],
                                  *s["kv_scales"])
        return s["k_out"], s["v_out"]
    if op == "decode":
        return _plain_attention(s, s["q"])
    if op == "step":
        q = _plain_rotate(s)
        return q, _plain_attention(s, q)
    if op == "rotate":
        return _plain_rotate(s), _values(s)
    if op == "store":
        _put_fp4(s, s["k_new"], s["v_new"])
    return _plain_rows(s)


def _values(s):
    return s["pool"] if s["pool"].dtype != torch.uint8 else s["pool"].view(torch.float8_e4m3fn)


def _quantise(x, g):
    """Codes, two a byte, and scales of rows of x whose tensor's scale is g."""
    x = x.float().unflatten(-1, (-1, 16))
    g = torch.tensor(g, device=x.device)  # binary32, and a divisor that is divided by
    sc = (x.abs().amax(-1) / (g * 6)).clamp(max=448.0).to(torch.float8_e4m3fn)
    d = (sc.float() * g)[..., None]
    a = torch.where(d > 0, x.abs() / d, 0.0)
    # Nearest of 0, .5, 1, 1.5, 2, 3, 4, 6; a tie goes to the even code.
    code = ((a > 0.25).to(torch.uint8) + (a >= 0.75) + (a > 1.25) + (a >= 1.75) + (a > 2.5)
            + (a >= 3.5) + (a > 5.0))
    code = (code + 8 * ((d > 0) & torch.signbit(x))).to(torch.uint8).flatten(-2)
    return code[..., 0::2] | (code[..., 1::2] << 4), sc.view(torch.uint8)


def _lut():
    """Both elements of every byte of codes."""
    one = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=DEV)
    one = torch.cat([one, -one])
    at = torch.arange(256, device=DEV)
    return torch.stack([one[at % 16], one[at // 16]], 1)


def _put_fp4(s, k, v):
    """Rows into the 4-bit pool's slots."""
    case = s["case"]
    bs, d = case["block"], case["dim"]
    slots = s["slots"].long()
    _, split = _tile(case)
    for side, (x, g) in enumerate(zip((k, v), s["kv_scales"])):
        codes, sc = _quantise(x, g)
        part = s["pool"][:, :, side]
        part[:, :, :split].unflatten(2, (bs, d // 2))[slots // bs, :, slots % bs] = codes
        part[:, :, split:].unflatten(2, (bs, d // 16))[slots // bs, :, slots % bs] = sc


def _side(s, rows, side):
    """K or V, in 32 bits, of tiles [..., 2, tile] of the pool."""
    case = s["case"]
    _, split = _tile(case)
    x = _lut().index_select(0, rows[..., side, :split].int().flatten())
    x = x.view(*rows.shape[:-2], case["block"], case["dim"] // 16, 16)
    sc = rows[..., side, split:].contiguous().view(torch.float8_e4m3fn).float()
    x = x.mul_(sc.view(*x.shape[:-1], 1)).mul_(torch.tensor(s["kv_scales"][side], device=DEV))
    return x.flatten(-2)


def _plain_rows(s):
    """The slots' K and V rows."""
    case = s["case"]
    bs, d = case["block"], case["dim"]
    slots = s["slots"].long()
    _, split = _tile(case)
    out = []
    for side, g in enumerate(s["kv_scales"]):
        part = s["pool"][:, :, side]
        codes = part[:, :, :split].unflatten(2, (bs, d // 2))[slots // bs, :, slots % bs]
        sc = part[:, :, split:].unflatten(2, (bs, d // 16))[slots // bs, :, slots % bs]
        x = _lut()[codes.long()].view(*codes.shape[:2], d // 16, 16)
        x = x * sc.view(torch.float8_e4m3fn).float()[..., None] * torch.tensor(g, device=DEV)
        out.append(x.flatten(-2).to(torch.bfloat16))
    return tuple(out)


def _plain_attention(s, q):
    """softmax(scale * q.K^T) V over every sequence's tokens, in 32 bits."""
    case = s["case"]
    b, kvh, d = case["b"], case["kv_heads"], case["dim"]
    g = case["heads"] // kvh
    rows = s["pool"][s["tables"].clamp(min=0).long()].transpose(1, 2)  # [b, kv heads, blocks, ..]
    k = _side(s, rows, 0).reshape(b, kvh, -1, d)
    x = torch.matmul(q.float().view(b, kvh, g, d), k.transpose(2, 3)) * s["scale"]
    del k
    pos = torch.arange(x.shape[-1], device=DEV)
    x.masked_fill_(pos >= s["seq_lens"].long()[:, None, None, None], -math.inf)
    p = x.sub_(x.amax(-1, keepdim=True)).exp_()
    o = torch.matmul(p, _side(s, rows, 1).reshape(b, kvh, -1, d))
    return (o / p.sum(-1, keepdim=True)).view(b, kvh * g, d).to(torch.bfloat16)


def _turned(x, cos, sin, interleaved):
    """The first 2 * pairs elements of every head turned by their pairs' angles."""
    rot = 2 * cos.shape[-1]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if interleaved else (x[..., :rot // 2],
                                                                   x[..., rot // 2:rot])
    turned = (a * cos - b * sin, b * cos + a * sin)
    turned = torch.stack(turned, -1).flatten(-2) if interleaved else torch.cat(turned, -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_rotate(s):
    """q turned; K turned and V in the pool."""
    case = s["case"]
    hq, hk, d = case["heads"], case["kv_heads"], case["dim"]
    q, k, v = s["qkv"].view(-1, hq + 2 * hk, d).split([hq, hk, hk], 1)
    q, k = q.float(), k.float()
    if case["norm"]:
        q = q * torch.rsqrt(q.square().mean(-1, keepdim=True) + EPS) * s["q_weight"].float()
        k = k * torch.rsqrt(k.square().mean(-1, keepdim=True) + EPS) * s["k_weight"].float()
    pairs = case["rot"] // 2
    if s["pair_axis"] is None:
        pos = s["positions"][0].long()[:, None]
    else:
        pos = s["positions"].long()[s["pair_axis"].long()].T
    at = torch.arange(pairs, device=DEV)
    cos, sin = s["cos_sin"][pos, at][:, None], s["cos_sin"][pos, at + pairs][:, None]
    q, k = (_turned(x, cos, sin, case["interleaved"]).to(torch.bfloat16) for x in (q, k))
    if case["pool"] == "fp4":
        _put_fp4(s, k, v)
        return q
    slots, bs = s["slots"].long(), case["block"]
    for side, x in enumerate((k, v)):
        if case["pool"] == "fp8":
            g = torch.tensor(s["kv_scales"][side], device=DEV)
            x = (x.float() / g).clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)
        s["pool"][:, side].transpose(1, 2)[slots // bs, slots % bs] = x
    return q


# ------------------------------------------------------------------ what a pass cannot do without
def work(case):
    row = 2 * case["kv_heads"] * case["dim"]  # elements of K and V of a token
    if case["op"] == "store":  # the new rows read, codes written and read, rows written
        return {"bytes": case["n"] * row * (2 + 2 * 9 / 16 + 2), "flops": 4 * case["n"] * row}
    if case["op"] == "load":
        return {"bytes": case["n"] * row * (9 / 16 + 2), "flops": 2 * case["n"] * row}
    done = {"bytes": 0, "flops": 0}
    if case["op"] in ("rotate", "step"):
        n = case["n"] if case["op"] == "rotate" else case["b"]
        q = case["heads"] * case["dim"]
        byte = {"bf16": 2, "fp8": 1, "fp4": 9 / 16}[case["pool"]]
        done["bytes"] = n * (2 * (q + row) + 2 * q + byte * row + 4 * case["rot"])
        done["flops"] = n * (q + row / 2) * (8 if case["norm"] else 4)
    if case["op"] in ("decode", "step"):
        keys = sum(_spread(case["ctx_lo"], case["ctx_hi"], case["b"], case["log"]))
        done["bytes"] += (keys * row * 9 / 16 + 4 * case["b"] * case["heads"] * case["dim"]
                          + 4 * keys // case["block"])
        done["flops"] += 4 * case["heads"] * case["dim"] * keys
    return done


# ------------------------------------------------------------------ the definitions, in 64 bits
def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "decode":
        return _exact_attention(s, s["q"].double())
    if case["op"] in ("rotate", "step"):
        return _exact_rotate(s)
    if case["op"] == "store":
        return tuple(_exact_value(*_exact_codes(x, g), g)
                     for x, g in zip((s["k_new"], s["v_new"]), s["kv_scales"]))
    return _exact_rows(s)


def _e4m3(byte):
    """The value of e4m3 codes, from the format's definition."""
    e, m = (byte // 8 % 16).double(), (byte % 8).double()
    x = torch.where(e > 0, (8 + m) * 2.0 ** (e - 10), m * 2.0 ** -9)
    x = torch.where(byte % 128 == 127, math.nan, x)
    return torch.where(byte >= 128, -x, x)


def _e2m1(code):
    e, m = (code // 2 % 4).double(), (code % 2).double()
    x = torch.where(e > 0, (2 + m) * 2.0 ** (e - 2), m / 2)
    return torch.where(code >= 8, -x, x)


def _nearest(x, grid):
    """Index of the nearest of an increasing grid's values; between two, the even index."""
    up = torch.searchsorted(grid, x.contiguous()).clamp(1, len(grid) - 1)
    low, high = x - grid[up - 1], grid[up] - x
    return torch.where((high < low) | ((high == low) & (up % 2 == 0)), up, up - 1)


def _exact_codes(x, g):
    x = x.double().unflatten(-1, (-1, 16))
    g = float(torch.tensor(g))
    sc = _nearest(x.abs().amax(-1) / (6 * g), _e4m3(torch.arange(127, device=DEV)))
    d = (_e4m3(sc) * g)[..., None]
    code = _nearest(torch.where(d > 0, x.abs() / d, 0.0), _e2m1(torch.arange(8, device=DEV)))
    return code + 8 * ((d > 0) & torch.signbit(x)), sc


def _exact_value(code, sc, g):
    return (_e2m1(code) * _e4m3(sc)[..., None] * float(torch.tensor(g))).flatten(-2)


def _exact_rows(s):
    """The rows in the slots, every byte found by its offset in the pool."""
    case, pool = s["case"], s["pool"].flatten()
    block, d, heads = case["block"], case["dim"], case["kv_heads"]
    tile = block * d * 9 // 16
    slot = s["slots"].long()[:, None, None]
    head, i = torch.arange(heads, device=DEV)[:, None], torch.arange(d, device=DEV)
    out = []
    for side, g in enumerate(s["kv_scales"]):
        at = ((slot // block * heads + head) * 2 + side) * tile
        codes = pool[at + slot % block * (d // 2) + i // 2].long()
        sc = pool[at + block * d // 2 + slot % block * (d // 16) + i // 16].long()
        x = _e2m1(torch.where(i % 2 == 1, codes // 16, codes % 16)) * _e4m3(sc)
        out.append(x * float(torch.tensor(g)))
    return tuple(out)


def _exact_attention(s, q, new=None):
    """Sequence after sequence; `new`: the last token's K and V rows."""
    case = s["case"]
    block, d, kvh = case["block"], case["dim"], case["kv_heads"]
    g = case["heads"] // kvh
    out = torch.empty(q.shape, dtype=torch.float64, device=DEV)
    for b, n in enumerate(s["seq_lens"].tolist()):
        ids = s["tables"][b, :-(-n // block)].long()
        for h in range(kvh):
            kv = []
            for side in (0, 1):
                raw = s["pool"][ids, h, side].long()
                codes, sc = raw.split([block * d // 2, block * d // 16], 1)
                code = torch.stack([codes % 16, codes // 16], 2).view(-1, d // 16, 16)[:n]
                kv.append(_exact_value(code, sc.reshape(-1, d // 16)[:n], s["kv_scales"][side]))
                if new is not None:
                    kv[side][n - 1] = new[side][b, h]
            x = (q[b, h * g:(h + 1) * g] @ kv[0].T) * s["scale"]
            out[b, h * g:(h + 1) * g] = torch.softmax(x, 1) @ kv[1]
    return out


def _exact_rotate(s):
    case = s["case"]
    hq, hk, d, rot = case["heads"], case["kv_heads"], case["dim"], case["rot"]
    x = s["qkv"].double().view(-1, hq + 2 * hk, d).clone()
    if case["norm"]:
        for w, lo, hi in ((s["q_weight"], 0, hq), (s["k_weight"], hq, hq + hk)):
            size = torch.sqrt((x[:, lo:hi] ** 2).sum(2, keepdim=True) / d + EPS)
            x[:, lo:hi] = x[:, lo:hi] / size * w.double()
    # Every pair as a complex number, turned by its own.
    pair = torch.arange(rot // 2)
    first = 2 * pair if case["interleaved"] else pair
    second = first + 1 if case["interleaved"] else pair + rot // 2
    for j in pair.tolist():
        axis = 0 if s["pair_axis"] is None else int(s["pair_axis"][j])
        at = s["cos_sin"][s["positions"][axis].long()].double()
        turn = torch.complex(at[:, j], at[:, j + rot // 2])[:, None]
        z = torch.complex(x[:, :hq + hk, first[j]], x[:, :hq + hk, second[j]]) * turn
        x[:, :hq + hk, first[j]], x[:, :hq + hk, second[j]] = z.real, z.imag
    q, k, v = x[:, :hq], x[:, hq:hq + hk], x[:, hq + hk:]
    if case["op"] == "step":
        new = [_exact_value(*_exact_codes(y.to(torch.bfloat16), g), g)
               for y, g in zip((k, v), s["kv_scales"])]
        return q, _exact_attention(s, q.to(torch.bfloat16).double(), new)
    pool = s["pool"]
    pool = (pool if case["pool"] == "bf16" else pool.view(torch.float8_e4m3fn)).double()
    block = case["block"]
    for i, slot in enumerate(s["slots"].tolist()):
        for side, y in enumerate((k, v)):
            y = y[i]
            if case["pool"] == "fp8":
                y = (y.to(torch.bfloat16).double() / s["kv_scales"][side]).clamp(-448, 448)
            pool[slot // block, side, :, slot % block] = y
    return q, pool
