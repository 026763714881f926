"""Rotary positions, the writes that apply them and attention over a 4-bit cache: cases, plain forms and the calls that a user makes.

Four operators around the paged cache that this library writes, moves and attends to:

* rotate     new tokens' heads turned by their positions (part of the head, half or interleaved pairs, scaled frequencies, its transpose)
* write      queries and keys rotated, keys and values appended to the pages of a 16-bit cache
* write4     the same into a 4-bit cache: e2m1 codes with one e4m3 scale a group of 16 elements
* attention4 attention of new tokens (one, or a chunk) of every request over a 4-bit cache

A row of a 4-bit cache holds heads * dim / 2 bytes of codes (element 2 i in the low half of byte i), then heads * dim / 16 bytes of
scales, and is filled up to a multiple of 16 bytes.

``run`` computes a case either with elementary torch operations (``own`` false) or with the library's
entry points (``own`` true) on what ``prepare`` made.
"""
import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
_GRID = (0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0)  # what the codes 0 to 7 stand for; 8 to 15 are their negatives


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _rope(rot, offset=0, interleaved=False, scaling="none", factor=1.0, base=10000.0):
    return dict(rot=rot, offset=offset, interleaved=interleaved, scaling=scaling, factor=factor, base=base)


def _rotate(tokens, heads, dk, max_pos, rope, **kw):
    return dict(dict(op="rotate", tokens=tokens, heads=heads, dk=dk, max_pos=max_pos, inverse=False, mix=1, dtype="bf16", **rope), **kw)


def _write(op, reqs, q, kv, heads, kv_heads, dk, dv, block, layout, rope, **kw):
    c = dict(op=op, reqs=reqs, q_lo=q[0], q_hi=q[1], kv_lo=kv[0], kv_hi=kv[1], heads=heads, kv_heads=kv_heads, dk=dk, dv=dv, block=block,
             layout=layout, shift=0, mix=1, dtype="bf16", **rope)
    return dict(c, **kw)


def _attention(reqs, q, kv, heads, kv_heads, dk, block, layout, **kw):
    c = dict(op="attention4", reqs=reqs, q_lo=q[0], q_hi=q[1], kv_lo=kv[0], kv_hi=kv[1], heads=heads, kv_heads=kv_heads, dk=dk, dv=dk, block=block,
             layout=layout, causal=True, window=0, mix=1, dtype="bf16")
    return dict(c, **kw)


def listed():
    return [
        # the queries of a small decode step, far out in a scaled context: the smallest calls, where latency counts
        dict(_rotate(24, 32, 128, 1000000, _rope(128, scaling="yarn", factor=16.0)), name="rotate_decode"),
        # a prefill chunk's queries with the rotary part at the end of a 192-wide head, interleaved pairs
        dict(_rotate(8000, 20, 192, 32768, _rope(64, offset=128, interleaved=True)), name="rotate_chunk_part"),
        # one layer's write of a decode batch of the 32-layer preset (8 key heads of 128, pages of 16)
        dict(_write("write", 64, (1, 1), (4096, 12288), 32, 8, 128, 128, 16, "separate", _rope(128, scaling="bands", factor=8.0, base=500000.0)),
             name="write_decode"),
        # one layer's write of the latent preset: rows of 576, the last 64 rotary, no values and no queries
        dict(_write("write", 64, (1, 2), (200, 4000), 0, 1, 576, 0, 64, "latent", _rope(64, offset=512, interleaved=True), dtype="fp16"),
             name="write_latent"),
        # one layer's write of several prompts, pages of the 48-layer preset's layout
        dict(_write("write", 8, (1000, 2000), (1000, 4000), 32, 8, 128, 128, 16, "blocks_first", _rope(128)), name="write_prompts"),
        # the decode batch into 4 bits, after evictions: positions run ahead of the slots
        dict(_write("write4", 64, (1, 1), (2000, 4096), 32, 8, 128, 128, 16, "separate", _rope(128, scaling="linear", factor=4.0), shift=100000),
             name="write4_decode"),
        # prompts into 4 bits, half of a 64-wide head rotated
        dict(_write("write4", 5, (700, 3000), (700, 4000), 16, 4, 64, 64, 24, "kv_first", _rope(32), dtype="fp16"), name="write4_prompts_part"),
        # larger prompts into 4 bits
        dict(_write("write4", 8, (1000, 2000), (1000, 4000), 32, 8, 128, 128, 16, "blocks_first", _rope(128)), name="write4_prompts"),
        # a few requests verifying up to four drafted tokens each under a sliding window: the smallest attention calls
        dict(_attention(5, (1, 4), (100, 700), 14, 2, 64, 24, "kv_first", window=256, dtype="fp16"), name="attn4_verify_small"),
        # a decode batch of the 32-layer preset with long contexts
        dict(_attention(64, (1, 1), (4096, 12288), 32, 8, 128, 16, "separate"), name="attn4_decode_long"),
        # one long request
        dict(_attention(1, (3, 3), (120000, 120000), 32, 8, 128, 64, "blocks_first"), name="attn4_one_long"),
        # large prefill chunks over earlier context, pages of the 48-layer preset's layout
        dict(_attention(4, (2048, 4096), (4096, 8192), 32, 8, 128, 16, "blocks_first"), name="attn4_chunk_large"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _draw_rope(rng, dk):
    rot = rng.choice([x for x in (16, 32, 64, 96, 128) if x <= dk])
    return _rope(rot, offset=rng.choice([0, dk - rot]), interleaved=rng.random() < 0.4, base=rng.choice([10000.0, 500000.0, 1000000.0]),
                 **rng.choice([dict(scaling="none"), dict(scaling="linear", factor=4.0), dict(scaling="base", factor=8.0),
                               dict(scaling="bands", factor=8.0), dict(scaling="yarn", factor=32.0)]))


def draw(rng):
    op = rng.choice(["rotate", "write", "write4", "write4", "attention4", "attention4", "attention4"])
    while True:
        c = dict(op=op, mix=rng.randrange(1 << 30), dtype=rng.choice(["bf16", "fp16"]))
        if op == "rotate":
            dk = rng.choice([16, 64, 80, 96, 128, 192, 256])
            c.update(_rotate(_log(rng, 1, 16384), _log(rng, 1, 128), dk, _log(rng, 16, 2000000), _draw_rope(rng, dk), mix=c["mix"], dtype=c["dtype"],
                             inverse=rng.random() < 0.3))
        else:
            hi = _log(rng, 1, 16384)
            q_hi = 1 if rng.random() < 0.4 else min(hi, _log(rng, 1, 4096))
            lo = max(1, int(hi * rng.uniform(0.2, 1.0)))
            kv_heads = rng.choice([1, 2, 3, 4, 8, 8, 16])
            dk = rng.choice([32, 64, 96, 128, 128, 128])
            c.update(reqs=_log(rng, 1, 128), q_lo=min(lo, 1 if q_hi == 1 else max(1, int(q_hi * rng.uniform(0.2, 1.0)))), q_hi=q_hi, kv_lo=lo, kv_hi=hi,
                     kv_heads=kv_heads, heads=kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8, 16]), dk=dk, dv=dk,
                     block=rng.choice([8, 16, 16, 24, 32, 64, 128]), layout=rng.choice(["separate", "blocks_first", "kv_first"]))
            if op == "attention4":
                c.update(causal=rng.random() < 0.8, window=0)
                if c["causal"] and rng.random() < 0.3:
                    c["window"] = _log(rng, 1, 4096)
            else:
                c.update(_draw_rope(rng, dk), shift=rng.choice([0, 0, 1000, 1000000]))
                if op == "write" and rng.random() < 0.25:
                    c.update(heads=0, kv_heads=1, dk=576, dv=0, layout="latent")
                    c.update(_rope(64, offset=512, interleaved=rng.random() < 0.5))
        if _cost(c) <= 1.0:
            return c


def _cost(c):
    """Of the largest listed cases: the plain form's score matrix and gathered rows; the values written."""
    if c["op"] == "rotate":
        return c["tokens"] * c["heads"] * c["dk"] / (8000 * 20 * 192)
    pool = c["reqs"] * c["kv_hi"] * c["kv_heads"] * (c["dk"] + c["dv"])
    if c["op"] == "attention4":
        return max(c["reqs"] * c["heads"] * c["q_hi"] * c["kv_hi"] / (4 * 32 * 4096 * 8192), pool / (64 * 12288 * 2048))
    return max(c["reqs"] * c["q_hi"] * (c["heads"] * c["dk"] + c["kv_heads"] * (c["dk"] + c["dv"])) / (8 * 2000 * 48 * 128), pool / (64 * 12288 * 2048))


def _lengths(c):
    """(new tokens, cached tokens with them) of every request, which go by the case alone."""
    r = random.Random(c["mix"] * 1000003 + c["reqs"])
    kv = [r.randint(c["kv_lo"], c["kv_hi"]) for _ in range(c["reqs"])]
    return [min(k, r.randint(c["q_lo"], c["q_hi"])) for k in kv], kv


def _visible(c):
    """Pairs of a query and a key that it sees, over all requests, and keys that some query sees."""
    pairs = keys = 0
    for q, k in zip(*_lengths(c)):
        first = k - q
        if not c["causal"]:
            pairs, keys = pairs + q * k, keys + k
        elif not c["window"]:
            pairs, keys = pairs + q * first + q * (q + 1) // 2, keys + k
        else:
            n = max(0, min(q, c["window"] - 1 - first))  # queries that see every key before them
            pairs += n * first + n * (n + 1) // 2 + (q - n) * c["window"]
            keys += min(k, q + c["window"] - 1)
    return pairs, keys


def work(c):
    if c["op"] == "rotate":
        return {"bytes": 4 * c["tokens"] * (c["heads"] * c["dk"] + 1), "flops": 3 * c["tokens"] * c["heads"] * c["rot"]}
    q, kv = _lengths(c)
    t, h, g = sum(q), c["heads"], c["kv_heads"]
    if c["op"] == "attention4":
        pairs, keys = _visible(c)
        return {"bytes": 2 * t * h * (c["dk"] + c["dv"]) + keys * g * (c["dk"] + c["dv"]) * 9 // 16 + 4 * t * h,
                "flops": 2 * pairs * h * (c["dk"] + c["dv"])}
    rows = t * g * (c["dk"] + c["dv"])
    once = 4 * t * h * c["dk"] + 2 * rows + 8 * t  # queries in and out, keys and values in, places
    if c["op"] == "write":
        return {"bytes": once + 2 * rows, "flops": 3 * t * (h + g) * c["rot"]}
    # into 4 bits: the rows as they are held, and the values that they stand for
    return {"bytes": once + rows * 9 // 16 + 2 * rows, "flops": 3 * t * (h + g) * c["rot"] + 4 * rows}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
def _frequencies(c, length=8192):
    """(angles a position, in radians, of every pair; what cosines and sines are multiplied by), in 64 bits."""
    d, f, kind = c["rot"], c["factor"], c["scaling"]
    base = c["base"] * (f ** (d / (d - 2)) if kind == "base" else 1.0)
    i = torch.arange(d // 2, dtype=torch.float64)
    w = base ** (-2.0 * i / d)
    if kind == "linear":
        w = w / f
    elif kind == "bands":  # long waves by the factor, short ones as they are
        turns = length * w / (2 * math.pi)
        mix = ((turns - 1.0) / (4.0 - 1.0)).clamp(0.0, 1.0)
        w = w * (mix + (1 - mix) / f)
    elif kind == "yarn":
        at = [d * math.log(length / (n * 2 * math.pi)) / (2 * math.log(base)) for n in (32.0, 1.0)]
        low, high = max(math.floor(at[0]), 0), min(math.ceil(at[1]), d - 1)
        mix = ((i - low) / max(high - low, 1e-3)).clamp(0.0, 1.0)
        w = w * (1 - mix) + w / f * mix
    return w, (0.1 * math.log(f) + 1.0 if kind == "yarn" else 1.0)


def _turns(c):
    """The frequencies as 64-bit fractions of a turn (2^64 is one), and the magnitude."""
    w, magnitude = _frequencies(c)
    t = [int(round(x / (2 * math.pi) * 2.0 ** 64)) for x in w.tolist()]
    return torch.tensor([x - (1 << 64) if x >= 1 << 63 else x for x in t], dtype=torch.int64, device="cuda"), magnitude


def _tables(c, gen, block, spare=1.125):
    """A block table with the pages of all requests scattered over the pool, and the pool's size."""
    need = [-(-k // block) for k in _lengths(c)[1]]
    num = int(sum(need) * spare) + 1
    ids = torch.randperm(num, generator=gen, device="cuda").to(torch.int32)
    col = torch.arange(max(need), device="cuda")
    count = torch.tensor(need, device="cuda")
    at = (count.cumsum(0) - count)[:, None] + col
    return torch.where(col < count[:, None], ids[at.clamp(max=num - 1)], -1).to(torch.int32).contiguous(), num


def _randn(gen, dtype, *shape):
    return torch.randn(shape, generator=gen, device="cuda", dtype=dtype)


def _row_bytes(heads, dim):
    return -(-heads * dim * 9 // 256) * 16


def _pages(layout, num, block, *row, make):
    """Tensors of a paged cache: [keys, values], or one of both."""
    if layout in ("separate", "latent"):
        return [make(num, block, *r) for r in row]
    return [make(*((num, 2, block) if layout == "blocks_first" else (2, num, block)), *row[0])]


def _packed(gen, num, block, heads, dim):
    """Random rows of a 4-bit cache, [num, block, row bytes]: any codes, and scales that give values of about one."""
    n = heads * dim
    rows = torch.zeros(num, block, _row_bytes(heads, dim), dtype=torch.uint8, device="cuda")
    z = torch.randint(0, 256, (num, block, n // 2), generator=gen, device="cuda", dtype=torch.uint8)
    rows[..., :n // 2] = z
    scale = torch.rand((num, block, n // 16), generator=gen, device="cuda") * 0.35 + 0.15
    rows[..., n // 2:n // 2 + n // 16] = scale.to(torch.float8_e4m3fn).view(torch.uint8)
    return rows


def prepare(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype = _DTYPES[c["dtype"]]
    s = {"case": c}
    if c["op"] == "rotate":
        s["x"] = _randn(gen, dtype, c["tokens"], c["heads"], c["dk"])
        s["pos"] = torch.randint(0, c["max_pos"], (c["tokens"],), generator=gen, device="cuda", dtype=torch.int32)
        s["turns"], s["magnitude"] = _turns(c)
        if own:
            _plan(s)
        return s
    q, kv = _lengths(c)
    lens, new = torch.tensor(kv, device="cuda"), torch.tensor(q, device="cuda")
    s["kv_lens"] = lens.to(torch.int32)
    s["q_offsets"] = torch.tensor([sum(q[:i]) for i in range(len(q) + 1)], dtype=torch.int32, device="cuda")
    s["table"], num = _tables(c, gen, c["block"])
    if c["op"] == "attention4":
        s["q"] = _randn(gen, dtype, sum(q), c["heads"], c["dk"])
        s["scale"], s["k_scale"], s["v_scale"] = c["dk"] ** -0.5, 1.0, 0.75
        if c["layout"] == "separate":
            s["cache"] = [_packed(gen, num, c["block"], c["kv_heads"], d) for d in (c["dk"], c["dv"])]
        else:
            both = [_packed(gen, num, c["block"], c["kv_heads"], d) for d in (c["dk"], c["dv"])]
            s["cache"] = [torch.stack(both, 1 if c["layout"] == "blocks_first" else 0)]
    else:
        # keys and values of one projection's output, one after another in a token's row
        t, h, g, dk, dv = sum(q), c["heads"], c["kv_heads"], c["dk"], c["dv"]
        row = _randn(gen, dtype, t, h * dk + g * (dk + dv))
        s["q"] = row[:, :h * dk].unflatten(1, (h, dk)) if h else None
        s["k"] = row[:, h * dk:(h + g) * dk].unflatten(1, (g, dk))
        s["v"] = row[:, (h + g) * dk:].unflatten(1, (g, dv)) if dv else None
        s["req"] = torch.repeat_interleave(torch.arange(len(q), device="cuda"), new).to(torch.int32)
        i = torch.arange(t, device="cuda") - s["q_offsets"][:-1].repeat_interleave(new)
        s["pos"] = ((lens - new).repeat_interleave(new) + i).to(torch.int32)
        s["rope_pos"] = s["pos"] + c["shift"]
        s["turns"], s["magnitude"] = _turns(c)
        if c["op"] == "write":
            shapes = [(g, dk)] + ([(g, dv)] if dv else [])
            s["cache"] = _pages(c["layout"], num, c["block"], *shapes, make=lambda *a: torch.zeros(a, dtype=dtype, device="cuda"))
        else:
            s["k_scale"], s["v_scale"] = 1.0, 0.25
            shapes = [(_row_bytes(g, dk),), (_row_bytes(g, dv),)]
            s["cache"] = _pages(c["layout"], num, c["block"], *shapes, make=lambda *a: torch.zeros(a, dtype=torch.uint8, device="cuda"))
    if own:
        _plan(s)
    return s


def _plan(s):
    """What a program of the library keeps between calls: the cache's description, the rotation's, a workspace."""
    from paged_kv_cache_81_gb300 import pagedkv as K

    c = s["case"]
    if "turns" in s:
        s["rope"] = K.Rope(s["turns"], offset=c["offset"], interleaved=c["interleaved"], magnitude=s["magnitude"])
    if "cache" in s:
        kind = {"latent": "mla"}.get(c["layout"], c["layout"])
        s["paged"] = K.PagedCache.from_tensors([s["cache"][0]], kind)
        s["paged_v"] = K.PagedCache.from_tensors([s["cache"][1]], kind) if len(s["cache"]) > 1 else None
    if c["op"] == "attention4":
        s["workspace"] = K.kv_attention_workspace()


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s)
    if op == "rotate":
        return {"out": _turned(s, s["x"], s["pos"], inverse=s["case"]["inverse"])}
    if op == "write":
        return _append(s)
    if op == "write4":
        return _append4(s)
    return _attend4(s)


def _own(s):
    from paged_kv_cache_81_gb300 import pagedkv as K

    c, op = s["case"], s["case"]["op"]
    if op == "rotate":
        return {"out": K.kv_rotate(s["x"], s["pos"], s["rope"], inverse=c["inverse"])}
    if op == "attention4":
        out, lse = K.kv_attention_q4(s["q"], s["paged"], s["table"], s["q_offsets"], s["kv_lens"], s["scale"], kv_heads=c["kv_heads"],
                                     v_cache=s["paged_v"], k_scale=s["k_scale"], v_scale=s["v_scale"], causal=c["causal"], window=c["window"],
                                     workspace=s["workspace"])
        return {"out": out, "lse": lse}
    rope_pos = s["rope_pos"] if c["shift"] else None
    if op == "write":
        q = K.kv_rotate_write(s["q"], s["k"], s["v"], s["paged"], s["table"], s["req"], s["pos"], s["rope"], v_cache=s["paged_v"], rope_pos=rope_pos)
        return {"q": q, "cache": s["cache"]}
    q, k, v = K.kv_rotate_write_q4(s["q"], s["k"], s["v"], s["paged"], s["table"], s["req"], s["pos"], s["rope"], v_cache=s["paged_v"],
                                   rope_pos=rope_pos, k_scale=s["k_scale"], v_scale=s["v_scale"], held=True)
    return {"q": q, "k": k, "v": v}


def _turned(s, x, pos, inverse=False, wide=False):
    """Rows [tokens, heads, dim] rotated; `wide`: products in 64 bits, for values that are rounded to 4 bits afterwards."""
    c = s["case"]
    half, at = c["rot"] // 2, c["offset"]
    angle = (pos.long()[:, None] * s["turns"]).double() * (2 * math.pi / 2.0 ** 64)  # whole turns drop out of the product
    kind = torch.float64 if wide else torch.float32
    cos, sin = ((f(angle) * s["magnitude"]).to(kind)[:, None] for f in (torch.cos, torch.sin))
    if inverse:
        sin = -sin
    part = x[..., at:at + c["rot"]].to(kind)
    a, b = (part[..., 0::2], part[..., 1::2]) if c["interleaved"] else (part[..., :half], part[..., half:])
    new = (a * cos - b * sin, a * sin + b * cos)
    out = x.clone(memory_format=torch.contiguous_format)
    out[..., at:at + c["rot"]] = (torch.stack(new, -1).flatten(-2) if c["interleaved"] else torch.cat(new, -1)).float().to(x.dtype)
    return out


def _places(s):
    """(pages, slots) of the new tokens."""
    block = s["case"]["block"]
    return s["table"][s["req"].long(), s["pos"].long() // block].long(), s["pos"].long() % block


def _planes(s):
    """The caches of keys and of values, as [pages, block, ...row]; None where there are no values."""
    cache, layout = s["cache"], s["case"]["layout"]
    if layout in ("separate", "latent"):
        return cache[0], cache[1] if len(cache) > 1 else None
    return (cache[0][:, 0], cache[0][:, 1]) if layout == "blocks_first" else (cache[0][0], cache[0][1])


def _append(s):
    page, slot = _places(s)
    keys, values = _planes(s)
    keys[page, slot] = _turned(s, s["k"], s["rope_pos"])
    if values is not None:
        values[page, slot] = s["v"]
    return {"q": None if s["q"] is None else _turned(s, s["q"], s["rope_pos"]), "cache": s["cache"]}


def _quantised(x, scale):
    """(codes, scales) of rows [tokens, heads, dim]: every group of 16 with the scale that takes its largest to 6."""
    y = (x.float() * torch.tensor(1.0 / scale, dtype=torch.float32, device=x.device)).unflatten(-1, (-1, 16))
    most = y.abs().amax(-1)
    unit = (most / 6.0).clamp(max=448.0).to(torch.float8_e4m3fn).float().clamp(min=2.0 ** -9)
    z, size = unit[..., None], y.abs()
    # borders halfway between neighbours, exact in 32 bits; on a border the even code
    code = (size > 0.25 * z).to(torch.uint8)
    for border, above in ((0.75, False), (1.25, True), (1.75, False), (2.5, True), (3.5, False), (5.0, True)):
        code += (size > border * z) if above else (size >= border * z)
    return (code + 8 * torch.signbit(y).to(torch.uint8)).flatten(-2), unit


def _values(code, unit, scale, dtype):
    """What codes [..., dim] and scales [..., dim / 16] stand for."""
    grid = torch.tensor(_GRID + tuple(-x for x in _GRID), device=code.device)
    v = grid[code.int()].unflatten(-1, (-1, 16)) * unit[..., None]
    return (v.flatten(-2) * torch.tensor(scale, dtype=torch.float32, device=code.device)).to(dtype)


def _append4(s):
    page, slot = _places(s)
    held = []
    for rows, plane, scale in ((_turned(s, s["k"], s["rope_pos"], wide=True), _planes(s)[0], s["k_scale"]), (s["v"], _planes(s)[1], s["v_scale"])):
        code, unit = _quantised(rows, scale)
        held.append(_values(code, unit, scale, rows.dtype))
        packed = (code[..., 0::2] | code[..., 1::2] << 4).flatten(1)
        n = packed.shape[1]
        plane[page, slot, :n] = packed
        plane[page, slot, n:n + n // 8] = unit.to(torch.float8_e4m3fn).view(torch.uint8).flatten(1)
    return {"q": None if s["q"] is None else _turned(s, s["q"], s["rope_pos"]), "k": held[0], "v": held[1]}


def _rows4(s, plane, dim, scale, n):
    """The rows [requests, n, heads, dim] of a 4-bit cache in 32 bits, zero past every request's length."""
    c, h = s["case"], s["case"]["kv_heads"]
    at = torch.arange(n, device=plane.device)
    page = s["table"].long().clamp(min=0)[:, at // c["block"]]
    raw = plane[page, at % c["block"]]
    codes = raw[..., :h * dim // 2]
    code = torch.stack([codes & 15, codes >> 4], -1).flatten(-2).unflatten(-1, (h, dim))
    unit = raw[..., h * dim // 2:h * dim // 2 + h * dim // 16].view(torch.float8_e4m3fn).float().unflatten(-1, (h, dim // 16))
    del raw, codes
    return _values(code, unit, scale, torch.float32) * (at < s["kv_lens"][:, None])[..., None, None]


def _attend4(s):
    c, start, lens = s["case"], s["q_offsets"][:-1], s["kv_lens"]
    n = max(_lengths(c)[1])
    count = s["q_offsets"][1:] - start
    i = torch.arange(max(_lengths(c)[0]), device=lens.device)
    at = (start[:, None] + i).clamp(max=s["q"].shape[0] - 1).long()
    j = torch.arange(n, device=lens.device)
    pos = (lens - count)[:, None] + i
    sees = (j < lens[:, None, None]).expand(-1, i.numel(), -1)
    if c["causal"]:
        sees = sees & (j <= pos[:, :, None])
    if c["window"]:
        sees = sees & (j > pos[:, :, None] - c["window"])
    live = i < count[:, None]
    sees = sees & live[:, :, None]
    q = s["q"][at].float()
    r, m, h, d = q.shape
    g = c["kv_heads"]
    q = q.reshape(r, m, g, h // g, d).permute(0, 2, 1, 3, 4).reshape(r, g, -1, d)
    x = torch.matmul(q, _rows4(s, _planes(s)[0], c["dk"], s["k_scale"], n).permute(0, 2, 3, 1)).mul_(s["scale"])
    x = x.view(r, g, m, h // g, -1).masked_fill_(~sees[:, None, :, None, :], -math.inf)
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)
    x = x.sub_(top).exp_()
    total = x.sum(-1)
    lse = (total.log() + top[..., 0]).permute(0, 2, 1, 3).reshape(r, m, -1)[live]
    values = _rows4(s, _planes(s)[1], c["dv"], s["v_scale"], n)
    out = torch.matmul(x.view(r, g, m * (h // g), -1), values.permute(0, 2, 1, 3)).view(r, g, m, h // g, -1)
    out = torch.where(total[..., None] > 0, out / total[..., None], 0.0)
    return {"out": out.permute(0, 2, 1, 3, 4).reshape(r, m, h, -1)[live].to(s["q"].dtype), "lse": lse}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def _pairs(c):
    """(first, second) element of every rotated pair of a head."""
    half = c["rot"] // 2
    return [(c["offset"] + (2 * i if c["interleaved"] else i), c["offset"] + (2 * i + 1 if c["interleaved"] else i + half)) for i in range(half)]


def _exact_turned(c, s, x, pos, inverse=False):
    w, magnitude = _frequencies(c)
    x = x.double()
    out = x.clone()
    for i, (a, b) in enumerate(_pairs(c)):
        t = pos.double() * float(w[i])
        co, si = magnitude * torch.cos(t)[:, None], magnitude * torch.sin(t)[:, None] * (-1 if inverse else 1)
        out[..., a], out[..., b] = x[..., a] * co - x[..., b] * si, x[..., a] * si + x[..., b] * co
    return out


def _exact_held(x, scale):
    """Rows of values rounded to 4 bits, from the nearest of the sixteen that the group's scale gives."""
    y = x.double().unflatten(-1, (-1, 16)) * float(torch.tensor(1.0 / scale, dtype=torch.float32))
    unit = (y.abs().amax(-1, keepdim=True) / 6).clamp(max=448.0).float().to(torch.float8_e4m3fn).double().clamp(min=2.0 ** -9)
    grid = torch.tensor(_GRID, dtype=torch.float64, device=x.device)
    even = torch.tensor([0, 2, 4, 6, 1, 3, 5, 7], device=x.device)  # the even codes first: they win a draw
    z = y.abs() / unit
    near = (z[..., None] - grid[even]).abs().argmin(-1)
    return (torch.copysign(grid[even][near], y) * unit * scale).flatten(-2)


def exact(c, seed):
    """Pair by pair and request by request, head group by head group, from the definitions."""
    if work(c)["flops"] > 2e12:
        return None
    global own
    kept, own = own, False
    try:
        s = prepare(c, seed)
    finally:
        own = kept
    if c["op"] == "rotate":
        return {"out": _exact_turned(c, s, s["x"], s["pos"], c["inverse"])}
    if c["op"] in ("write", "write4"):
        q = None if s["q"] is None else _exact_turned(c, s, s["q"], s["rope_pos"])
        k = _exact_turned(c, s, s["k"], s["rope_pos"])
        if c["op"] == "write4":
            return {"q": q, "k": _exact_held(k.float().to(s["k"].dtype), s["k_scale"]), "v": _exact_held(s["v"], s["v_scale"])}
        cache = [x.double() for x in s["cache"]]
        keys, values = _planes({**s, "cache": cache})
        place = s["table"].long()[s["req"].long(), s["pos"].long() // c["block"]] * c["block"] + s["pos"].long() % c["block"]
        keys[place // c["block"], place % c["block"]] = k
        if values is not None:
            values[place // c["block"], place % c["block"]] = s["v"].double()
        return {"q": q, "cache": cache}
    q_lens, kv_lens = _lengths(c)
    group = c["heads"] // c["kv_heads"]
    grid = torch.tensor(_GRID + tuple(-x for x in _GRID), dtype=torch.float64, device="cuda")
    outs, lses, first = [], [], 0
    for r, (m, n) in enumerate(zip(q_lens, kv_lens)):
        slots = torch.arange(n, device="cuda")
        pages = s["table"][r].long()[slots // c["block"]]
        pos = n - m + torch.arange(m, device="cuda")[:, None]
        hidden = torch.zeros(m, n, dtype=torch.bool, device="cuda")
        if c["causal"]:
            hidden |= slots[None] > pos
        if c["window"]:
            hidden |= slots[None] <= pos - c["window"]
        out_r, lse_r = [], []
        for h in range(c["kv_heads"]):
            kv = []
            for plane, dim, scale in zip(_planes(s), (c["dk"], c["dv"]), (s["k_scale"], s["v_scale"])):
                raw = plane[pages, slots % c["block"]]
                code = raw[:, h * dim // 2:(h + 1) * dim // 2].long()
                unit = c["kv_heads"] * dim // 2 + h * dim // 16
                unit = raw[:, unit:unit + dim // 16].contiguous().view(torch.float8_e4m3fn).double().repeat_interleave(16, 1)
                value = torch.empty(n, dim, dtype=torch.float64, device="cuda")
                value[:, 0::2], value[:, 1::2] = grid[code % 16], grid[code // 16]
                kv.append(value * unit * scale)
            for i in range(h * group, h * group + group):
                x = (s["q"][first:first + m, i].double() @ kv[0].t()) * s["scale"]
                x[hidden] = -math.inf
                lse = torch.logsumexp(x, 1)
                out_r.append(torch.where(hidden, 0.0, torch.exp(x - lse[:, None])) @ kv[1])
                lse_r.append(lse)
        outs.append(torch.stack(out_r, 1))
        lses.append(torch.stack(lse_r, 1))
        first += m
    return {"out": torch.cat(outs), "lse": torch.cat(lses)}
