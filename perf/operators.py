"""The attention operators over the paged cache: their cases, their plain forms and the calls that a user makes.

Five operators that work on the cache which this library writes and moves:

* attention    new tokens (one, or a chunk) of every request against the request's paged keys and values
* latent       the same against one shared latent row a token (576 values: 512 of the latent, 64 of the rotary key)
* expand       the latent rows of every request multiplied out to per-head keys and values of another paged cache
* mass         the attention weight that every cached token receives from the new tokens, summed over heads and queries
* evict        the tokens of highest weight (and the first and last ones) kept, their rows gathered to other blocks

``run`` computes a case either with elementary torch operations (``own`` false) or with the library's
entry points (``own`` true) on what ``prepare`` made.
"""
import math
import random

import torch

own = False

_DTYPES = {"bf16": torch.bfloat16, "fp16": torch.float16}
_RANK, _ROPE = 512, 64  # the latent cache's row: 512 latent values, 64 rotary ones


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------
def _case(op, reqs, q, kv, heads, **kw):
    c = dict(op=op, reqs=reqs, q_lo=q[0], q_hi=q[1], kv_lo=kv[0], kv_hi=kv[1], heads=heads, mix=1, dtype="bf16")
    c.update(kw)
    return c


def listed():
    return [
        # a few requests verifying up to four drafted tokens each under a sliding window: the smallest calls,
        # where latency counts; odd page size and an odd number of query heads to a key head
        dict(_case("attention", 5, (1, 4), (100, 700), 14, kv_heads=2, dk=64, dv=64, block=24, layout="kv_first",
                   causal=True, window=256, dtype="fp16"), name="attn_verify_small"),
        # a decode batch of the 32-layer preset (8 key heads of 128, pages of 16) with long contexts
        dict(_case("attention", 64, (1, 1), (4096, 12288), 32, kv_heads=8, dk=128, dv=128, block=16,
                   layout="separate", causal=True, window=0), name="attn_decode_long"),
        # a prefill chunk against keys and values expanded from latents (192-wide keys, 128-wide values)
        dict(_case("attention", 3, (500, 2000), (1000, 6000), 16, kv_heads=16, dk=192, dv=128, block=64,
                   layout="separate", causal=True, window=0), name="attn_chunk_expanded"),
        # large prefill chunks over earlier context, pages of the 48-layer preset's layout
        dict(_case("attention", 4, (2048, 4096), (4096, 8192), 32, kv_heads=8, dk=128, dv=128, block=16,
                   layout="blocks_first", causal=True, window=0), name="attn_chunk_large"),
        # a small latent decode step, 16 heads (a tensor-parallel share)
        dict(_case("latent", 8, (1, 1), (200, 2000), 16, block=64, causal=True), name="latent_decode_small"),
        # a latent decode batch with every head on this GPU
        dict(_case("latent", 64, (1, 1), (4096, 12288), 128, block=64, causal=True), name="latent_decode_large"),
        # a short prompt's latents expanded
        dict(_case("expand", 3, (0, 0), (40, 500), 16, block=64, out_block=64), name="expand_small"),
        # several long prompts' latents expanded for their prefill chunks
        dict(_case("expand", 4, (0, 0), (4096, 8192), 32, block=64, out_block=64), name="expand_large"),
        # the weights that one decode step gives to the cache
        dict(_case("mass", 16, (1, 1), (2000, 6000), 32, kv_heads=8, dk=128, block=16, layout="separate",
                   causal=True, window=0), name="mass_decode"),
        # the weights that a prefill chunk gives to the cache
        dict(_case("mass", 4, (512, 1024), (4000, 8000), 32, kv_heads=8, dk=128, block=16, layout="blocks_first",
                   causal=True, window=0, dtype="fp16"), name="mass_chunk"),
        # a few short requests trimmed to 256 tokens in a page-shaped layer pair
        dict(_case("evict", 4, (0, 0), (300, 900), 1, dk=128, block=16, layout="blocks_first", tensors=2, budget=256,
                   sinks=4, recent=64), name="evict_small"),
        # sixteen long requests trimmed to 2048 tokens in 16 layers of separate keys and values
        dict(_case("evict", 16, (0, 0), (4000, 16000), 8, dk=128, block=16, layout="separate", tensors=32,
                   budget=2048, sinks=4, recent=512), name="evict_large"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["attention", "attention", "attention", "latent", "latent", "expand", "mass", "mass", "evict"])
    c = dict(op=op, mix=rng.randrange(1 << 30), dtype=rng.choice(["bf16", "fp16"]))
    while True:
        reqs = _log(rng, 1, 128)
        hi = _log(rng, 1, 16384)
        lo = max(1, int(hi * rng.uniform(0.2, 1.0)))
        q_hi = 1 if rng.random() < 0.4 else min(hi, _log(rng, 1, 4096))
        q_lo = 1 if q_hi == 1 else max(1, int(q_hi * rng.uniform(0.2, 1.0)))
        c.update(reqs=reqs, q_lo=min(q_lo, lo), q_hi=q_hi, kv_lo=lo, kv_hi=hi)
        if op in ("attention", "mass"):
            kv_heads = rng.choice([1, 2, 4, 8])
            c.update(kv_heads=kv_heads, heads=kv_heads * rng.choice([1, 2, 3, 4, 5, 7, 8, 16]),
                     block=rng.choice([8, 16, 16, 24, 32, 64, 128]), layout=rng.choice(["separate", "blocks_first", "kv_first"]),
                     causal=rng.random() < 0.8, window=0)
            if c["causal"] and rng.random() < 0.3:
                c["window"] = _log(rng, 1, 4096)
            c.update(dk=rng.choice([64, 128, 128]))
            if op == "attention":
                c["dv"] = c["dk"]
                if rng.random() < 0.25:
                    heads = rng.choice([8, 16, 32])
                    c.update(dk=192, dv=128, heads=heads, kv_heads=heads, layout="separate")
        elif op == "latent":
            c.update(heads=rng.choice([8, 16, 20, 32, 64, 128]), block=rng.choice([16, 32, 64]), causal=rng.random() < 0.8)
            if c["q_hi"] > 1:
                c.update(q_hi=min(c["q_hi"], 256))
                c.update(q_lo=min(c["q_lo"], c["q_hi"]))
        elif op == "expand":
            c.update(q_lo=0, q_hi=0, heads=rng.choice([4, 8, 16, 32]), block=rng.choice([16, 64]), out_block=rng.choice([16, 64, 128]))
        else:
            budget = _log(rng, 1, 4096)
            sinks = rng.randrange(0, min(8, budget) + 1)
            c.update(q_lo=0, q_hi=0, heads=rng.choice([1, 2, 4, 8]), dk=rng.choice([64, 128]), block=rng.choice([8, 16, 24, 64]),
                     layout=rng.choice(["separate", "blocks_first", "kv_first"]), tensors=2 * rng.randrange(1, 13), budget=budget,
                     sinks=sinks, recent=rng.randrange(0, budget - sinks + 1))
        if _cost(c) <= 1.0:
            return c


#: What the largest listed cases hold in the plain forms: values of the score matrix, of the gathered rows.
_MOST_SCORES, _MOST_ROWS = 4 * 32 * 4096 * 8192, 64 * 12288 * 2048


def _cost(c):
    rows = {"attention": c.get("kv_heads", 0) * (c.get("dk", 0) + c.get("dv", 0)), "latent": _RANK + _ROPE, "expand": 320 * c["heads"],
            "mass": c.get("kv_heads", 0) * c.get("dk", 0), "evict": c["heads"] * c.get("dk", 0) * 2 * c.get("tensors", 0)}[c["op"]]
    scores = c["reqs"] * c["heads"] * c["q_hi"] * c["kv_hi"] * (6 if c["op"] == "latent" else 2 if c["op"] == "mass" else 1)
    most = {"attention": _MOST_ROWS, "latent": _MOST_ROWS // 2, "expand": 4 * 8192 * 320 * 32, "mass": 16 * 6000 * 1024,
            "evict": 16 * 16000 * 1024 * 32}[c["op"]]
    return max(scores / _MOST_SCORES, c["reqs"] * c["kv_hi"] * rows / most)


def _lengths(c):
    """(query tokens, cached tokens) of every request, which go by the case alone."""
    r = random.Random(c["mix"] * 1000003 + c["reqs"])
    kv = [r.randint(c["kv_lo"], c["kv_hi"]) for _ in range(c["reqs"])]
    return [min(k, r.randint(c["q_lo"], c["q_hi"])) for k in kv], kv


def _visible(c):
    """Pairs of a query and a key that it sees, over all requests, and keys that some query sees."""
    pairs = keys = 0
    window = c.get("window", 0)
    for q, k in zip(*_lengths(c)):
        first = k - q
        if not c["causal"]:
            pairs, keys = pairs + q * k, keys + k
        elif not window:
            pairs, keys = pairs + q * first + q * (q + 1) // 2, keys + k
        else:
            n = max(0, min(q, window - 1 - first))  # queries that see every key before them
            pairs += n * first + n * (n + 1) // 2 + (q - n) * window
            keys += min(k, q + window - 1)
    return pairs, keys


def work(c):
    q, kv = _lengths(c)
    t, n, h = sum(q), sum(kv), c["heads"]
    if c["op"] == "attention":
        pairs, keys = _visible(c)
        return {"bytes": 2 * (t * h * (c["dk"] + c["dv"]) + keys * c["kv_heads"] * (c["dk"] + c["dv"])) + 4 * t * h,
                "flops": 2 * pairs * h * (c["dk"] + c["dv"])}
    if c["op"] == "latent":
        pairs, keys = _visible(c)
        return {"bytes": 2 * (t * h * (2 * _RANK + _ROPE) + keys * (_RANK + _ROPE)) + 4 * t * h,
                "flops": 2 * pairs * h * (2 * _RANK + _ROPE)}
    if c["op"] == "expand":
        return {"bytes": 2 * (n * (_RANK + _ROPE) + h * 256 * _RANK + n * h * 320), "flops": 2 * n * h * 256 * _RANK}
    if c["op"] == "mass":
        pairs, keys = _visible(c)
        return {"bytes": 2 * (t * h * c["dk"] + keys * c["kv_heads"] * c["dk"]) + 4 * t * h + 8 * n, "flops": 2 * pairs * h * c["dk"]}
    kept = sum(min(k, c["budget"]) for k in kv)
    row = 2 * c["heads"] * c["dk"] * c["tensors"] * (1 if c["layout"] == "separate" else 2)
    return {"bytes": 2 * kept * row + 4 * n + 12 * kept, "flops": 0}


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------
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


def _cache(gen, dtype, layout, num, block, heads, dk, dv=None, tensors=1):
    """Tensors of a paged cache, stacked: [tensors, ...]; for "separate" the keys' and then the values'."""
    if layout == "separate" and dv is not None:
        return [_randn(gen, dtype, num, block, heads, dk), _randn(gen, dtype, num, block, heads, dv)]
    shape = {"separate": (num, block, heads, dk), "blocks_first": (num, 2, block, heads, dk), "kv_first": (2, num, block, heads, dk)}[layout]
    return _randn(gen, dtype, tensors, *shape)


def prepare(c, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    dtype, (q, kv) = _DTYPES[c["dtype"]], _lengths(c)
    s = {"case": c, "kv_lens": torch.tensor(kv, dtype=torch.int32, device="cuda"),
         "q_offsets": torch.tensor([sum(q[:i]) for i in range(len(q) + 1)], dtype=torch.int32, device="cuda")}
    s["table"], num = _tables(c, gen, c["block"])
    if c["op"] in ("attention", "mass"):
        s["q"] = _randn(gen, dtype, sum(q), c["heads"], c["dk"])
        s["scale"] = c["dk"] ** -0.5
        dv = c.get("dv", c["dk"])
        s["cache"] = _cache(gen, dtype, c["layout"], num, c["block"], c["kv_heads"], c["dk"], dv)
        if c["op"] == "mass":
            s["lse"] = _attend(s, weights=False)["lse"]
            s["prev"] = torch.rand((c["reqs"], max(kv) + 3), generator=gen, device="cuda")
    elif c["op"] == "latent":
        s["q"] = _randn(gen, dtype, sum(q), c["heads"], _RANK + _ROPE)
        s["scale"] = 192 ** -0.5 * 0.5
        s["cache"] = _randn(gen, dtype, num, c["block"], _RANK + _ROPE)
    elif c["op"] == "expand":
        s["cache"] = _randn(gen, dtype, num, c["block"], _RANK + _ROPE)
        s["weight"] = _randn(gen, dtype, c["heads"], 256, _RANK) * _RANK ** -0.5
        s["out_table"], num = _tables(c, gen, c["out_block"])
        s["k_out"] = torch.zeros(num, c["out_block"], c["heads"], 192, dtype=dtype, device="cuda")
        s["v_out"] = torch.zeros(num, c["out_block"], c["heads"], 128, dtype=dtype, device="cuda")
    else:
        total = num
        # the kept rows go to pages of their own, which no request holds
        need = -(-c["budget"] // c["block"])
        used = torch.zeros(total + c["reqs"] * need, dtype=torch.bool, device="cuda")
        used[s["table"][s["table"] >= 0].long()] = True
        s["out_table"] = torch.nonzero(~used)[: c["reqs"] * need, 0].to(torch.int32).reshape(c["reqs"], need).contiguous()
        s["cache"] = _cache(gen, dtype, c["layout"], int(used.numel()), c["block"], c["heads"], c["dk"], tensors=c["tensors"])
        # weights as a few heavy tokens and a long tail give them, some of them equal
        score = torch.rand((c["reqs"], max(kv)), generator=gen, device="cuda").pow(8)
        s["score"] = torch.where(score < 1e-3, torch.zeros_like(score), score)
    if own:
        _plan(s)
    return s


def _plan(s):
    """What a program of the library keeps between calls: the cache's description, buffers for outputs and workspaces."""
    from paged_kv_cache_81_gb300 import pagedkv as K

    c = s["case"]
    if c["op"] in ("latent", "expand"):
        s["paged"] = K.PagedCache.from_tensors([s["cache"]], "mla")
    if c["op"] == "expand":
        s["paged_k"] = K.PagedCache.from_tensors([s["k_out"]], "separate")
        s["paged_v"] = K.PagedCache.from_tensors([s["v_out"]], "separate")
    elif c["op"] == "evict":
        s["paged"] = K.PagedCache.from_tensors(list(s["cache"]), c["layout"])
    elif c["op"] in ("attention", "mass"):
        if c["layout"] == "separate":
            s["paged"] = K.PagedCache.from_tensors([s["cache"][0]], "separate")
            s["paged_v"] = K.PagedCache.from_tensors([s["cache"][1]], "separate")
        else:
            s["paged"], s["paged_v"] = K.PagedCache.from_tensors([s["cache"][0]], c["layout"]), None
    if c["op"] in ("attention", "latent"):
        s["workspace"] = K.kv_attention_workspace()


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------
def run(s):
    op = s["case"]["op"]
    if own:
        return _own(s)
    if op == "attention":
        return _attend(s)
    if op == "latent":
        return _attend(s, latent=True)
    if op == "expand":
        return _expand(s)
    if op == "mass":
        return _mass(s)
    return _evict(s)


def _own(s):
    from paged_kv_cache_81_gb300 import pagedkv as K

    c, op = s["case"], s["case"]["op"]
    if op == "attention":
        out, lse = K.kv_attention(s["q"], s["paged"], s["table"], s["q_offsets"], s["kv_lens"], s["scale"], v_cache=s["paged_v"],
                                  causal=c["causal"], window=c["window"], workspace=s["workspace"])
        return {"out": out, "lse": lse}
    if op == "latent":
        out, lse = K.kv_latent_attention(s["q"], s["paged"], s["table"], s["q_offsets"], s["kv_lens"], s["scale"], causal=c["causal"],
                                         workspace=s["workspace"])
        return {"out": out, "lse": lse}
    if op == "expand":
        K.kv_latent_expand(s["paged"], s["table"], s["kv_lens"], s["weight"], s["paged_k"], s["paged_v"], s["out_table"])
        return {"k": s["k_out"], "v": s["v_out"]}
    if op == "mass":
        return {"score": K.kv_attention_mass(s["q"], s["paged"], s["table"], s["q_offsets"], s["kv_lens"], s["lse"], s["scale"],
                                             causal=c["causal"], window=c["window"], prev=s["prev"])}
    lens, kept, score = K.kv_evict(s["paged"], s["table"], s["kv_lens"], s["score"], c["budget"], sinks=c["sinks"], recent=c["recent"],
                                   out_table=s["out_table"])
    return {"lens": lens, "kept": kept, "score": score, "cache": s["cache"]}


def _rows(cache, table, block, lens, n):
    """The rows [requests, n, ...] of a cache [pages, block, ...] in 32 bits, zero past every request's length."""
    at = torch.arange(n, device=table.device)
    page = table.long().clamp(min=0)[:, at // block]
    return cache[page, at % block].float() * (at < lens[:, None]).reshape(*page.shape, *[1] * (cache.dim() - 2))


def _padded(s):
    """Queries [requests, longest, heads, d] in 32 bits, and what a query of every request may see of its keys."""
    c, start, lens = s["case"], s["q_offsets"][:-1], s["kv_lens"]
    count = s["q_offsets"][1:] - start
    i = torch.arange(max(_lengths(c)[0]), device=lens.device)
    at = (start[:, None] + i).clamp(max=s["q"].shape[0] - 1).long()
    j = torch.arange(max(_lengths(c)[1]), device=lens.device)
    pos = (lens - count)[:, None] + i
    sees = (j < lens[:, None, None]).expand(-1, i.numel(), -1)
    if c["causal"]:
        sees = sees & (j <= pos[:, :, None])
    if c.get("window", 0):
        sees = sees & (j > pos[:, :, None] - c["window"])
    return s["q"][at].float(), sees & (i < count[:, None])[:, :, None], i < count[:, None]


def _planes(s):
    """(keys, values) of an attention case's cache, as [pages, block, heads, d]."""
    layout, cache = s["case"]["layout"], s["cache"]
    if layout == "separate":
        return cache[0], cache[1]
    return (cache[0][:, 0], cache[0][:, 1]) if layout == "blocks_first" else (cache[0][0], cache[0][1])


def _scores(s, keys):
    """Scaled products [requests, key heads, queries * group, keys] of a padded batch, -inf where a query may not see."""
    q, sees, live = _padded(s)
    r, m, h, d = q.shape
    groups = keys.shape[2]
    q = q.reshape(r, m, groups, h // groups, d).permute(0, 2, 1, 3, 4).reshape(r, groups, -1, d)
    x = torch.matmul(q, keys.permute(0, 2, 3, 1)).mul_(s["scale"])
    hidden = ~sees[:, None, :, None, :]
    return x.view(r, groups, m, h // groups, -1).masked_fill_(hidden, -math.inf), live


def _attend(s, latent=False, weights=True):
    c = s["case"]
    n = max(_lengths(c)[1])
    if latent:
        keys = _rows(s["cache"], s["table"], c["block"], s["kv_lens"], n)[:, :, None]
        values = keys[..., :_RANK]
    else:
        keys, values = (_rows(x, s["table"], c["block"], s["kv_lens"], n) if x is not None else None
                        for x in (_planes(s)[0], _planes(s)[1] if weights else None))
    x, live = _scores(s, keys)
    del keys
    r, groups, m, g, _ = x.shape
    top = x.amax(-1, keepdim=True).clamp(min=-1e30)
    x = x.sub_(top).exp_()
    total = x.sum(-1)
    lse = (total.log() + top[..., 0]).permute(0, 2, 1, 3).reshape(r, m, -1)[live]
    if not weights:
        return {"lse": lse}
    out = torch.matmul(x.view(r, groups, m * g, -1), values.permute(0, 2, 1, 3)).view(r, groups, m, g, -1)
    out = torch.where(total[..., None] > 0, out / total[..., None], 0.0)
    return {"out": out.permute(0, 2, 1, 3, 4).reshape(r, m, groups * g, -1)[live].to(s["q"].dtype), "lse": lse}


def _mass(s):
    c = s["case"]
    n = max(_lengths(c)[1])
    x, live = _scores(s, _rows(_planes(s)[0], s["table"], c["block"], s["kv_lens"], n))
    lse = torch.zeros((*live.shape, c["heads"]), device=live.device)
    lse[live] = s["lse"]
    r, groups, m, g, _ = x.shape
    lse = lse.view(r, m, groups, g).permute(0, 2, 1, 3)[..., None]
    got = x.sub_(torch.where(torch.isfinite(lse), lse, 0.0)).exp_().sum((1, 2, 3))
    score = s["prev"].clone()
    score[:, :n] += got
    return {"score": score}


def _expand(s):
    c = s["case"]
    n = max(_lengths(c)[1])
    rows = _rows(s["cache"], s["table"], c["block"], s["kv_lens"], n)
    at = torch.arange(n, device=rows.device)
    live = at < s["kv_lens"][:, None]
    page, slot = s["out_table"].long().clamp(min=0)[:, at // c["out_block"]][live], (at % c["out_block"]).expand_as(live)[live]
    rows = rows[live]
    both = torch.matmul(rows[:, :_RANK], s["weight"].float().view(-1, _RANK).t()).view(-1, c["heads"], 256)
    rope = rows[:, None, _RANK:].expand(-1, c["heads"], -1)
    s["k_out"][page, slot] = torch.cat([both[..., :128], rope], -1).to(s["k_out"].dtype)
    s["v_out"][page, slot] = both[..., 128:].to(s["v_out"].dtype)
    return {"k": s["k_out"], "v": s["v_out"]}


def _evict(s):
    c, lens = s["case"], s["kv_lens"].long()
    n, budget = s["score"].shape[1], c["budget"]
    at = torch.arange(n, device=lens.device)
    rank = torch.where((at < c["sinks"]) | (at >= lens[:, None] - c["recent"]), math.inf, s["score"])
    rank = torch.where(at < lens[:, None], rank, -math.inf)
    order = torch.sort(rank, dim=1, descending=True, stable=True).indices[:, :budget]
    held = torch.zeros_like(rank, dtype=torch.bool).scatter_(1, order, True) & (at < lens[:, None])
    new = lens.clamp(max=budget)
    # kept tokens in their order: held ones first, by index
    kept = torch.sort((~held).to(torch.int8), dim=1, stable=True).indices[:, :budget]
    kept = torch.nn.functional.pad(kept, (0, budget - kept.shape[1]))
    i = torch.arange(budget, device=lens.device)
    live = i < new[:, None]
    req = torch.arange(lens.numel(), device=lens.device)[:, None]
    src = (s["table"].long()[req, kept // c["block"]][live], (kept % c["block"])[live])
    dst = (s["out_table"].long()[:, i // c["block"]][live], (i % c["block"]).expand_as(live)[live])
    cache = s["cache"]
    if c["layout"] == "separate":
        cache[:, dst[0], dst[1]] = cache[:, src[0], src[1]]
    elif c["layout"] == "kv_first":
        cache[:, :, dst[0], dst[1]] = cache[:, :, src[0], src[1]]
    else:
        flat = cache.transpose(1, 2)
        flat[:, :, dst[0], dst[1]] = flat[:, :, src[0], src[1]]
    score = torch.where(live, s["score"][req, kept], 0.0)
    return {"lens": new.to(torch.int32), "kept": torch.where(live, kept, -1).to(torch.int32), "score": score, "cache": cache}


# ---------------------------------------------------------------------------
# the definitions in 64 bits
# ---------------------------------------------------------------------------
def exact(c, seed):
    """Request by request, head group by head group, from the definitions."""
    if c["op"] == "evict" or work(c)["flops"] > 2e12:
        return None
    global own
    kept, own = own, False
    try:
        s = prepare(c, seed)
    finally:
        own = kept
    q_lens, kv_lens = _lengths(c)
    if c["op"] == "expand":
        k, v = s["k_out"].double(), s["v_out"].double()
        w = s["weight"].double()
        for r, n in enumerate(kv_lens):
            slots = [(int(b) * c["block"] + o) for b in s["table"][r].tolist() if b >= 0 for o in range(c["block"])][:n]
            outs = [(int(b) * c["out_block"] + o) for b in s["out_table"][r].tolist() if b >= 0 for o in range(c["out_block"])][:n]
            rows = s["cache"].view(-1, _RANK + _ROPE)[torch.tensor(slots, device="cuda")].double()
            outs = torch.tensor(outs, device="cuda")
            for h in range(c["heads"]):
                k.view(-1, c["heads"], 192)[outs, h] = torch.cat([rows[:, :_RANK] @ w[h, :128].t(), rows[:, _RANK:]], 1)
                v.view(-1, c["heads"], 128)[outs, h] = rows[:, :_RANK] @ w[h, 128:].t()
        return {"k": k, "v": v}
    kv_heads = c.get("kv_heads", 1)
    group = c["heads"] // kv_heads
    keys, values = (s["cache"][:, :, None], s["cache"][:, :, None, :_RANK]) if c["op"] == "latent" else _planes(s)
    outs, lses = [], []
    score = s["prev"].double() if c["op"] == "mass" else None
    first = 0
    for r, (m, n) in enumerate(zip(q_lens, kv_lens)):
        slots = torch.arange(n, device="cuda")
        pages = s["table"][r].long()[slots // c["block"]]
        pos = n - m + torch.arange(m, device="cuda")[:, None]
        hidden = torch.zeros(m, n, dtype=torch.bool, device="cuda")
        if c["causal"]:
            hidden |= slots[None] > pos
        if c.get("window", 0):
            hidden |= slots[None] <= pos - c["window"]
        out_r, lse_r = [], []
        for h in range(kv_heads):
            k = keys[pages, slots % c["block"], h].double()
            v = values[pages, slots % c["block"], h].double()
            for i in range(h * group, h * group + group):
                x = (s["q"][first:first + m, i].double() @ k.t()) * s["scale"]
                x[hidden] = -math.inf
                if score is not None:
                    lse = s["lse"][first:first + m, i].double()
                    score[r, :n] += torch.where(hidden, 0.0, torch.exp(x - lse[:, None])).sum(0)
                    continue
                lse = torch.logsumexp(x, 1)
                p = torch.where(hidden, 0.0, torch.exp(x - lse[:, None]))
                out_r.append(p @ v)
                lse_r.append(lse)
        if score is None:
            outs.append(torch.stack(out_r, 1))
            lses.append(torch.stack(lse_r, 1))
        first += m
    return {"score": score} if score is not None else {"out": torch.cat(outs), "lse": torch.cat(lses)}
