"""Attention mass and eviction on the GPU, and a request's life through both."""
from __future__ import annotations

import math
from types import SimpleNamespace

import numpy as np
import pytest
import torch

from paged_kv_cache_81_gb300 import pagedkv as K
from tests.attention_support import Batch, check, close, hidden, reference

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


def mass_reference(b, lse, scale, causal, window, width, prev=None):
    want = torch.zeros(len(b.kv_lens), width, dtype=torch.float64) if prev is None else prev.double().cpu().clone()
    tol = want.abs() * 2.0 ** -23
    first = 0
    for r, (m, n) in enumerate(zip(b.q_lens, b.kv_lens)):
        x = b.q_cpu[first:first + m].double()
        norm = lse[first:first + m].double().cpu()  # [m, h]
        first += m
        k = b.k_rows[r].double().repeat_interleave(b.heads // b.kv_heads, 1)
        s = torch.einsum("mhd,nhd->mhn", x, k) * scale
        size = torch.einsum("mhd,nhd->mhn", x.abs(), k.abs()) * scale
        p = torch.where(hidden(m, n, causal, window)[:, None], 0.0, torch.exp(s - norm[..., None]))
        p = torch.where(torch.isfinite(norm)[..., None], p, 0.0)
        big = float(size.max() + norm[torch.isfinite(norm)].abs().max()) if m and n and torch.isfinite(norm).any() else 0.0
        got = p.sum((0, 1))
        c = min(n, width)
        want[r, :c] += got[:c]
        # products and the exponent in 32 bits, the sum of m * heads terms
        tol[r, :c] += got[:c] * 2.0 ** -23 * (b.dk + 16 + math.sqrt(m * b.heads)) * (1 + big)
    return want, tol + 2.0 ** -40


def mass_check(b, causal=True, window=0, prev=None, width=None, in_place=False):
    scale = b.dk ** -0.5
    _, lse = b.run(scale, causal, window) if b.layout != "keys" else (None, None)
    width = max(b.kv_lens) + 5 if width is None else width
    before = None if prev is None else prev.clone()
    K.kv_get_last_error(clear=True)
    got = K.kv_attention_mass(b.q, b.cache, b.table, b.offsets, b.lens, lse, scale, causal=causal, window=window, prev=prev, width=width,
                              score=prev if in_place else None)
    assert K.kv_get_last_error(clear=True) == 0
    want, tol = mass_reference(b, lse, scale, causal, window, width, before)
    close(got[:, :width], want, tol, "mass")
    return got, lse


@pytest.mark.parametrize("q_lens,kv_lens", [([1], [1]), ([1], [128]), ([1], [129]), ([0, 4, 1], [3, 4, 300]), ([150, 2], [400, 90]), ([40], [40]), ([9], [4])])
@pytest.mark.parametrize("heads,kv_heads,dk,dtype", [(4, 4, 64, BF), (8, 2, 128, FP), (14, 2, 72, BF), (6, 1, 192, BF)])
def test_mass(q_lens, kv_lens, heads, kv_heads, dk, dtype):
    mass_check(Batch(q_lens, kv_lens, heads, kv_heads, dk, 64, dtype=dtype, seed=len(q_lens) + dk))


@pytest.mark.parametrize("causal,window", [(False, 0), (True, 1), (True, 100), (True, 128)])
@pytest.mark.parametrize("block,layout", [(16, "blocks_first"), (24, "kv_first"), (128, "separate"), (1, "separate")])
def test_mass_masks_and_pages(causal, window, block, layout):
    b = Batch([1, 3, 200], [500, 129, 300], 8, 2, 64, block=block, layout=layout, seed=window)
    if window:
        for r in range(3):  # entries before every window may be stale
            b.table[r, : max(0, b.kv_lens[r] - b.q_lens[r] - window + 1) // block] = -1
    mass_check(b, causal, window)


@pytest.mark.parametrize("in_place", [False, True])
def test_mass_adds_to_what_was(in_place):
    b = Batch([2, 1], [200, 700], 8, 2, 128, seed=2)
    prev = torch.rand(2, 720, device="cuda")
    mass_check(b, prev=prev, width=720, in_place=in_place)


def test_mass_narrow_and_strided_scores():
    b = Batch([2, 1], [200, 700], 8, 2, 128, seed=2)
    scale = b.dk ** -0.5
    _, lse = b.run(scale)
    wide = torch.full((2, 900), 3.0, device="cuda")
    got = K.kv_attention_mass(b.q, b.cache, b.table, b.offsets, b.lens, lse, scale, score=wide[:, 7:], width=150)
    want, tol = mass_reference(b, lse, scale, True, 0, 150)
    close(got[:, :150], want, tol, "mass")
    assert torch.all(wide[:, :7] == 3) and torch.all(wide[:, 157:] == 3)


def test_mass_of_every_row_sums_to_the_rows():
    b = Batch([60, 1], [900, 5000], 16, 4, 64, seed=2)
    got, lse = mass_check(b)
    assert abs(float(got[0].double().sum()) - 60 * 16) < 1e-3 and abs(float(got[1].double().sum()) - 16) < 1e-3


def test_mass_repeats_and_replays():
    b = Batch([1, 100], [9000, 900], 8, 2, 64, seed=2)
    scale = b.dk ** -0.5
    _, lse = b.run(scale)
    args = (b.q, b.cache, b.table, b.offsets, b.lens, lse, scale)
    want = K.kv_attention_mass(*args).clone()
    for _ in range(10):
        assert torch.equal(want, K.kv_attention_mass(*args))
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = K.kv_attention_mass(*args)
    got.fill_(7)
    g.replay()
    g.replay()
    torch.cuda.synchronize()
    assert torch.equal(want, got)


# ---------------------------------------------------------------------------
# eviction
# ---------------------------------------------------------------------------
def keep_reference(score, n, budget, sinks, recent):
    """Indices that stay, by sorting (score descending, index ascending); NaN last."""
    if n <= budget:
        return list(range(n))
    sure = set(range(sinks)) | set(range(n - recent, n))
    rest = [j for j in range(n) if j not in sure]
    rest.sort(key=lambda j: (math.isnan(score[j]), -score[j] if not math.isnan(score[j]) else 0.0, j))
    return sorted(sure | set(rest[: budget - len(sure)]))


def evict_case(kv_lens, score, budget, sinks, recent, *, layout="separate", tensors=2, block=16, row=32, in_place=False, seed=0):
    g = torch.Generator().manual_seed(seed)
    n = len(kv_lens)
    need = [-(-x // block) for x in kv_lens]
    extra = -(-budget // block)
    pages = sum(need) + n * extra + 2
    ids = torch.randperm(pages, generator=g).to(torch.int32)
    table = torch.full((n, max(need + [1])), -1, dtype=torch.int32)
    at = 0
    for r in range(n):
        table[r, :need[r]] = ids[at:at + need[r]]
        at += need[r]
    out_table = ids[at:at + n * extra].reshape(n, extra).contiguous()
    shape = {"separate": (pages, block, row), "blocks_first": (pages, 2, block, row), "kv_first": (2, pages, block, row)}[layout]
    host = [torch.randint(-2 ** 15, 2 ** 15, shape, generator=g, dtype=torch.int16) for _ in range(tensors)]
    dev = [t.cuda().view(BF) for t in host]
    cache = K.PagedCache.from_tensors(dev, layout)
    K.kv_get_last_error(clear=True)
    lens, kept, out_score = K.kv_evict(cache, table.cuda(), torch.tensor(kv_lens, dtype=torch.int32, device="cuda"), score.cuda(), budget,
                                       sinks=sinks, recent=recent, out_table=None if in_place else out_table.cuda())
    assert K.kv_get_last_error(clear=True) == 0
    if in_place:
        out_table = table
    want = [t.clone() for t in host]

    def rows(t, page, slot):
        return t[page, slot] if layout == "separate" else t[page, :, slot] if layout == "blocks_first" else t[:, page, slot].transpose(0, 1)

    for r in range(n):
        keep = keep_reference(score[r].tolist(), kv_lens[r], budget, sinks, recent)
        assert int(lens[r]) == len(keep)
        assert kept[r].tolist() == keep + [-1] * (budget - len(keep)), r
        np.testing.assert_array_equal(out_score[r].cpu().numpy(), np.array([score[r, j] for j in keep] + [0.0] * (budget - len(keep)), np.float32))
        j, i = torch.tensor(keep, dtype=torch.long), torch.arange(len(keep))
        src = (table[r].long()[j // block], j % block)
        dst = (out_table[r].long()[i // block], i % block)
        for t, w in zip(host, want):
            x = rows(t, *src)
            if layout == "separate":
                w[dst[0], dst[1]] = x
            elif layout == "blocks_first":
                w[dst[0], :, dst[1]] = x
            else:
                w[:, dst[0], dst[1]] = x.transpose(0, 1)
    for t, w in zip(dev, want):
        assert torch.equal(t.view(torch.int16).cpu(), w)


def scores(n, width, seed, kind="heavy"):
    g = torch.Generator().manual_seed(seed)
    s = torch.rand(n, width, generator=g)
    if kind == "heavy":
        s = torch.where(s < 0.6, torch.zeros_like(s), s ** 4)
    elif kind == "ties":
        s = torch.randint(0, 3, (n, width), generator=g).float()
    elif kind == "equal":
        s = torch.full_like(s, 0.25)
    elif kind == "signed":
        s = torch.randn(n, width, generator=g) * 10.0 ** torch.randint(-30, 30, (n, width), generator=g).float()
        s[:, ::7], s[:, 1::11] = 0.0, -0.0
    elif kind == "wild":
        s = torch.randn(n, width, generator=g)
        s[:, ::5], s[:, 1::13], s[:, 2::17] = float("nan"), float("inf"), float("-inf")
    return s


@pytest.mark.parametrize("kind", ["heavy", "ties", "equal", "signed", "wild"])
@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("layout", ["separate", "blocks_first", "kv_first"])
def test_evict(kind, in_place, layout):
    lens = [300, 0, 1, 64, 65, 1000, 77]
    evict_case(lens, scores(7, 1000, 3, kind), 64, 4, 20, layout=layout, in_place=in_place)


@pytest.mark.parametrize("budget,sinks,recent", [(0, 0, 0), (1, 0, 0), (1, 1, 0), (1, 0, 1), (10, 5, 5), (10, 10, 0), (10, 0, 10), (37, 3, 0), (500, 4, 100)])
@pytest.mark.parametrize("in_place", [False, True])
def test_budgets(budget, sinks, recent, in_place):
    evict_case([200, 10, 501, 37], scores(4, 501, 1), budget, sinks, recent, in_place=in_place, block=24)


@pytest.mark.parametrize("row,block,tensors", [(8, 16, 1), (24, 8, 3), (72, 64, 2), (576, 64, 3), (1024, 16, 2), (4096, 4, 1), (5000, 2, 1)])
@pytest.mark.parametrize("in_place", [False, True])
def test_row_sizes(row, block, tensors, in_place):
    evict_case([700, 333], scores(2, 700, 5), 200, 4, 32, row=row, block=block, tensors=tensors, in_place=in_place)


@pytest.mark.parametrize("in_place", [False, True])
def test_long_lists(in_place):
    evict_case([30000, 9000], scores(2, 30000, 5, "heavy"), 5000, 4, 512, row=8, block=64, tensors=1, in_place=in_place)


def test_scores_in_place():
    s = scores(2, 400, 8).cuda()
    want = s.clone().cpu()
    pages = torch.arange(2 * 25, dtype=torch.int32, device="cuda").view(2, 25)
    cache = K.PagedCache.from_tensors([torch.zeros(50, 16, 8, dtype=BF, device="cuda")], "separate")
    lens = torch.tensor([400, 350], dtype=torch.int32, device="cuda")
    _, kept, out = K.kv_evict(cache, pages, lens, s, 100, sinks=2, recent=9, out_score=s)
    for r, n in enumerate((400, 350)):
        keep = keep_reference(want[r].tolist(), n, 100, 2, 9)
        assert kept[r].tolist() == keep and s[r, :100].tolist() == want[r][keep].tolist()
        assert torch.equal(s[r, 100:].cpu(), want[r, 100:])


def test_bad_pages_and_short_tables():
    cache = K.PagedCache.from_tensors([torch.zeros(20, 16, 8, dtype=BF, device="cuda")], "separate")
    table = torch.arange(10, dtype=torch.int32, device="cuda").view(1, 10)
    table[0, 3] = 77
    s = torch.ones(1, 160, device="cuda")
    lens = torch.tensor([160], dtype=torch.int32, device="cuda")
    K.kv_get_last_error(clear=True)
    K.kv_evict(cache, table, lens, s, 100, recent=50)
    assert K.kv_get_last_error(clear=True) == K.KV_DERR_TABLE
    out_table = torch.tensor([[11]], dtype=torch.int32, device="cuda")
    table[0, 3] = 3
    new, kept, _ = K.kv_evict(cache, table, lens, s, 100, recent=50, out_table=out_table)
    assert K.kv_get_last_error(clear=True) == K.KV_DERR_TABLE
    assert int(new[0]) == 100 and kept[0, :50].tolist() == list(range(50))
    lens.fill_(1000)
    new, _, _ = K.kv_evict(cache, table, lens, s, 200)
    assert K.kv_get_last_error(clear=True) == K.KV_DERR_TABLE and int(new[0]) == 160


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
def test_a_requests_life():
    """Tokens are written through the block table, a chunk and two decode steps attend to them, the weights of all
    steps and both layers are summed, the cache is trimmed in place, and decoding goes on over what stayed."""
    heads, kv_heads, d, block, lens = 8, 2, 64, 16, [200, 90, 333]
    budget, sinks, recent, scale = 80, 4, 24, 64 ** -0.5
    layers = [Batch(lens, [n + 3 for n in lens], heads, kv_heads, d, block=block, layout="blocks_first", seed=s) for s in (1, 2)]
    table = layers[0].table
    for b in layers:
        b.table = table
        b.tensors[0].fill_(float("nan"))
    cache = K.PagedCache.from_tensors([b.tensors[0] for b in layers], "blocks_first")
    rows = [[[x.cuda() for x in b.k_rows], [x.cuda() for x in b.v_rows]] for b in layers]
    score = torch.zeros(3, max(lens) + 8, device="cuda")
    held = [0, 0, 0]
    weights = [torch.zeros(n + 3, dtype=torch.float64) for n in lens]
    K.kv_get_last_error(clear=True)
    g = torch.Generator().manual_seed(5)
    for step, new in enumerate((lens, [1, 1, 1], [1, 1, 1])):
        req = torch.cat([torch.full((n,), r) for r, n in enumerate(new)]).to(torch.int32).cuda()
        pos = torch.cat([torch.arange(h, h + n) for h, n in zip(held, new)]).to(torch.int32).cuda()
        fresh = [torch.cat([layer[plane][r][h:h + n] for r, (h, n) in enumerate(zip(held, new))]) for layer in rows for plane in range(2)]
        K.kv_write_tokens(cache, fresh, table, req, pos)
        held = [h + n for h, n in zip(held, new)]
        kv = torch.tensor(held, dtype=torch.int32, device="cuda")
        offsets = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device="cuda")
        for i, b in enumerate(layers):
            q = torch.randn(sum(new), heads, d, generator=g).to(BF)
            out, lse = K.kv_attention(q.cuda(), cache, table, offsets, kv, scale, k_tensor=i)
            o, l, to, tl = reference(q, [k[:h] for k, h in zip(b.k_rows, held)], [v[:h] for v, h in zip(b.v_rows, held)], new, scale)
            close(out, o, to, "out")
            close(lse, l, tl, "lse")
            K.kv_attention_mass(q.cuda(), cache, table, offsets, kv, lse, scale, k_tensor=i, prev=score, score=score)
            b.q_cpu, b.q_lens, b.kv_lens = q, list(new), list(held)
            keep = [k for k in b.k_rows]
            b.k_rows = [k[:h] for k, h in zip(b.k_rows, held)]
            got, _ = mass_reference(b, lse, scale, True, 0, max(held))
            b.k_rows = keep
            for r, h in enumerate(held):
                weights[r][:h] += got[r, :h]
    for r, h in enumerate(held):
        assert float((score[r, :h].double().cpu() - weights[r][:h]).abs().max()) < 1e-3 and torch.all(score[r, h:] == 0)
    keeps = [keep_reference(score[r].tolist(), h, budget, sinks, recent) for r, h in enumerate(held)]
    lens_dev, kept, _ = K.kv_evict(cache, table, torch.tensor(held, dtype=torch.int32, device="cuda"), score, budget, sinks=sinks, recent=recent)
    assert [kept[r, :len(k)].tolist() for r, k in enumerate(keeps)] == keeps
    q = torch.randn(3, heads, d, generator=g).to(BF)
    offsets = torch.arange(4, dtype=torch.int32, device="cuda")
    for i, b in enumerate(layers):
        out, lse = K.kv_attention(q.cuda(), cache, table, offsets, lens_dev, scale, k_tensor=i)
        o, l, to, tl = reference(q, [k[j] for k, j in zip(b.k_rows, keeps)], [v[j] for v, j in zip(b.v_rows, keeps)], [1, 1, 1], scale)
        close(out, o, to, "out")
        close(lse, l, tl, "lse")
    assert K.kv_get_last_error(clear=True) == 0


def test_lengths_in_place():
    """A trimmed request's new length may be written over its old one."""
    s = scores(40, 3000, 8).cuda()
    cache = K.PagedCache.from_tensors([torch.zeros(40 * 47, 64, 8, dtype=BF, device="cuda")], "separate")
    table = torch.arange(40 * 47, dtype=torch.int32, device="cuda").view(40, 47)
    old = [3000 - 70 * i for i in range(40)]
    lens = torch.tensor(old, dtype=torch.int32, device="cuda")
    new, kept, _ = K.kv_evict(cache, table, lens, s, 700, sinks=2, recent=9, new_lens=lens)
    assert new is lens and lens.tolist() == [min(n, 700) for n in old]
    for r, n in enumerate(old):
        assert kept[r].tolist() == keep_reference(s[r].tolist(), n, 700, 2, 9) + [-1] * (700 - min(n, 700))


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("width,budget,sinks,recent", [(100, 64, 4, 20), (100, 160, 0, 0), (0, 64, 4, 20), (280, 64, 0, 64), (299, 30, 0, 1), (300, 30, 0, 1)])
def test_scores_narrower_than_the_cache(width, budget, sinks, recent, in_place):
    """Tokens that came after the scores were taken count as 0; none is dropped for it, the last ones least of all."""
    lens = [300, 90, 100, 101, 400]
    s = torch.zeros(5, 400)
    s[:, :width] = scores(5, 400, 2)[:, :width]
    g = torch.Generator().manual_seed(width)
    block, row = 16, 16
    need = [-(-n // block) for n in lens]
    table = torch.full((5, max(need)), -1, dtype=torch.int32)
    ids = torch.randperm(sum(need) + 5 * 10, generator=g).to(torch.int32)
    for r, n in enumerate(need):
        table[r, :n] = ids[sum(need[:r]):sum(need[:r]) + n]
    out_table = table if in_place else ids[sum(need):].view(5, 10).contiguous()
    host = torch.randint(-2 ** 15, 2 ** 15, (len(ids), block, row), generator=g, dtype=torch.int16)
    dev = host.cuda().view(BF)
    K.kv_get_last_error(clear=True)
    new, kept, out = K.kv_evict(K.PagedCache.from_tensors([dev], "separate"), table.cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
                                s[:, :width].contiguous().cuda(), budget, sinks=sinks, recent=recent, out_table=None if in_place else out_table.cuda())
    assert K.kv_get_last_error(clear=True) == 0
    got = dev.view(torch.int16).cpu()
    for r, n in enumerate(lens):
        keep = keep_reference(s[r].tolist(), n, budget, sinks, recent)
        assert int(new[r]) == len(keep) == min(n, budget)
        assert kept[r].tolist() == keep + [-1] * (budget - len(keep))
        assert out[r].tolist() == s[r][keep].tolist() + [0.0] * (budget - len(keep))
        j, i = torch.tensor(keep), torch.arange(len(keep))
        assert torch.equal(got[out_table[r].long()[i // block], i % block], host[table[r].long()[j // block], j % block])


def test_narrow_scores_in_place_of_longer_lists():
    """out_score may be the score's buffer when the budget is larger than the columns that hold scores."""
    buf = torch.full((2, 300), 7.0, device="cuda")
    buf[:, :50] = scores(2, 50, 4).cuda()
    want = buf.cpu()
    cache = K.PagedCache.from_tensors([torch.zeros(2 * 30, 16, 8, dtype=BF, device="cuda")], "separate")
    table = torch.arange(60, dtype=torch.int32, device="cuda").view(2, 30)
    _, kept, _ = K.kv_evict(cache, table, torch.tensor([400, 70], dtype=torch.int32, device="cuda"), buf[:, :50], 100, sinks=2, recent=60,
                            out_score=buf)
    for r, n in enumerate((400, 70)):
        s = torch.zeros(n)
        s[:50] = want[r, :50]
        keep = keep_reference(s.tolist(), n, 100, 2, 60)
        assert kept[r, :len(keep)].tolist() == keep
        assert buf[r, :100].tolist() == s[keep].tolist() + [0.0] * (100 - len(keep))
    assert torch.equal(buf[:, 100:].cpu(), want[:, 100:])


@pytest.mark.parametrize("narrow", [False, True])
def test_trimming_again_and_again(narrow):
    """Decode steps and trims in turn: the newest tokens always stay, and a new token's weight starts at nothing.
    narrow: the trimmed scores are handed on as they are, and tokens past their columns count as 0."""
    heads, kv_heads, d, block, budget, sinks, recent, scale, slots = 4, 2, 64, 16, 48, 4, 16, 64 ** -0.5, 96
    g = torch.Generator().manual_seed(3)
    lens = [70, 40, 48]
    table = torch.randperm(18, generator=g).to(torch.int32).view(3, 6).cuda()
    pool = torch.zeros(18, 2, block, kv_heads, d, dtype=BF, device="cuda")
    cache = K.PagedCache.from_tensors([pool], "blocks_first")
    k_rows, v_rows = ([torch.zeros(0, kv_heads, d, dtype=BF) for _ in lens] for _ in range(2))
    score = torch.zeros(3, slots, device="cuda")
    held, names, count = [0, 0, 0], [[], [], []], [0, 0, 0]  # names: each held token's number in its request's life
    K.kv_get_last_error(clear=True)
    for step in range(12):
        new = lens if step == 0 else [1, 1, 1]
        req = torch.cat([torch.full((n,), r) for r, n in enumerate(new)]).to(torch.int32).cuda()
        pos = torch.cat([torch.arange(h, h + n) for h, n in zip(held, new)]).to(torch.int32).cuda()
        k_new, v_new = ([torch.randn(n, kv_heads, d, generator=g).to(BF) for n in new] for _ in range(2))
        K.kv_write_tokens(cache, [torch.cat(k_new).cuda(), torch.cat(v_new).cuda()], table, req, pos)
        k_rows, v_rows = ([torch.cat(x) for x in zip(rows, fresh)] for rows, fresh in ((k_rows, k_new), (v_rows, v_new)))
        for r, n in enumerate(new):
            names[r] += range(count[r], count[r] + n)
            count[r] += n
            assert torch.all(score[r, held[r]:] == 0)  # of tokens that were trimmed nothing is left for the new ones
        held = [h + n for h, n in zip(held, new)]
        kv = torch.tensor(held, dtype=torch.int32, device="cuda")
        offsets = torch.tensor([0] + list(np.cumsum(new)), dtype=torch.int32, device="cuda")
        q = torch.randn(sum(new), heads, d, generator=g).to(BF)
        out, lse = K.kv_attention(q.cuda(), cache, table, offsets, kv, scale)
        o, l, to, tl = reference(q, k_rows, v_rows, new, scale)
        close(out, o, to, "out")
        close(lse, l, tl, "lse")
        b = SimpleNamespace(q_cpu=q, q_lens=new, kv_lens=held, k_rows=k_rows, heads=heads, kv_heads=kv_heads, dk=d)
        want, tol = mass_reference(b, lse, scale, True, 0, score.shape[1], score)
        score = K.kv_attention_mass(q.cuda(), cache, table, offsets, kv, lse, scale, prev=score)
        close(score, want, tol, "mass")
        if step % 2 == 0 or narrow:
            known = [(score[r].tolist() + [0.0] * held[r])[:held[r]] for r in range(3)]
            keeps = [keep_reference(known[r], held[r], budget, sinks, recent) for r in range(3)]
            kv, kept, heavy = K.kv_evict(cache, table, kv, score, budget, sinks=sinks, recent=recent)
            held = [min(h, budget) for h in held]
            assert kv.tolist() == held
            for r, keep in enumerate(keeps):
                assert kept[r, :held[r]].tolist() == keep, (step, r)
                names[r] = [names[r][j] for j in keep]
                k_rows[r], v_rows[r] = k_rows[r][keep], v_rows[r][keep]
            if narrow:
                score = heavy
            else:
                score.zero_()[:, :budget] = heavy
        for r in range(3):
            tail = min(recent, count[r])
            assert names[r][-tail:] == list(range(count[r] - tail, count[r])), (step, r)
    assert K.kv_get_last_error(clear=True) == 0
