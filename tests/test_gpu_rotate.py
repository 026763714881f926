"""kv_rotate, kv_rotate_write and kv_rotate_write_q4 on the GPU against 64-bit references."""
from __future__ import annotations

import math

import pytest
import torch

from paged_kv_cache_81_gb300 import pagedkv as K
from tests.attention_support import close
from tests.rotate_support import held, packed, plane, q4_pages, quantised, rotated, tolerance

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


def randn(seed, dtype, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(dtype)


def positions(seed, n, most):
    return torch.randint(0, most, (n,), generator=torch.Generator().manual_seed(seed), dtype=torch.int32)


def check_rotate(x, pos, turns, **kw):
    rope = K.Rope(turns.cuda(), offset=kw.get("offset", 0), interleaved=kw.get("interleaved", False), magnitude=kw.get("magnitude", 1.0))
    out = K.kv_rotate(x.cuda(), pos.cuda(), rope, inverse=kw.get("inverse", False))
    want, size = rotated(x, turns, pos, **kw)
    close(out, want, tolerance(want, size, x.dtype), "rotated")
    return out


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("heads,dim,rot,offset", [(1, 16, 16, 0), (3, 64, 64, 0), (5, 80, 32, 48), (2, 128, 128, 0), (4, 192, 64, 128), (7, 128, 32, 40),
                                                  (1, 576, 64, 512), (2, 512, 512, 0), (33, 24, 16, 8)])
def test_heads_and_parts(dtype, interleaved, heads, dim, rot, offset):
    turns, _ = K.kv_rope_frequencies(rot)
    check_rotate(randn(heads, dtype, 9, heads, dim), positions(dim, 9, 5000), turns, offset=offset, interleaved=interleaved)


@pytest.mark.parametrize("tokens", [1, 2, 152, 1025])
@pytest.mark.parametrize("inverse", [False, True])
def test_tokens(tokens, inverse):
    turns, _ = K.kv_rope_frequencies(32)
    check_rotate(randn(1, BF, tokens, 3, 48), positions(2, tokens, 100), turns, offset=8, inverse=inverse)


@pytest.mark.parametrize("scaling", ["none", "linear", "base", "bands", "yarn"])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_far_positions(scaling, dtype):
    """The angle of a far position is as good as that of a near one, up to the largest and to negative ones."""
    turns, m = K.kv_rope_frequencies(128, 500000.0, scaling=scaling, factor=8.0)
    pos = torch.tensor([0, 1, -1, 8191, 1 << 20, (1 << 31) - 1, -(1 << 31), 123456789], dtype=torch.int32)
    check_rotate(randn(3, dtype, 8, 2, 128), pos, turns, magnitude=m)


def test_every_angle_of_a_turn():
    """Angles all around the turn, and on the steps that the kernel takes it in, by pairs (1, 0) and (0, 1)."""
    g = torch.Generator().manual_seed(5)
    turns = torch.cat([torch.arange(128, dtype=torch.int64) << 55, (torch.arange(64, dtype=torch.int64) << 57) + 1,
                       torch.randint(-(1 << 62), 1 << 62, (64,), generator=g)])
    x = torch.zeros(16, 2, 512, dtype=BF)
    x[:, 0, :256] = 1
    x[:, 1, 256:] = 1
    pos = torch.tensor([0, 1, 2, 3, 5, 7, 64, 65, 127, 255, 256, 257, -1, -2, 511, 100003], dtype=torch.int32)
    check_rotate(x, pos, turns)


def test_rotation_undone_and_gradient():
    """inverse is the transposed map: <R x, y> = <x, R^T y>, against differences of the forward map too."""
    turns, m = K.kv_rope_frequencies(64, scaling="yarn", factor=4.0)
    rope = K.Rope(turns.cuda(), offset=32, magnitude=m)
    x, y = (randn(s, FP, 40, 6, 96).cuda() for s in (1, 2))
    pos = positions(3, 40, 100000).cuda()
    fx, by = K.kv_rotate(x, pos, rope), K.kv_rotate(y, pos, rope, inverse=True)
    a, b = (fx.double() * y.double()).sum(-1), (x.double() * by.double()).sum(-1)
    # both sides are rounded once, elements by 2^-11 of their size, at most m (|a| + |b|) each
    size = m * 2 * (x.double().abs().amax(-1) * y.double().abs().sum(-1) + y.double().abs().amax(-1) * x.double().abs().sum(-1))
    assert torch.all((a - b).abs() <= 2.0 ** -11 * 1.01 * size)
    # a difference of the forward map along one element is a column of it (the map is linear): 2 x - x
    e = torch.zeros_like(x)
    e[:, :, 40] = 1.0
    column = K.kv_rotate(e, pos, rope).double()
    want = (column * y.double()).sum(-1)
    assert torch.all((want - by[:, :, 40].double()).abs() <= 2.0 ** -11 * 1.01 * m * 3 * y.double().abs().amax(-1))


def test_in_place_strides_and_rows_around():
    turns, _ = K.kv_rope_frequencies(64)
    rope = K.Rope(turns.cuda(), offset=16)
    pos = positions(1, 30, 4000)
    base = randn(4, BF, 31, 9, 104).cuda()
    was = base.clone()
    x = base[:30, 2:7, 8:104]
    want, size = rotated(x.cpu(), turns, pos, offset=16)
    out = K.kv_rotate(x, pos.cuda(), rope, out=x)
    assert out.data_ptr() == x.data_ptr()
    close(x, want, tolerance(want, size, BF), "in place")
    was[:30, 2:7, 8:104] = x
    assert torch.equal(base, was)
    # heads first, into another layout
    y = randn(5, BF, 30, 5, 96).cuda().permute(1, 0, 2).contiguous().permute(1, 0, 2)
    want, size = rotated(y.cpu(), turns, pos, offset=16)
    close(K.kv_rotate(y, pos.cuda(), rope), want, tolerance(want, size, BF), "heads first")


def test_special_values_stay_special():
    """Infinities and NaN in what does not rotate pass; in what does they make their pair infinite or NaN, nothing else."""
    turns, _ = K.kv_rope_frequencies(16)
    x = torch.ones(2, 1, 32, dtype=BF)
    x[0, 0, 20], x[0, 0, 21], x[1, 0, 3] = float("inf"), float("nan"), float("nan")
    out = K.kv_rotate(x.cuda(), torch.tensor([5, 5], dtype=torch.int32).cuda(), K.Rope(turns.cuda())).cpu()
    assert out[0, 0, 20] == float("inf") and torch.isnan(out[0, 0, 21]) and torch.isfinite(out[0, 0, :20]).all()
    assert torch.isnan(out[1, 0, 3]) and torch.isnan(out[1, 0, 11]) and torch.isfinite(out[1, 0]).sum() == 30


# ---------------------------------------------------------------------------
# writes
# ---------------------------------------------------------------------------
class New:
    """New tokens of a ragged batch as parts of one projection's rows, their places, and what the cache should hold."""

    def __init__(self, q_lens, kv_lens, heads, kv_heads, dk, dv, *, block=16, dtype=BF, seed=0, shift=0, spread=1.0):
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // block) for n in kv_lens]
        self.pages, self.block, self.heads, self.kv_heads, self.dk, self.dv, self.dtype = sum(need) + 3, block, heads, kv_heads, dk, dv, dtype
        ids = torch.randperm(self.pages, generator=g)
        self.table = torch.full((len(kv_lens), max([1] + need) + 1), -1, dtype=torch.int32)
        at = 0
        for r, n in enumerate(need):
            self.table[r, :n] = ids[at:at + n].to(torch.int32)
            at += n
        places = [(r, n - m + i) for r, (m, n) in enumerate(zip(q_lens, kv_lens)) for i in range(m)]
        order = torch.randperm(len(places), generator=g).tolist()  # a batch's tokens need not be sorted
        self.req = torch.tensor([places[i][0] for i in order], dtype=torch.int32)
        self.pos = torch.tensor([places[i][1] for i in order], dtype=torch.int32)
        self.rope_pos = self.pos + shift
        t = len(places)
        row = (torch.randn(t, heads * dk + kv_heads * (dk + dv) + 8, generator=g) * spread).to(dtype).cuda()
        self.q = row[:, :heads * dk].unflatten(1, (heads, dk)) if heads else None
        self.k = row[:, heads * dk:(heads + kv_heads) * dk].unflatten(1, (kv_heads, dk))
        self.v = row[:, (heads + kv_heads) * dk:-8].unflatten(1, (kv_heads, dv)) if dv else None

    def slots(self):
        req, pos = self.req.long(), self.pos.long()
        return self.table[req, pos // self.block].long(), pos % self.block

    def args(self):
        return self.q, self.k, self.v

    def where(self):
        return self.table.cuda(), self.req.cuda(), self.pos.cuda()


def pages16(n, layout, fill=7.0):
    def make(*shape):
        return torch.full(shape, fill, dtype=n.dtype, device="cuda")
    if layout in ("separate", "mla"):
        t = [make(n.pages, n.block, n.kv_heads, d) for d in (n.dk, n.dv) if d]
        return t, K.PagedCache.from_tensors(t[:1], layout), K.PagedCache.from_tensors(t[1:], layout) if n.dv else None
    t = [make(*((n.pages, 2, n.block) if layout == "blocks_first" else (2, n.pages, n.block)), n.kv_heads, n.dk)]
    return t, K.PagedCache.from_tensors(t, layout), None


def check_write(n, layout="separate", rot=None, offset=0, interleaved=False, magnitude=1.0, **kw):
    rot = n.dk if rot is None else rot
    turns, _ = K.kv_rope_frequencies(rot)
    rope = K.Rope(turns.cuda(), offset=offset, interleaved=interleaved, magnitude=magnitude)
    t, cache, v_cache = pages16(n, layout)
    K.kv_get_last_error(clear=True)
    q = K.kv_rotate_write(*n.args(), cache, *n.where(), rope, v_cache=v_cache, rope_pos=n.rope_pos.cuda(), **kw)
    assert K.kv_get_last_error(clear=True) == 0
    how = dict(offset=offset, interleaved=interleaved, magnitude=magnitude)
    page, slot = n.slots()
    if n.heads:
        want, size = rotated(n.q.cpu(), turns, n.rope_pos, **how)
        close(q, want, tolerance(want, size, n.dtype), "q")
    else:
        assert q is None
    want, size = rotated(n.k.cpu(), turns, n.rope_pos, **how)
    got = plane(t, "separate" if layout == "mla" else layout, 0).cpu()
    close(got[page, slot], want, tolerance(want, size, n.dtype), "k")
    got[page, slot] = 7.0
    assert torch.all(got == 7.0)
    if n.dv:
        got = plane(t, layout, 1).cpu()
        assert torch.equal(got[page, slot], n.v.cpu())
        got[page, slot] = 7.0
        assert torch.all(got == 7.0)
    return q, t


@pytest.mark.parametrize("layout", ["separate", "blocks_first", "kv_first"])
@pytest.mark.parametrize("q_lens,kv_lens,block", [([1], [1], 16), ([1, 1, 1], [5, 700, 33], 16), ([0, 7, 0, 40], [3, 7, 9, 90], 24), ([300], [300], 1)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_write(layout, q_lens, kv_lens, block, dtype):
    check_write(New(q_lens, kv_lens, 6, 2, 64, 64, block=block, dtype=dtype, seed=block), layout)


@pytest.mark.parametrize("heads,kv_heads,dk,dv,rot,offset", [(1, 1, 16, 8, 16, 0), (8, 8, 128, 64, 32, 96), (5, 1, 192, 128, 64, 128), (32, 8, 128, 128, 128, 0)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_write_heads(heads, kv_heads, dk, dv, rot, offset, interleaved):
    check_write(New([3, 20], [50, 20], heads, kv_heads, dk, dv, seed=dk, shift=1000), "separate", rot, offset, interleaved, magnitude=1.25)


def test_write_latent_rows_without_values_and_queries():
    check_write(New([1, 30, 2], [1, 300, 64], 0, 1, 576, 0, block=64, dtype=FP, seed=3), "mla", 64, 512, True)


def test_write_without_rotation_is_write_tokens():
    n = New([4, 9], [30, 9], 2, 2, 64, 64, seed=2)
    t, cache, v_cache = pages16(n, "separate")
    q = K.kv_rotate_write(*n.args(), cache, *n.where(), None, v_cache=v_cache)
    u, both, _ = pages16(n, "separate")
    K.kv_write_tokens(K.PagedCache.from_tensors(u, "separate"), [n.k.contiguous(), n.v.contiguous()], *n.where())
    assert torch.equal(q, n.q) and all(torch.equal(a, b) for a, b in zip(t, u))


def test_write_into_named_tensors_and_queries_in_place():
    n = New([4, 9], [30, 9], 4, 2, 64, 64, seed=2)
    t = [torch.full((n.pages, n.block, 2, 64), 7.0, dtype=BF, device="cuda") for _ in range(4)]
    turns, _ = K.kv_rope_frequencies(64)
    rope = K.Rope(turns.cuda())
    before = n.q.cpu()
    q = K.kv_rotate_write(*n.args(), K.PagedCache.from_tensors(t, "separate"), *n.where(), rope, k_tensor=3, v_tensor=1, q_out=n.q)
    assert q is n.q
    want, size = rotated(before, turns, n.pos)
    close(n.q, want, tolerance(want, size, BF), "q")
    page, slot = n.slots()
    want, size = rotated(n.k.cpu(), turns, n.pos)
    close(t[3].cpu()[page, slot], want, tolerance(want, size, BF), "k")
    assert torch.equal(t[1].cpu()[page, slot], n.v.cpu())
    assert torch.all(t[0] == 7) and torch.all(t[2] == 7)


def check_q4(n, layout="separate", rot=None, offset=0, interleaved=False, magnitude=1.0, k_scale=1.0, v_scale=1.0, keep=True):
    """Codes, scales and held values are those of the definition, bit for bit."""
    rot = n.dk if rot is None else rot
    turns, _ = K.kv_rope_frequencies(rot)
    rope = K.Rope(turns.cuda(), offset=offset, interleaved=interleaved, magnitude=magnitude)
    t, cache, v_cache = q4_pages(layout, n.pages, n.block, n.kv_heads, n.dk, n.dv)
    K.kv_get_last_error(clear=True)
    got = K.kv_rotate_write_q4(*n.args(), cache, *n.where(), rope, v_cache=v_cache, rope_pos=n.rope_pos.cuda(), k_scale=k_scale, v_scale=v_scale,
                               held=keep)
    assert K.kv_get_last_error(clear=True) == 0
    how = dict(offset=offset, interleaved=interleaved, magnitude=magnitude)
    q = got[0] if keep else got
    if n.heads:
        want, size = rotated(n.q.cpu(), turns, n.rope_pos, **how)
        close(q, want, tolerance(want, size, n.dtype), "q")
    page, slot = n.slots()
    keys = rotated(n.k.cpu(), turns, n.rope_pos, **how)[0].float().to(n.dtype)
    for which, (rows, scale) in enumerate(((keys, k_scale), (n.v.cpu(), v_scale))):
        code, b = quantised(rows, scale)
        if keep:
            assert torch.equal(got[1 + which].cpu(), held(code, b, scale, n.dtype)), "held values"
        want = packed(code, b)
        used = code.shape[1] * code.shape[2] * 9 // 16
        pages = plane(t, layout, which).cpu()
        assert torch.equal(pages[page, slot][:, :used], want[:, :used]), "codes and scales"
        pages[page, slot, :used] = 0x77
        assert torch.all(pages == 0x77)  # nothing else is written, the bytes that fill a row up among it
    return got, t


@pytest.mark.parametrize("layout", ["separate", "blocks_first", "kv_first"])
@pytest.mark.parametrize("q_lens,kv_lens,block", [([1], [1], 16), ([1, 1, 1], [5, 700, 33], 16), ([0, 7, 0, 40], [3, 7, 9, 90], 24)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_q4_write(layout, q_lens, kv_lens, block, dtype):
    check_q4(New(q_lens, kv_lens, 6, 2, 64, 64, block=block, dtype=dtype, seed=block), layout, v_scale=0.25)


@pytest.mark.parametrize("heads,kv_heads,dk,dv,rot,offset", [(1, 1, 32, 32, 16, 16), (8, 8, 128, 64, 32, 96), (0, 3, 96, 32, 32, 40), (32, 16, 128, 128, 128, 0),
                                                             (2, 1, 128, 96, 64, 8)])
@pytest.mark.parametrize("interleaved", [False, True])
def test_q4_write_heads(heads, kv_heads, dk, dv, rot, offset, interleaved):
    check_q4(New([3, 60], [50, 60], heads, kv_heads, dk, dv, seed=dk, shift=1000000, spread=3.0), "separate", rot, offset, interleaved, magnitude=1.25,
             k_scale=0.75, v_scale=2.0)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_q4_many_elements_bit_for_bit(dtype):
    """Two million keys at far positions: no code depends on how an angle was rounded."""
    check_q4(New([500] * 4, [500] * 4, 0, 8, 128, 128, dtype=dtype, seed=9, shift=1 << 20), "blocks_first", keep=False)


@pytest.mark.parametrize("spread", [2.0 ** -20, 2.0 ** -9, 1000.0, 60000.0])
@pytest.mark.parametrize("scale", [1.0, 0.1, 37.0])
def test_q4_small_and_large_values(spread, scale):
    """Below the smallest scale and above the largest."""
    check_q4(New([40], [40], 0, 2, 64, 64, dtype=BF, seed=1, spread=spread), rot=32, k_scale=scale, v_scale=scale)


def test_q4_every_step_and_border():
    """Values on the borders between codes and one step of bf16 around them, for every scale: ties go to the even code."""
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 0.0])
    bytes_ = torch.arange(1, 127, dtype=torch.uint8)
    rows = (bytes_.view(torch.float8_e4m3fn).float()[:, None] * torch.cat([border, torch.tensor([6.0, -6.0])])).to(BF)
    up = (rows.view(torch.int16) + 1).view(BF)
    down = torch.where(rows == 0, -rows, (rows.view(torch.int16) - 1).view(BF))
    for x in (up, down):
        x[:, 14:] = rows[:, 14:]  # the largest keeps the scale
    v = torch.cat([torch.stack([rows, -rows], 1), torch.stack([up, -down], 1), torch.stack([down, -up], 1)]).reshape(-1, 1, 32)
    n = New([v.shape[0]], [v.shape[0]], 0, 1, 32, 32, seed=1)
    n.v = v.cuda()
    check_q4(n, rot=16)


def test_q4_infinities_are_the_largest_values():
    n = New([2], [2], 0, 1, 32, 32, seed=1)
    n.v = n.v.clone()
    n.v[0, 0, 3], n.v[1, 0, 20] = float("inf"), -float("inf")
    t, cache, v_cache = q4_pages("separate", n.pages, n.block, 1, 32, 32)
    _, _, v = K.kv_rotate_write_q4(*n.args(), cache, *n.where(), None, v_cache=v_cache, held=True)
    assert v[0, 0, 3] == 2688 and v[1, 0, 20] == -2688 and torch.isfinite(v).all()


@pytest.mark.parametrize("four", [False, True])
def test_invalid_tokens_write_nothing_and_are_reported(four):
    n = New([6], [40], 2, 2, 64, 64, seed=4)
    t, cache, v_cache = q4_pages("separate", n.pages, n.block, 2, 64, 64) if four else pages16(n, "separate")
    call = K.kv_rotate_write_q4 if four else K.kv_rotate_write
    rope = K.Rope.make(64)
    good = call(*n.args(), cache, *n.where(), rope, v_cache=v_cache, rope_pos=n.pos.cuda())
    first = [x.clone() for x in t]
    for x, y in zip(t, first):
        x.fill_(0x77 if four else 7.0)
    table, req, pos = n.where()
    for i, (r, p) in enumerate([(1, 0), (-1, 0), (0, -1), (0, 1 << 30), (0, 48)]):
        req[i], pos[i] = r, p  # the last names a table entry of -1
    K.kv_get_last_error(clear=True)
    q = call(*n.args(), cache, table, req, pos, rope, v_cache=v_cache, rope_pos=n.pos.cuda())
    assert K.kv_get_last_error(clear=True) == K.KV_DERR_TABLE
    assert torch.equal(q, good)  # queries go by rope_pos alone
    page, slot = (x[5:] for x in n.slots())
    for x, y in zip(t, first):
        assert torch.equal(x[page, slot], y[page, slot])
        x[page, slot] = 0x77 if four else 7.0
        assert torch.all(x == (0x77 if four else 7.0))
    n.table[0, :2] = n.pages
    table, req, pos = n.where()
    call(*n.args(), cache, table, req, pos, rope, v_cache=v_cache)
    assert K.kv_get_last_error(clear=True) in (K.KV_DERR_SLOT, 0)
    pos[:] = 3
    call(*n.args(), cache, table, req, pos, rope, v_cache=v_cache)
    assert K.kv_get_last_error(clear=True) == K.KV_DERR_SLOT


def test_a_page_that_only_one_cache_has_is_refused_for_both():
    n = New([1], [1], 0, 1, 64, 64, seed=1)
    n.table[0, 0] = 2
    k, v = (torch.full((p, 16, 1, 64), 7.0, dtype=BF, device="cuda") for p in (3, 2))
    K.kv_get_last_error(clear=True)
    K.kv_rotate_write(*n.args(), K.PagedCache.from_tensors([k], "separate"), *n.where(), None, v_cache=K.PagedCache.from_tensors([v], "separate"))
    assert K.kv_get_last_error(clear=True) == K.KV_DERR_SLOT
    assert torch.all(k == 7) and torch.all(v == 7)


def test_nothing_to_write():
    n = New([0, 0], [4, 9], 2, 2, 64, 64, seed=1)
    t, cache, v_cache = pages16(n, "separate")
    q = K.kv_rotate_write(*n.args(), cache, *n.where(), K.Rope.make(64), v_cache=v_cache)
    assert q.shape == (0, 2, 64) and torch.all(t[0] == 7)


@pytest.mark.parametrize("four", [False, True])
def test_streams_and_graphs(four):
    n = New([9, 3], [40, 30], 4, 2, 64, 64, seed=4)
    rope = K.Rope.make(64)
    where = n.where()

    def fresh():
        return q4_pages("blocks_first", n.pages, n.block, 2, 64, 64) if four else pages16(n, "blocks_first")

    def go(cache, **kw):
        return (K.kv_rotate_write_q4 if four else K.kv_rotate_write)(*n.args(), cache, *where, rope, **kw)
    t, cache, _ = fresh()
    want = go(cache).clone()
    torch.cuda.synchronize()
    s = torch.cuda.Stream()
    u, other, _ = fresh()
    torch.cuda.synchronize()
    got = go(other, stream=s)
    s.synchronize()
    assert torch.equal(got, want) and torch.equal(t[0], u[0])
    u, other, _ = fresh()
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        got = go(other)
    for _ in range(3):
        u[0].fill_(0x77 if four else 7.0)
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, want) and torch.equal(t[0], u[0])


def test_python_refusals():
    n = New([2], [20], 2, 2, 64, 64, seed=1)
    t, cache, v_cache = pages16(n, "separate")
    q4, cache4, v4 = q4_pages("separate", n.pages, n.block, 2, 64, 64)
    rope = K.Rope.make(64)
    where = n.where()
    q, k, v = n.args()
    for args, kw in (((q.float(), k, v, cache), {}), ((q, k.half(), v, cache), {}), ((q[:1], k, v, cache), {}), ((q, k, v[:, :1], cache), {}),
                     ((q, k, v, cache4), dict(v_cache=v4)), ((q, k, v, cache), dict(v_cache=None)), ((q, k.cpu(), v, cache), {}),
                     ((None, k, v, cache), dict(q_out=q)), ((q, k, v, cache), dict(q_out=q[:1])), ((q, k, v, cache), dict(rope_pos=where[2].long())),
                     ((q, k, v, cache), dict(k_tensor=1 << 40))):
        with pytest.raises(ValueError):
            K.kv_rotate_write(*args, *where, rope, **{**dict(v_cache=v_cache), **kw})
    with pytest.raises(ValueError):
        K.kv_rotate_write_q4(q, k, v, cache, *where, rope, v_cache=v_cache)
    with pytest.raises(ValueError):
        K.Rope(torch.zeros(4, device="cuda"))
    with pytest.raises(ValueError):
        K.Rope(torch.zeros(4, dtype=torch.int64))
    with pytest.raises(ValueError):
        K.kv_rotate(q, where[2][:1], rope)
    with pytest.raises(K.KvError):
        K.kv_rotate(q, where[2], K.Rope.make(128))


# ---------------------------------------------------------------------------
# many tokens, wide strides, far pages
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("heads,dim,tokens,interleaved", [(128, 64, 21000, False), (9, 16, 200000, True), (40, 128, 45000, False), (1, 576, 150000, True)])
def test_many_tokens_as_few(heads, dim, tokens, interleaved):
    """A long call, whose blocks take many tokens each, gives what short ones give."""
    x = torch.randn(tokens, heads, dim, generator=torch.Generator("cuda").manual_seed(dim), device="cuda", dtype=BF)
    pos = positions(heads, tokens, 1 << 30).cuda()
    rope = K.Rope.make(16, offset=dim - 16, interleaved=interleaved)
    out = K.kv_rotate(x, pos, rope)
    for at in range(0, tokens, 300):
        assert torch.equal(out[at:at + 300], K.kv_rotate(x[at:at + 300], pos[at:at + 300], rope))
    assert torch.equal(K.kv_rotate(x, pos, rope, out=x), out)


@pytest.mark.parametrize("four", [False, True])
@pytest.mark.parametrize("heads,kv_heads,dk,tokens", [(16, 4, 64, 72000), (32, 8, 128, 21000), (0, 1, 32, 180000), (90, 20, 64, 11000)])
def test_many_tokens_written_as_few(four, heads, kv_heads, dk, tokens):
    g = torch.Generator("cuda").manual_seed(dk)
    row = torch.randn(tokens, (heads + 2 * kv_heads) * dk, generator=g, device="cuda", dtype=FP)
    q, k, v = (x.unflatten(1, (-1, dk)) if x.shape[1] else None for x in row.split([heads * dk, kv_heads * dk, kv_heads * dk], 1))
    pages = tokens // 16 + 3
    table = torch.randperm(pages, generator=g, device="cuda").to(torch.int32)[None]
    pos = torch.randperm(tokens, generator=g, device="cuda").to(torch.int32)
    req = torch.zeros_like(pos)
    req[::97] = -1  # written nowhere
    rope, at = K.Rope.make(dk), torch.randint(0, 1 << 30, (tokens,), generator=g, device="cuda", dtype=torch.int32)
    width = K.kv_q4_row_bytes(kv_heads, dk) if four else kv_heads * dk
    call = K.kv_rotate_write_q4 if four else K.kv_rotate_write
    kw = dict(held=True, k_scale=0.5) if four else {}

    def run(spans):
        t = [torch.full((pages, 16, width), 7, dtype=torch.uint8 if four else FP, device="cuda") for _ in range(2)]
        cache, v_cache = (K.PagedCache.from_tensors([x], "separate") for x in t)
        got = [call(q[a:b] if heads else None, k[a:b], v[a:b], cache, table, req[a:b], pos[a:b], rope, v_cache=v_cache, rope_pos=at[a:b], **kw) for a, b in spans]
        return t, got
    few, parts = run([(a, min(a + 300, tokens)) for a in range(0, tokens, 300)])
    many, whole = run([(0, tokens)])
    assert all(torch.equal(a, b) for a, b in zip(few, many))
    joined = [torch.cat(x) if x[0] is not None else None for x in zip(*parts)] if four else [torch.cat(parts) if heads else None]
    for a, b in zip(joined, whole[0] if four else whole):
        assert (a is None and b is None) or torch.equal(a, b)
    K.kv_get_last_error(clear=True)


def test_q4_many_key_heads():
    check_q4(New([3, 20], [50, 20], 2, 136, 128, 128, seed=1))


@pytest.mark.parametrize("four", [False, True])
def test_write_padded_rows_and_pages_past_4_gib(four):
    n = New([3, 20], [50, 20], 4, 2, 64, 64, seed=1)
    t, cache, v_cache = q4_pages("separate", n.pages, 16, 2, 64, 64) if four else pages16(n, "separate")
    call, rope = K.kv_rotate_write_q4 if four else K.kv_rotate_write, K.Rope.make(64)
    want = call(*n.args(), cache, *n.where(), rope, v_cache=v_cache)
    flat = [x.flatten(2) for x in t]
    width = flat[0].shape[2]
    pad = 16 // flat[0].element_size()
    far = (5 << 30) // (16 * (width + pad) * flat[0].element_size())
    wide = [torch.empty(far + n.pages, 16, width + pad, dtype=x.dtype, device="cuda") for x in flat]
    for x in wide:
        x[far:].fill_(0x77 if four else 7.0)
    n.table = torch.where(n.table < 0, n.table, n.table + far)
    caches = [K.PagedCache.from_tensors([x[:, :, :width]], "separate") for x in wide]
    got = call(*n.args(), caches[0], *n.where(), rope, v_cache=caches[1])
    assert torch.equal(got, want)
    for x, y in zip(flat, wide):
        assert torch.equal(y[far:, :, :width], x) and torch.all(y[far:, :, width:] == (0x77 if four else 7.0))
