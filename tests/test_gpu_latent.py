"""Latent attention (absorbed form) and the expansion of latents, on the GPU against 64-bit references."""
from __future__ import annotations

import pytest
import torch

from paged_kv_cache_81_gb300 import pagedkv as K
from tests.attention_support import NAN, U, Batch, close, reference

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16
SCALE = 0.05


class Latent(Batch):
    def __init__(self, q_lens, kv_lens, heads, *, block=64, dtype=BF, seed=0):
        super().__init__(q_lens, kv_lens, heads, 1, 576, 8, block=block, dtype=dtype, seed=seed)
        self.v_rows = [k[..., :512] for k in self.k_rows]
        self.latent = K.PagedCache.from_tensors([self.tensors[0].view(self.pages, block, 576)], "mla")

    def run(self, scale=SCALE, causal=True, window=0, **kw):
        return K.kv_latent_attention(self.q, self.latent, self.table, self.offsets, self.lens, scale, causal=causal, window=window, **kw)


def check(b, causal=True, window=0, **kw):
    K.kv_get_last_error(clear=True)
    out, lse = b.run(SCALE, causal, window, **kw)
    assert K.kv_get_last_error(clear=True) == 0
    o, l, to, tl = reference(b.q_cpu, b.k_rows, b.v_rows, b.q_lens, SCALE, causal, window)
    close(out, o, to, "out")
    close(lse, l, tl, "lse")
    return out, lse


@pytest.mark.parametrize("q_lens,kv_lens", [([1], [1]), ([1], [63]), ([1], [64]), ([1], [65]), ([1, 1], [1, 500]), ([0, 3, 1], [9, 3, 0]),
                                            ([20, 2], [130, 400]), ([5], [2])])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_lengths(q_lens, kv_lens, dtype):
    check(Latent(q_lens, kv_lens, 16, dtype=dtype, seed=len(q_lens)))


@pytest.mark.parametrize("heads", [1, 7, 16, 20, 64, 100, 128, 130, 131, 160, 192, 256])
def test_heads(heads):
    check(Latent([1, 3], [200, 90], heads, seed=heads))


@pytest.mark.parametrize("block", [1, 2, 16, 24, 48, 64, 128, 17])
def test_pages(block):
    check(Latent([1, 6], [250, 99], 16, block=block, seed=block))


@pytest.mark.parametrize("causal,window", [(False, 0), (True, 1), (True, 64), (True, 100)])
def test_masks(causal, window):
    check(Latent([1, 9, 40], [300, 129, 90], 8, seed=window), causal, window)


@pytest.mark.parametrize("reqs,kv,heads", [(1, 9000, 16), (2, 5000, 128), (5, 700, 32), (90, 130, 128), (3, 2100, 2)])
def test_split_contexts(reqs, kv, heads):
    check(Latent([1] * reqs, [kv - i for i in range(reqs)], heads, seed=kv))


def test_repeated_calls_and_graph():
    b = Latent([1, 2, 1], [3000, 900, 1500], 32, seed=4)
    ws = K.kv_attention_workspace()
    want = [x.clone() for x in check(b, workspace=ws)]
    for _ in range(20):
        assert all(torch.equal(x, y) for x, y in zip(want, b.run(workspace=ws)))
    assert int(ws[:16384].sum()) == 0
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        got = b.run()
    for _ in range(3):
        for x in got:
            x.fill_(1)
        g.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))


def test_strided_rows_and_padding():
    b = Latent([2, 1], [70, 200], 16, seed=4)
    wide = torch.full((5, 20, 584), NAN, dtype=BF, device="cuda")
    wide[:3, 1:17, 8:] = b.q
    b.q = wide[:, 1:17, 8:]
    out = torch.full((5, 17, 512), 2.0, dtype=BF, device="cuda")
    lse = torch.full((5, 16), 4.0, device="cuda")
    b.q_cpu = b.q_cpu[:3]
    got = b.run(out=out[:, 1:], lse=lse)
    o, l, to, tl = reference(b.q_cpu, b.k_rows, b.v_rows, b.q_lens, SCALE)
    close(got[0][:3], o, to, "out")
    close(got[1][:3], l, tl, "lse")
    assert torch.all(out[3:] == 2) and torch.all(out[:, 0] == 2) and torch.all(lse[3:] == 4)


def test_bad_pages_read_as_zeros():
    b = Latent([1, 1], [300, 100], 16, block=32, seed=4)
    b.table[0, 4] = -1
    b.table[1, 3] = b.pages + 9
    b.k_rows[0][128:160] = 0
    b.k_rows[1][96:] = 0
    K.kv_get_last_error(clear=True)
    out, lse = b.run()
    assert K.kv_get_last_error(clear=True) == K.KV_DERR_TABLE
    o, l, to, tl = reference(b.q_cpu, b.k_rows, b.v_rows, b.q_lens, SCALE)
    close(out, o, to, "out")
    close(lse, l, tl, "lse")


# ---------------------------------------------------------------------------
# expansion
# ---------------------------------------------------------------------------
def expand_case(kv_lens, heads, block, out_block, dtype, seed=0):
    g = torch.Generator().manual_seed(seed)
    src = Latent([1] * len(kv_lens), kv_lens, 1, block=block, dtype=dtype, seed=seed)
    dst = Batch([1] * len(kv_lens), kv_lens, heads, heads, 192, 128, block=out_block, dtype=dtype, seed=seed + 1)
    for t in dst.tensors:
        t.fill_(9.0)
    w = (torch.randn(heads, 256, 512, generator=g) / 16).to(dtype)
    return src, dst, w


def expand_reference(src, w, r):
    rows = src.k_rows[r][:, 0].double()
    both = torch.einsum("hod,nd->nho", w.double(), rows[:, :512])
    mag = torch.einsum("hod,nd->nho", w.double().abs(), rows[:, :512].abs())
    tol = U[w.dtype] * both.abs() * 1.01 + 528 * 2.0 ** -24 * mag + 2.0 ** -25
    rope = rows[:, None, 512:].expand(-1, w.shape[0], -1)
    return torch.cat([both[..., :128], rope], -1), both[..., 128:], torch.cat([tol[..., :128], torch.zeros_like(rope)], -1), tol[..., 128:]


@pytest.mark.parametrize("kv_lens", [[1], [127], [128], [129], [0, 3, 0], [300, 1, 140]])
@pytest.mark.parametrize("heads,block,out_block,dtype", [(1, 64, 64, BF), (5, 16, 128, FP), (16, 24, 16, BF)])
def test_expand(kv_lens, heads, block, out_block, dtype):
    src, dst, w = expand_case(kv_lens, heads, block, out_block, dtype)
    K.kv_get_last_error(clear=True)
    K.kv_latent_expand(src.latent, src.table, src.lens, w.cuda(), dst.cache, dst.v_cache, dst.table)
    assert K.kv_get_last_error(clear=True) == 0
    k, v = (t.cpu() for t in dst.tensors)
    seen = torch.zeros(k.shape[:2], dtype=torch.bool)
    for r, n in enumerate(kv_lens):
        want_k, want_v, tol_k, tol_v = expand_reference(src, w, r)
        at = torch.arange(n)
        page, slot = dst.table_cpu[r].long()[at // out_block], at % out_block
        close(k[page, slot], want_k, tol_k, "k")
        close(v[page, slot], want_v, tol_v, "v")
        seen[page, slot] = True
    assert torch.all(k[~seen] == 9) and torch.all(v[~seen] == 9)


def test_expand_bad_pages():
    src, dst, w = expand_case([200, 90], 4, 16, 32, BF)
    src.table[0, 1] = -3
    dst.table[1, 1] = 1 << 29
    K.kv_get_last_error(clear=True)
    K.kv_latent_expand(src.latent, src.table, src.lens, w.cuda(), dst.cache, dst.v_cache, dst.table)
    assert K.kv_get_last_error(clear=True) == K.KV_DERR_TABLE
    src.k_rows[0][16:32] = 0
    k = dst.tensors[0].cpu()
    for r, keep in ((0, range(200)), (1, [j for j in range(90) if not 32 <= j < 64])):
        want_k, _, tol_k, _ = expand_reference(src, w, r)
        at = torch.tensor(list(keep))
        close(k[dst.table_cpu[r].long()[at // 32], at % 32], want_k[at], tol_k[at], "k")
    assert int((k == 9).all(-1).all(-1).sum()) == dst.pages * 32 - 200 - (90 - 32)


def test_expanded_and_absorbed_forms_agree():
    """Attention over expanded keys and values is latent attention with the projections absorbed: out = W_v o,
    q = [W_k^T q_nope ; q_rope].  Each form against the 64-bit definition of the whole."""
    heads, lens = 8, [300, 65]
    src, dst, w = expand_case(lens, heads, 64, 64, BF, seed=3)
    g = torch.Generator().manual_seed(9)
    q = torch.randn(2, heads, 192, generator=g).to(BF)
    scale = 192 ** -0.5
    offsets = torch.tensor([0, 1, 2], dtype=torch.int32, device="cuda")
    K.kv_latent_expand(src.latent, src.table, src.lens, w.cuda(), dst.cache, dst.v_cache, dst.table)
    out, lse = K.kv_attention(q.cuda(), dst.cache, dst.table, offsets, src.lens, scale, v_cache=dst.v_cache)
    wk, wv = w[:, :128].double(), w[:, 128:].double()
    absorbed = torch.cat([torch.einsum("thd,hdr->thr", q[..., :128].double(), wk), q[..., 128:].double()], -1).to(BF)
    o2, lse2 = K.kv_latent_attention(absorbed.cuda(), src.latent, src.table, offsets, src.lens, scale)
    o2 = torch.einsum("thr,hor->tho", o2.double().cpu(), wv)
    for r, n in enumerate(lens):
        k, v, _, _ = expand_reference(src, w, r)
        s = torch.einsum("hd,nhd->hn", q[r].double(), k) * scale
        size = torch.einsum("hd,nhd->hn", q[r].double().abs(), k.abs()) * scale
        p = torch.softmax(s, -1)
        want = torch.einsum("hn,nho->ho", p, v)
        # a score is off by at most u of its size (keys, or queries, rounded once); weights by twice that; values,
        # weights and the result are rounded once each
        d = 2.0 ** -8 * size.amax(-1)[:, None]
        tol = (2 * d * torch.exp(2 * d) + 3 * 2.0 ** -8) * torch.einsum("hn,nho->ho", p, v.abs()) + 2.0 ** -8 * want.abs()
        assert bool(((out[r].double().cpu() - want).abs() <= tol).all())
        latent_mag = torch.einsum("hn,nr->hr", p, src.k_rows[r][:, 0, :512].double().abs())
        tol2 = (2 * d * torch.exp(2 * d) + 3 * 2.0 ** -8) * torch.einsum("hr,hor->ho", latent_mag, wv.abs())
        assert bool(((o2[r] - want).abs() <= tol2).all())
        assert bool(((lse[r].cpu() - torch.logsumexp(s, -1)).abs() <= d[:, 0] + 1e-4).all())
        assert bool(((lse2[r].cpu() - torch.logsumexp(s, -1)).abs() <= 2.0 ** -8 * 4 * size.amax(-1) + 1e-4).all())


# Many requests of few rows take a kernel of their own: up to 64 rows a request on average, and no more rows than requests.
SHORT = [1, 31, 32, 33, 63, 64, 65, 95, 97, 128, 500, 3, 2, 129, 40, 0, 1300, 10, 20, 160]


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 1), (True, 32), (True, 50)])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_many_requests(causal, window, dtype):
    q_lens = [(1, 1, 2, 0, 5, 1)[i % 6] for i in range(60)]
    check(Latent(q_lens, SHORT * 3, 16, dtype=dtype, seed=window), causal, window)


@pytest.mark.parametrize("heads,reqs", [(1, 20), (7, 20), (16, 24), (33, 40), (64, 64), (48, 80), (5, 300)])
def test_many_requests_heads(heads, reqs):
    check(Latent([1] * reqs, [(SHORT[i % 20] + i) % 900 for i in range(reqs)], heads, seed=heads))


@pytest.mark.parametrize("block", [1, 3, 8, 16, 17, 24, 32, 256])
def test_many_requests_pages(block):
    check(Latent([1, 2] * 10, SHORT, 4, block=block, seed=block))


@pytest.mark.parametrize("reqs,heads", [(20, 16), (70, 64)])
def test_many_requests_split_contexts(reqs, heads):
    b = Latent([1] * reqs, [2500 - 30 * i for i in range(reqs)], heads, seed=reqs)
    ws = K.kv_attention_workspace()
    want = [x.clone() for x in check(b, workspace=ws)]
    for _ in range(10):
        assert all(torch.equal(x, y) for x, y in zip(want, b.run(workspace=ws)))
    assert int(ws[:16384].sum()) == 0
    # a long unit before short ones and one request of all the rows: units of more than one unit a request
    check(Latent([40] + [1] * 39, [4000] + [5] * 39, 16, seed=1))


def test_many_requests_padding_and_bad_pages():
    b = Latent([1, 2, 0, 1] * 6, [70, 200, 10, 33] * 6, 12, seed=4)
    b.q = torch.cat([b.q, torch.full((9, 12, 576), NAN, dtype=BF, device="cuda")])
    out, lse = torch.full((33, 12, 512), 2.0, dtype=BF, device="cuda"), torch.full((33, 12), 4.0, device="cuda")
    K.kv_get_last_error(clear=True)
    b.run(out=out, lse=lse)
    assert K.kv_get_last_error(clear=True) == 0
    o, l, to, tl = reference(b.q_cpu[:24], b.k_rows, b.v_rows, b.q_lens, SCALE)
    close(out[:24], o, to, "out")
    close(lse[:24], l, tl, "lse")
    assert (out[24:] == 2).all() and (lse[24:] == 4).all()

    b.table[1, 2] = b.pages  # tokens 128-191 of request 1
    b.k_rows[1][128:192] = 0
    b.run(out=out, lse=lse)
    assert K.kv_get_last_error(clear=True) != 0
    o, l, to, tl = reference(b.q_cpu[:24], b.k_rows, b.v_rows, b.q_lens, SCALE)
    close(out[:24], o, to, "out")
    close(lse[:24], l, tl, "lse")


def test_many_requests_with_more_heads_than_rows():
    check(Latent([1, 0, 0] * 10, SHORT + SHORT[:10], 67, seed=3))


def test_capacity_is_the_same_for_many_requests():
    """A table that could hold more tokens than short tiles can count still works."""
    b = Latent([1] * 64, [40 + i for i in range(64)], 8, block=1024, seed=3)
    table = torch.full((64, 1 << 20), -1, dtype=torch.int32, device="cuda")  # 2^30 tokens a request
    table[:, : b.table.shape[1]] = b.table
    b.table = table
    check(b)


@pytest.mark.parametrize("heads,reqs", [(16, 300), (100, 150)])
def test_many_short_contexts(heads, reqs):
    """Pieces of many units: their ends move to the units' edges."""
    b = Latent([1] * reqs, [(37 * i) % 1000 + 1 for i in range(reqs)], heads, seed=heads)
    want = check(b)
    for _ in range(5):
        assert all(torch.equal(x, y) for x, y in zip(want, b.run()))


@pytest.mark.parametrize("heads", [1, 3])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_expand_tile_after_tile(heads, dtype):
    """Few heads and many token tiles: a CTA replaces its latents in tensor memory after every few products."""
    lens, block = [60000, 33333], 64
    g = torch.Generator(device="cuda").manual_seed(heads)
    need = [-(-n // block) for n in lens]
    ids = torch.randperm(sum(need), generator=g, device="cuda").to(torch.int32)
    table = torch.full((2, need[0]), -1, dtype=torch.int32, device="cuda")
    table[0], table[1, : need[1]] = ids[: need[0]], ids[need[0]:]
    pool = torch.randn(sum(need), block, 576, generator=g, device="cuda").to(dtype)
    w = (torch.randn(heads, 256, 512, generator=g, device="cuda") / 16).to(dtype)
    k, v = (torch.zeros(sum(need), block, heads, d, dtype=dtype, device="cuda") for d in (192, 128))
    latent, k_cache, v_cache = K.PagedCache.from_tensors([pool], "mla"), *(K.PagedCache.from_tensors([x], "separate") for x in (k, v))
    kv_lens = torch.tensor(lens, dtype=torch.int32, device="cuda")
    first = None
    for _ in range(8):
        k.fill_(9), v.fill_(9)
        K.kv_latent_expand(latent, table, kv_lens, w, k_cache, v_cache, table)
        if first is None:
            first = k.clone(), v.clone()
        assert torch.equal(k, first[0]) and torch.equal(v, first[1])
    for r, n in enumerate(lens):
        at = torch.arange(n, device="cuda")
        page, slot = table[r].long()[at // block], at % block
        rows = pool[page, slot].double()
        for h in range(heads):
            want = rows[:, :512] @ w[h].double().t()
            # rounded once; sums of 512 terms and the order of 32 bits as in expand_reference
            tol = U[dtype] * want.abs() * 1.01 + 528 * 2.0 ** -24 * (rows[:, :512].abs() @ w[h].double().abs().t()) + 2.0 ** -25
            got = torch.cat([k[page, slot, h, :128], v[page, slot, h]], 1).double()
            assert bool(((got - want).abs() <= tol).all())
            assert torch.equal(k[page, slot, h, 128:].double(), rows[:, 512:])
