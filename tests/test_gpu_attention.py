"""kv_attention on the GPU against 64-bit references: shapes, masks, page layouts, strides, streams, graphs."""
from __future__ import annotations

import math

import pytest
import torch

from paged_kv_cache_81_gb300 import pagedkv as K
from tests.attention_support import NAN, Batch, check, close, reference

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


@pytest.mark.parametrize("q_lens,kv_lens", [
    ([1], [1]), ([1], [2]), ([1], [127]), ([1], [128]), ([1], [129]), ([1, 1, 1], [1, 500, 16]),
    ([0, 3, 0, 1], [5, 3, 0, 40]), ([5, 1], [5, 300]), ([130], [130]), ([64, 1, 65], [64, 700, 200]), ([300], [1000]),
])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_lengths(q_lens, kv_lens, dtype):
    check(Batch(q_lens, kv_lens, 8, 2, 128, dtype=dtype, seed=len(kv_lens)))


@pytest.mark.parametrize("dk,dv", [(8, 8), (40, 24), (64, 64), (64, 128), (72, 64), (80, 80), (128, 128), (128, 64), (136, 128), (192, 128), (192, 64)])
def test_head_widths(dk, dv):
    check(Batch([1, 70], [200, 333], 4, 2, dk, dv, dtype=FP, seed=dk))


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (3, 3), (3, 1), (14, 2), (10, 2), (128, 1), (200, 2), (64, 64)])
def test_head_groups(heads, kv_heads):
    check(Batch([1, 5, 40], [300, 77, 131], heads, kv_heads, 64, seed=heads))


@pytest.mark.parametrize("block", [1, 2, 3, 8, 16, 17, 24, 48, 64, 128, 192, 256, 384])
@pytest.mark.parametrize("layout", ["separate", "blocks_first", "kv_first"])
def test_pages(block, layout):
    check(Batch([1, 9, 140], [400, 9, 390], 4, 1, 64, block=block, layout=layout, seed=block))


@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 1), (True, 2), (True, 100), (True, 128), (True, 129), (True, 5000)])
def test_masks(causal, window):
    check(Batch([1, 3, 200, 0], [700, 129, 300, 9], 6, 2, 128, block=16, seed=window), causal=causal, window=window)


def test_more_new_tokens_than_cached():
    """Positions before the cache see nothing when causal: out 0, lse -inf."""
    b = Batch([9, 130], [4, 3], 4, 2, 64, seed=5)
    out, lse = check(b)
    assert torch.all(out[:5] == 0) and torch.all(lse[:5] == float("-inf"))
    check(b, causal=False)


@pytest.mark.parametrize("reqs,kv", [(1, 20000), (2, 9000), (3, 4111)])
def test_long_contexts_are_split(reqs, kv):
    """A few rows over many tiles: every CTA holds a fragment, and the fragments are joined."""
    check(Batch([1] * reqs, [kv] * reqs, 8, 2, 128, seed=kv))
    check(Batch([3] * reqs, [kv] * reqs, 8, 1, 64, dtype=FP, seed=kv))
    check(Batch([1] * reqs, [kv] * reqs, 2, 2, 64, dtype=FP, seed=kv))  # one row a unit
    check(Batch([150] + [1] * (reqs - 1), [kv] * reqs, 4, 1, 192, 128, seed=kv))


@pytest.mark.parametrize("q_len,heads,kv_heads,kv,dim", [(1, 128, 1, 9000, 128), (4, 32, 1, 33333, 128), (16, 16, 2, 8200, 128), (1, 100, 1, 6700, 64),
                                                         (7, 9, 1, 25000, 64)])
def test_many_pieces_of_many_rows(q_len, heads, kv_heads, kv, dim):
    """Units of more than a dozen pieces are joined in two stages, in the same order every time."""
    b = Batch([q_len], [kv], heads, kv_heads, dim, block=64, seed=kv)
    ws = K.kv_attention_workspace()
    want = [x.clone() for x in check(b, workspace=ws)]
    for _ in range(20):
        got = b.run(dim ** -0.5, workspace=ws)
        assert all(torch.equal(x, y) for x, y in zip(want, got))
    assert int(ws[:16384].sum()) == 0
    # one long request before short ones: equal pieces, of which some hold the ends of two units
    check(Batch([q_len] + [1] * 30, [kv] + [300] * 30, heads, kv_heads, dim, block=64, seed=kv))


def test_many_short_requests():
    lens = [1 + 37 * i % 300 for i in range(700)]
    check(Batch([1] * 700, lens, 4, 2, 64, block=8, seed=1))


@pytest.mark.parametrize("spread", [1e-3, 30.0])
def test_flat_and_peaked_scores(spread):
    """Weights that are all alike, and ones where a single key takes it all and the maximum moves by hundreds."""
    check(Batch([2, 40], [900, 500], 4, 2, 128, spread=spread, seed=3))
    check(Batch([2, 40], [900, 500], 4, 2, 64, spread=spread, dtype=FP, seed=4))


def test_growing_scores_rescale():
    """Keys whose scores rise from tile to tile, so that every tile moves the maximum."""
    b = Batch([1], [1500], 4, 1, 64, seed=8)
    q = torch.ones_like(b.q_cpu)
    rows = torch.full_like(b.k_rows[0], 1.0) * (torch.arange(1500) / 100.0).to(BF)[:, None, None]
    for j in range(1500):
        b.tensors[0][b.table_cpu[0, j // 16], j % 16] = rows[j].cuda()
    b.k_rows[0], b.q_cpu, b.q = rows, q, q.cuda()
    check(b, scale=1.0)


def test_strides_of_q_and_out():
    b = Batch([3, 70], [90, 200], 6, 2, 64, seed=2)
    wide = torch.full((73, 9, 96), NAN, dtype=BF, device="cuda")
    wide[:, 2:8, 16:80] = b.q
    b.q = wide[:, 2:8, 16:80]
    base = torch.full((73, 8, 72), 7.0, dtype=BF, device="cuda")
    out, _ = check(b, out=base[:, 1:7, 8:])
    assert out.data_ptr() == base[:, 1:7, 8:].data_ptr()
    assert torch.all(base[:, 0] == 7) and torch.all(base[:, 7] == 7) and torch.all(base[:, :, :8] == 7)


def test_heads_first_q():
    b = Batch([5, 200], [90, 300], 4, 2, 128, seed=2)
    b.q = b.q.permute(1, 0, 2).contiguous().permute(1, 0, 2)
    check(b)


def test_rows_behind_the_last_sequence_stay():
    b = Batch([3, 2], [90, 20], 4, 2, 64, seed=2)
    b.q = torch.cat([b.q, torch.full((4, 4, 64), NAN, dtype=BF, device="cuda")])
    out = torch.full((9, 4, 64), 3.0, dtype=BF, device="cuda")
    lse = torch.full((9, 4), 5.0, device="cuda")
    check(b, out=out, lse=lse)
    assert torch.all(out[5:] == 3) and torch.all(lse[5:] == 5)


def test_pages_before_the_window_are_not_read():
    """Table entries wholly before every window may be stale: -1 or any other page."""
    b = Batch([1, 30], [500, 400], 4, 2, 64, block=16, seed=6)
    t = b.table
    t[0, : (500 - 64) // 16] = -1
    t[1, : (400 - 30 - 64 + 1) // 16] = 1 << 30
    check(b, window=64)


def test_values_of_unused_slots_never_matter():
    b = Batch([1, 4], [130, 7], 4, 2, 64, block=64, seed=9)
    first = [x.clone() for x in check(b)]
    for t in b.tensors:
        t[torch.isnan(t)] = float("inf")
    second = check(b)
    assert all(torch.equal(x, y) for x, y in zip(first, second))


def test_bad_table_entries_read_as_zeros():
    b = Batch([1, 1], [100, 50], 4, 2, 64, block=16, layout="blocks_first", seed=6)
    b.table[0, 2] = -7
    b.table[1, 0] = b.pages
    for r, page in ((0, 2), (1, 0)):
        b.k_rows[r][page * 16:(page + 1) * 16] = 0
        b.v_rows[r][page * 16:(page + 1) * 16] = 0
    K.kv_get_last_error(clear=True)
    out, lse = b.run(0.125)
    assert K.kv_get_last_error(clear=True) == K.KV_DERR_TABLE
    o, l, to, tl = reference(b.q_cpu, b.k_rows, b.v_rows, b.q_lens, 0.125)
    close(out, o, to, "out")
    close(lse, l, tl, "lse")


def test_lengths_outside_the_table_are_clamped():
    b = Batch([1, 1], [64, 64], 4, 2, 64, block=16, seed=6)
    want = [x.clone() for x in check(b)]
    b.table = b.table[:, :4].contiguous()
    b.lens = torch.tensor([1 << 30, -5], dtype=torch.int32, device="cuda")
    out, lse = b.run(64 ** -0.5)
    assert K.kv_get_last_error(clear=True) == K.KV_DERR_TABLE
    assert torch.equal(out[0], want[0][0]) and torch.equal(lse[0], want[1][0])
    assert torch.all(out[1] == 0) and torch.all(lse[1] == float("-inf"))


def test_inconsistent_offsets_are_clamped():
    b = Batch([2, 2], [64, 64], 4, 2, 64, block=16, seed=6)
    want = b.run(0.125)[0].clone()
    b.offsets = torch.tensor([0, 2, 1 << 20], dtype=torch.int32, device="cuda")
    K.kv_get_last_error(clear=True)
    assert torch.equal(b.run(0.125)[0], want)
    assert K.kv_get_last_error(clear=True) == K.KV_DERR_LIST
    b.offsets = torch.tensor([0, 4, 2], dtype=torch.int32, device="cuda")
    b.run(0.125)
    assert K.kv_get_last_error(clear=True) == K.KV_DERR_LIST


def test_nothing_to_do():
    b = Batch([0, 0], [5, 9], 4, 2, 64, seed=1)
    out, lse = b.run(0.125)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)


def test_same_call_same_bits_and_workspace_left_zero():
    b = Batch([1, 200, 1, 7], [9000, 900, 3000, 5000], 8, 2, 128, seed=1)
    ws = K.kv_attention_workspace()
    first = [x.clone() for x in b.run(0.1, workspace=ws)]
    for _ in range(20):
        again = b.run(0.1, workspace=ws)
        assert all(torch.equal(x, y) for x, y in zip(first, again))
    assert int(ws[:16384].sum()) == 0
    assert all(torch.equal(x, y) for x, y in zip(first, b.run(0.1)))


def test_another_stream():
    b = Batch([1, 60], [3000, 900], 8, 2, 64, seed=1)
    want = [x.clone() for x in b.run(0.1)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = b.run(0.1, stream=s)  # its outputs and workspace belong to that stream
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    with torch.cuda.stream(s):
        got = b.run(0.1)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))


def test_two_streams_at_once():
    bs = [Batch([1, 60, 3], [3000, 900, 2000], 8, 2, 64, seed=i) for i in range(2)]
    want = [[x.clone() for x in b.run(0.1)] for b in bs]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in bs]
    got = [[], []]
    for _ in range(10):
        for i, (b, s) in enumerate(zip(bs, streams)):
            with torch.cuda.stream(s):
                got[i].append(b.run(0.1))
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        assert all(torch.equal(x, y) for r in runs for x, y in zip(w, r))


def test_captured_graph_follows_the_lengths():
    b = Batch([1, 1, 1], [3000, 900, 40], 8, 2, 64, seed=1)
    b.run(0.1)
    s = torch.cuda.Stream()
    graphs, outs = [], []
    for _ in range(2):  # two graphs, neither given a workspace: each has its own
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(b.run(0.1))
        graphs.append(g)
    for lens in ([3000, 900, 40], [1, 500, 39], [2999, 0, 17]):
        b.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        torch.cuda.synchronize()
        streams = [torch.cuda.Stream() for _ in graphs]
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        o, l, to, tl = reference(b.q_cpu, [k[:n] for k, n in zip(b.k_rows, lens)], [v[:n] for v, n in zip(b.v_rows, lens)], b.q_lens, 0.1)
        for out, lse in outs:
            close(out, o, to, "out")
            close(lse, l, tl, "lse")


def test_cache_of_several_layers_and_one_tensor_list():
    """Keys and values of a layer named by their tensors in one description."""
    a, b = Batch([2], [70], 4, 2, 64, seed=1), Batch([2], [70], 4, 2, 64, seed=1)
    cache = K.PagedCache.from_tensors([a.tensors[1], a.tensors[0], b.tensors[0], b.tensors[1]], "separate")
    want = a.run(0.125)
    got = K.kv_attention(a.q, cache, a.table, a.offsets, a.lens, 0.125, k_tensor=2, v_tensor=3)
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    got = K.kv_attention(a.q, cache, a.table, a.offsets, a.lens, 0.125, k_tensor=1, v_tensor=0)
    assert all(torch.equal(x, y) for x, y in zip(want, got))


def test_large_pool_offsets_past_32_bits():
    """Pages beyond 4 GiB of one tensor."""
    block, pages = 64, 140000  # 140000 * 64 * 512 bytes = 4.6 GB
    k = torch.empty(pages, block, 2, 128, dtype=BF, device="cuda")
    v = torch.empty(pages, block, 2, 128, dtype=BF, device="cuda")
    ids = torch.tensor([[139999, 5, 131073, 70000]], dtype=torch.int32)
    g = torch.Generator().manual_seed(0)
    kr, vr = (torch.randn(250, 2, 128, generator=g).to(BF) for _ in range(2))
    for j in range(4):
        n = min(64, 250 - 64 * j)
        k[ids[0, j], :n], v[ids[0, j], :n] = kr[64 * j:64 * j + n].cuda(), vr[64 * j:64 * j + n].cuda()
    q = torch.randn(2, 4, 128, generator=g).to(BF)
    out, lse = K.kv_attention(q.cuda(), K.PagedCache.from_tensors([k], "separate"), ids.cuda(), torch.tensor([0, 2], dtype=torch.int32, device="cuda"),
                              torch.tensor([250], dtype=torch.int32, device="cuda"), 0.1, v_cache=K.PagedCache.from_tensors([v], "separate"))
    o, l, to, tl = reference(q, [kr], [vr], [2], 0.1)
    close(out, o, to, "out")
    close(lse, l, tl, "lse")


def test_capture_of_a_named_stream():
    """A call that names the capturing stream: its outputs and workspace are the graph's, not the stream's."""
    b = Batch([1, 2], [900, 300], 8, 2, 64, seed=3)
    s = torch.cuda.Stream()
    want = [x.clone() for x in b.run(0.1)]
    b.run(0.1, stream=s)  # the stream has a workspace of its own by now
    torch.cuda.synchronize()
    kept = len(K._workspaces)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g, stream=s):
        got = b.run(0.1, stream=s)
    for _ in range(2):
        for x in got:
            x.zero_()
        g.replay()
    torch.cuda.synchronize()
    assert len(K._workspaces) == kept
    assert all(torch.equal(x, y) for x, y in zip(want, got))


@pytest.mark.parametrize("window", [2 ** 30, 2 ** 31 - 1])
def test_windows_longer_than_any_context(window):
    b = Batch([1, 3, 200, 9], [700, 129, 300, 4], 6, 2, 128, seed=1)
    want = check(b)
    got = b.run(128 ** -0.5, True, window)
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    args = (b.q, b.cache, b.table, b.offsets, b.lens, want[1], 128 ** -0.5)
    assert torch.equal(K.kv_attention_mass(*args), K.kv_attention_mass(*args, window=window))


@pytest.mark.parametrize("causal,window", [(True, 0), (False, 0), (True, 150)])
def test_many_short_units(causal, window):
    """Pieces of many units: their ends move to the units' edges."""
    q = [300 + 7 * i for i in range(48)]
    b = Batch(q, [n + 13 * i for i, n in enumerate(q)], 12, 12, 64, seed=window, dtype=FP)
    want = check(b, causal=causal, window=window)
    for _ in range(5):
        assert all(torch.equal(x, y) for x, y in zip(want, b.run(64 ** -0.5, causal, window)))


@pytest.mark.parametrize("more_keys", [True, False])
@pytest.mark.parametrize("dtype,dv", [(BF, 64), (FP, 128)])
def test_pools_of_different_sizes(more_keys, dtype, dv):
    """A page that only one of the two pools has is outside the cache: zeros from both, whatever that page holds."""
    b = Batch([1, 3], [100, 50], 4, 2, 64, dv, block=16, dtype=dtype, seed=6)
    large = 0 if more_keys else 1
    pools = [b.tensors[0], b.tensors[1]]
    more = torch.full((9, *pools[large].shape[1:]), NAN, dtype=dtype, device="cuda")
    pools[large] = torch.cat([pools[large], more])
    b.tensors = pools
    b.cache, b.v_cache = (K.PagedCache.from_tensors([x], "separate") for x in pools)
    check(b)  # the pages that both have
    b.table[0, 2] = b.pages  # the first that one lacks, the last that the other has, and one that neither has
    b.table[0, 4] = b.pages + 8
    b.table[1, 0] = b.pages + 9
    for r, page in ((0, 2), (0, 4), (1, 0)):
        b.k_rows[r][page * 16:(page + 1) * 16] = 0
        b.v_rows[r][page * 16:(page + 1) * 16] = 0
    K.kv_get_last_error(clear=True)
    out, lse = b.run(0.125)
    assert K.kv_get_last_error(clear=True) == K.KV_DERR_TABLE
    o, l, to, tl = reference(b.q_cpu, b.k_rows, b.v_rows, b.q_lens, 0.125)
    close(out, o, to, "out")
    close(lse, l, tl, "lse")


@pytest.mark.parametrize("op,n_reqs", [("attention", 8400), ("attention", 16400), ("mass", 4200), ("mass", 8200), ("latent", 16500), ("latent", 33000)])
def test_offsets_that_name_the_same_tokens_again_and_again(op, n_reqs):
    """Every other request takes the whole batch: their steps pass 2^31, and 2^32, although the batch is within the limits.
    It is reported, nothing is computed, and the next call is right."""
    tokens, heads, kv_heads, dk, dv, block = (8192, 16, 1, 576, 512, 64) if op == "latent" else (32768, 32, 8, 64, 64, 16)
    pool = torch.zeros(4, block, kv_heads * dk, dtype=BF, device="cuda")
    cache = K.PagedCache.from_tensors([pool], "separate")
    q = torch.zeros(tokens, heads, dk, dtype=BF, device="cuda")
    table = torch.zeros(n_reqs, tokens // block, dtype=torch.int32, device="cuda")
    offsets = torch.zeros(n_reqs + 1, dtype=torch.int32, device="cuda")
    offsets[1::2] = tokens
    lens = torch.full((n_reqs,), tokens, dtype=torch.int32, device="cuda")
    lse = torch.full((tokens, heads), 5.0, device="cuda")
    # steps of one such request: rows of 64 (latent), 256 or, for the mass, tokens in steps of 32, against tiles of 32 or 128 keys
    if op == "latent":
        each = sum((4 * u + 3) // 32 + 1 for u in range(tokens // 4))
    elif op == "mass":
        each = sum((tokens - 128 * t + 31) // 32 * kv_heads for t in range(tokens // 128))
    else:
        each = sum((64 * u + 63) // 128 + 1 for u in range(tokens // 64)) * kv_heads
    assert each * (n_reqs // 2) >= 2 ** 31
    K.kv_get_last_error(clear=True)
    if op == "mass":
        out = torch.full((n_reqs, 40), 3.0, device="cuda")
        K.kv_attention_mass(q, cache, table, offsets, lens, lse, 0.1, score=out)
    else:
        out = torch.full((tokens, heads, dv), 3.0, dtype=BF, device="cuda")
        call = K.kv_latent_attention if op == "latent" else K.kv_attention
        call(q, cache, table, offsets, lens, 0.1, out=out, lse=lse, **({} if op == "latent" else dict(v_cache=cache)))
    assert K.kv_get_last_error(clear=True) == K.KV_DERR_LIST
    assert bool((out == 3).all()) and bool((lse == 5).all())
    check(Batch([1, 60], [300, 200], 8, 2, 64, seed=1))


@pytest.mark.parametrize("op", ["attention", "latent", "latent of many heads"])
@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("score", [10.0, 18.0, 21.0])
def test_many_light_weights_behind_a_heavy_one(op, dtype, score):
    """One key takes nearly all; the 8191 others, of weight e^-score each, hold all the value there is.  Their sum has to be
    in the output as it is in the sum of the weights, though each of them is below what an fp16 number can hold."""
    n, reqs, block = 8192, 160, 64
    heads, dk, dv = {"attention": (1, 64, 64), "latent": (1, 576, 512), "latent of many heads": (128, 576, 512)}[op]
    at = 0 if op == "attention" else 512  # the rotary part is no value
    q = torch.zeros(reqs, heads, dk, dtype=dtype, device="cuda")
    q[:, :, at] = 1
    keys = torch.zeros(n // block, block, dk, dtype=dtype, device="cuda")
    if op == "attention":
        values = torch.ones(n // block, block, dv, dtype=dtype, device="cuda")
        values[0, 0] = 0
    else:
        keys[:, :, :512] = 1
        keys[0, 0] = 0
    keys[0, 0, at] = score
    table = torch.arange(n // block, dtype=torch.int32, device="cuda").repeat(reqs, 1)
    lens, offsets = torch.full((reqs,), n, dtype=torch.int32, device="cuda"), torch.arange(reqs + 1, dtype=torch.int32, device="cuda")
    cache = K.PagedCache.from_tensors([keys], "separate")
    if op == "attention":
        out, lse = K.kv_attention(q, cache, table, offsets, lens, 1.0, v_cache=K.PagedCache.from_tensors([values], "separate"))
    else:
        out, lse = K.kv_latent_attention(q, cache, table, offsets, lens, 1.0)
    light = (n - 1) * math.exp(-score)
    want = light / (1 + light)
    # every weight is alike, so their roundings add up: half a step of the type (bf16), or half of fp16's smallest step, 2^-25, of
    # weights held 2^7 times as large; then the output's rounding, and 32-bit sums and exponentials
    u = 2.0 ** -8 if dtype is BF else 2.0 ** -11
    tol = 2 * u * want * 1.01 + (n * 2.0 ** -32 if dtype is FP else 0.0) + 2.0 ** -17 * want
    assert float((out.double() - want).abs().max()) <= tol
    assert float((lse.double() - (score + math.log1p(light))).abs().max()) <= 2.0 ** -21 * (score + 1)
