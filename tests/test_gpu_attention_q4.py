"""kv_attention_q4 on the GPU against 64-bit references: shapes, masks, page layouts, strides, streams, graphs, and a request's life."""
from __future__ import annotations

import math
import os
import subprocess
import sys

import pytest
import torch

from paged_kv_cache_81_gb300 import pagedkv as K
from tests.attention_support import NAN, close, hidden
from tests.q4_support import Q4Batch, check, reference
from tests.rotate_support import U, VALUES, held, packed, plane, quantised, q4_pages, rotated

pytestmark = pytest.mark.gpu

BF, FP = torch.bfloat16, torch.float16


@pytest.mark.parametrize("q_lens,kv_lens", [
    ([1], [1]), ([1], [2]), ([1], [31]), ([1], [64]), ([1], [129]), ([1, 1, 1], [1, 500, 16]),
    ([0, 3, 0, 1], [5, 3, 0, 40]), ([5, 1], [5, 300]), ([130], [130]), ([64, 1, 65], [64, 700, 200]), ([300], [1000]),
])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_lengths(q_lens, kv_lens, dtype):
    check(Q4Batch(q_lens, kv_lens, 8, 2, 128, dtype=dtype, seed=len(kv_lens)))


@pytest.mark.parametrize("dk,dv", [(32, 32), (32, 64), (64, 64), (64, 128), (96, 96), (96, 32), (128, 128), (128, 64), (128, 96)])
@pytest.mark.parametrize("q_lens", [[1, 2], [1, 70]])
def test_head_widths(dk, dv, q_lens):
    check(Q4Batch(q_lens, [200, 333], 4, 2, dk, dv, dtype=FP, seed=dk, k_scale=0.5, v_scale=3.0))


@pytest.mark.parametrize("heads,kv_heads", [(1, 1), (3, 3), (3, 1), (14, 2), (10, 2), (16, 1), (5, 5), (6, 6), (7, 7), (32, 8), (18, 9), (10, 10), (11, 11), (12, 12),
                                            (32, 16), (64, 64), (17, 1), (40, 1), (128, 1), (200, 2)])
@pytest.mark.parametrize("q_lens", [[1, 1, 2], [1, 5, 40], [2, 7, 120]])
def test_head_groups(heads, kv_heads, q_lens):
    check(Q4Batch(q_lens, [300, 77, 131], heads, kv_heads, 64, seed=heads))
    if kv_heads < 20:
        check(Q4Batch(q_lens, [300, 77, 131], heads, kv_heads, 128, dtype=FP, seed=heads))


@pytest.mark.parametrize("block", [1, 2, 3, 8, 16, 17, 24, 48, 64, 128, 192, 384])
@pytest.mark.parametrize("layout", ["separate", "blocks_first", "kv_first"])
@pytest.mark.parametrize("long", [3, 140])
def test_pages(block, layout, long):
    check(Q4Batch([1, 2, long], [400, 9, 390], 4, 1, 64, block=block, layout=layout, seed=block))


@pytest.mark.parametrize("kv_heads", [11, 13, 17, 19])
@pytest.mark.parametrize("block", [1, 3, 17])
@pytest.mark.parametrize("rows", [1, 8, 12, 16, 32])
@pytest.mark.parametrize("dim", [64, 128])
def test_heads_that_come_one_by_one_in_odd_pages(kv_heads, block, rows, dim):
    """Key heads in a prime number, more than a block takes together, whose rows come one by one."""
    check(Q4Batch([rows // 4 or 1] * 3, [600, 33, 1100], kv_heads * min(rows, 4), kv_heads, dim, block=block, dtype=FP if rows == 12 else BF, seed=rows))


@pytest.mark.parametrize("causal,window", [(False, 0), (True, 0), (True, 1), (True, 2), (True, 100), (True, 128), (True, 129), (True, 5000)])
@pytest.mark.parametrize("long", [4, 200])
def test_masks(causal, window, long):
    check(Q4Batch([1, 3, long, 0], [700, 129, 300, 9], 6, 2, 128, block=16, seed=window), causal=causal, window=window)


def test_more_new_tokens_than_cached():
    """Positions before the cache see nothing when causal: out 0, lse -inf."""
    for q_lens in ([3, 2], [9, 130]):
        b = Q4Batch(q_lens, [2, 1], 4, 2, 64, seed=5)
        out, lse = check(b)
        assert torch.all(out[:q_lens[0] - 2] == 0) and torch.all(lse[:q_lens[0] - 2] == float("-inf"))
        check(b, causal=False)


@pytest.mark.parametrize("reqs,kv", [(1, 20000), (2, 9000), (3, 4111)])
def test_long_contexts_are_split(reqs, kv):
    """A few rows over many tiles: every CTA holds a fragment, and the fragments are joined."""
    check(Q4Batch([1] * reqs, [kv] * reqs, 8, 2, 128, seed=kv))
    check(Q4Batch([3] * reqs, [kv] * reqs, 8, 1, 64, dtype=FP, seed=kv))
    check(Q4Batch([1] * reqs, [kv] * reqs, 16, 16, 64, dtype=FP, seed=kv))
    check(Q4Batch([1] * reqs, [kv] * reqs, 2, 2, 64, dtype=FP, seed=kv))  # one row a unit
    check(Q4Batch([50] + [1] * (reqs - 1), [kv] * reqs, 4, 1, 128, 128, seed=kv))


def test_many_pieces_same_bits():
    """Units of many pieces are joined in the same order every time."""
    for q_len, heads, kv_heads, kv, dim in ((1, 32, 8, 40000, 128), (4, 32, 8, 33333, 128), (16, 16, 2, 8200, 128), (1, 100, 1, 6700, 64)):
        b = Q4Batch([q_len], [kv], heads, kv_heads, dim, block=64, seed=kv)
        ws = K.kv_attention_workspace()
        want = [x.clone() for x in check(b, workspace=ws)]
        for _ in range(20):
            assert all(torch.equal(x, y) for x, y in zip(want, b.run(dim ** -0.5, workspace=ws)))
        assert int(ws[:16384].sum()) == 0
        check(Q4Batch([q_len] + [1] * 30, [kv] + [300] * 30, heads, kv_heads, dim, block=64, seed=kv))


@pytest.mark.parametrize("kv_heads", [1, 2, 3, 4, 8, 16, 32])
@pytest.mark.parametrize("group", [1, 6])
@pytest.mark.parametrize("dim", [64, 128])
def test_many_requests_of_whole_rows(kv_heads, group, dim):
    """So many requests that a block takes all heads of a row, some of them with new tokens beyond one unit, the longest cut."""
    g = torch.Generator().manual_seed(kv_heads)
    lens = torch.randint(1, 250, (160,), generator=g).tolist()
    lens[7], lens[33] = 3000, 0
    q_lens = [3 if i % 5 == 0 else 1 for i in range(160)]
    for q, dtype in ((q_lens, BF), ([2 * n for n in q_lens], FP)):
        check(Q4Batch(q, [max(n, m) if n else 0 for n, m in zip(lens, q)], group * kv_heads, kv_heads, dim, block=24 if group + kv_heads == 8 else 16,
                      dtype=dtype, seed=dim))


@pytest.mark.parametrize("kv_heads", [1, 2, 4, 6, 8, 16, 32])
@pytest.mark.parametrize("tokens", [1, 4, 60])
@pytest.mark.parametrize("dim", [64, 128])
def test_tables_as_wide_as_long_contexts(kv_heads, tokens, dim):
    """Few requests that may be long: whole rows of heads, in many pieces."""
    b = Q4Batch([tokens, 1], [4000, 100], 3 * kv_heads, kv_heads, dim, seed=dim)
    b.table = torch.cat([b.table, torch.full((2, 40000), -1, dtype=torch.int32, device="cuda")], 1)
    check(b)


@pytest.mark.parametrize("dtype", [BF, FP])
def test_many_units_of_one_tile(dtype):
    """Prompts whose units have a tile or two each, so that the next unit's queries come while the last one is still being written."""
    lens = [1 + 53 * i % 150 for i in range(900)]
    check(Q4Batch(lens, lens, 4, 1, 64, dtype=dtype, seed=2))
    check(Q4Batch([n // 2 + 33 for n in lens[:300]], [n + 40 for n in lens[:300]], 8, 2, 128, dtype=dtype, seed=3))


@pytest.mark.parametrize("dtype", [BF, FP])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("shorts", [1, 3, 12])
def test_cut_units_before_short_ones(dtype, dim, shorts):
    """Long prompts, whose units are cut and joined, with prompts of one tile and at most 128 rows behind each: the half of a
    block that joins is late for those. The same bits every time, and no wait that runs out."""
    q_lens, kv_lens = [], []
    for i in range(8):
        q_lens += [300] + [20 + (7 * i + 5 * j) % 13 for j in range(shorts)]
        kv_lens += [2000 + 250 * i] + [33 + (31 * i + 17 * j) % 96 for j in range(shorts)]
    b = Q4Batch(q_lens, kv_lens, 8, 2, dim, dtype=dtype, seed=shorts)
    ws = K.kv_attention_workspace()
    want = [x.clone() for x in check(b, workspace=ws)]
    for _ in range(100):
        assert all(torch.equal(x, y) for x, y in zip(want, b.run(dim ** -0.5, workspace=ws)))
    assert K.kv_get_last_error(clear=True) == 0 and int(ws[:16384].sum()) == 0


def test_many_short_requests():
    lens = [1 + 37 * i % 300 for i in range(700)]
    check(Q4Batch([1] * 700, lens, 4, 2, 64, block=8, seed=1))
    check(Q4Batch([i % 3 for i in range(700)], lens, 16, 2, 64, block=8, seed=1))


@pytest.mark.parametrize("spread", [1e-3, 1e-20, 30.0])
@pytest.mark.parametrize("long", [2, 40, 100])
def test_flat_and_peaked_scores(spread, long):
    """Weights that are all alike, and ones where a single key takes it all and the maximum moves by hundreds."""
    check(Q4Batch([2, long], [900, 500], 4, 2, 128, spread=spread, seed=3))
    if spread > 1e-6:  # fp16 holds nothing smaller
        check(Q4Batch([2, long], [900, 500], 4, 2, 64, spread=spread, dtype=FP, seed=4))


@pytest.mark.parametrize("tokens", [4, 64, 200])
@pytest.mark.parametrize("dim", [64, 128])
def test_queries_of_very_different_sizes(tokens, dim):
    """Rows of 2^-100 and of 2^60 beside one another, a row of zeros, and elements far below their row's largest."""
    b = Q4Batch([tokens], [300], 4, 2, dim, seed=6)
    q = b.q_cpu.float()
    q[0] *= 2.0 ** -100
    q[1] = 0
    q[2, :, 1::2] *= 2.0 ** -30
    b.q_cpu = q.to(BF)
    b.q = b.q_cpu.cuda()
    check(b)
    q[0] = q[0] * 2.0 ** 80 * 2.0 ** 80  # the factor at once is no 32-bit number
    b.q_cpu = q.to(BF)
    b.q = b.q_cpu.cuda()
    check(b, scale=2.0 ** -62)


def large_scores(q_lens, kv_lens, heads, kv_heads, dim, dtype, seed):
    """A batch whose products q . K are 2752512 or -2752512 and a whole number of up to 108 beside it: exact in 32 bits, at any scale."""
    b = Q4Batch(q_lens, kv_lens, heads, kv_heads, dim, dtype=dtype, seed=seed)
    g = torch.Generator().manual_seed(seed)
    for r, n in enumerate(kv_lens):
        code = torch.zeros(n, kv_heads, dim, dtype=torch.long)
        code[..., 0] = 7
        code[..., 16:32] = torch.randint(0, 16, (n, kv_heads, 16), generator=g)
        unit = torch.ones(n, kv_heads, dim // 16)
        unit[..., 0] = 448.0
        unit = unit.to(torch.float8_e4m3fn)
        j = torch.arange(n)
        b.tensors[0][b.table_cpu[r, j // 16].long(), j % 16] = packed(code, unit.view(torch.uint8)).cuda()
        b.rows[0][r] = VALUES[code] * unit.double().repeat_interleave(16, -1)
    q = torch.zeros(sum(q_lens), heads, dim)
    q[..., 0], q[..., 16], q[..., 17] = 1024.0, 2.0, 16.0
    q[1::3, :, 0] *= -1
    if dtype == BF:
        q[:, 1::2] *= 2.0 ** 20  # another power of two is taken off these rows
    b.q_cpu = q.to(dtype)
    b.q = b.q_cpu.cuda()
    return b


@pytest.mark.parametrize("scale", [0.125, 1.0, 3.0, 6.0, 16.0, 1024.0, 2.0 ** 40, 1e30])
@pytest.mark.parametrize("q_lens,kv_lens,heads", [([1], [3000], 8), ([3], [3000], 8), ([1] * 30, [150 + 7 * i for i in range(30)], 4), ([100], [3000], 4),
                                                  ([60, 9] * 10, [150, 70] * 10, 4)])
@pytest.mark.parametrize("dim", [64, 128])
@pytest.mark.parametrize("dtype", [BF, FP])
def test_scores_of_any_size(scale, q_lens, kv_lens, heads, dim, dtype):
    """Finite scores up to 3e36: weights that neither pass what fp16 holds nor vanish, out of the differences alone.

    The products are exact. A weight's exponent, c (s - m) + 7, is off by the rounding of c, of the product and of the sum, each 2^-24 of at
    most 45 (what weighs less is lost anyway), and 2^x by 2^-22: 2^-16 in all covers it twice over."""
    b = large_scores(q_lens, kv_lens, heads, 2, dim, dtype, seed=len(q_lens) + dim)
    rows = scale * 2.0 ** -20 if dtype == BF else scale  # of the rows that are 2^20 times as large
    K.kv_get_last_error(clear=True)
    for s in {scale, rows}:
        if s < 1e-30:
            continue
        out, lse = b.run(s)
        at = 0
        for k, v, m in zip(*b.rows, q_lens):
            x, n, group = b.q_cpu[at:at + m].double(), k.shape[0], heads // 2
            kd, vd = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
            z = torch.einsum("mhd,nhd->mhn", x, kd) * float(torch.tensor(s, dtype=torch.float32))
            hide = hidden(m, n, True, 0)[:, None]
            z = z.masked_fill(hide, -math.inf)
            top = z.amax(-1, keepdim=True)
            p = torch.exp(z - top)
            total = p.sum(-1, keepdim=True)
            p /= total
            o, mag = (torch.einsum("mhn,nhd->mhd", p, y) for y in (vd, vd.abs()))
            want = (top + total.log())[..., 0]
            close(out[at:at + m], o, U[dtype] * o.abs() * 1.01 + (2.0 ** -11 * 1.01 + 2.0 ** -16) * mag + n * 2.0 ** -25 * vd.abs().max(), "out")
            fine = want.abs() < 3e38  # the others are no 32-bit numbers
            close(lse[at:at + m][fine.cuda()], want[fine], 2.0 ** -22 * want[fine].abs() + 2.0 ** -15, "lse")
            at += m
    assert K.kv_get_last_error(clear=True) == 0


def test_growing_scores_rescale():
    """Keys whose scores rise from tile to tile, so that every tile moves the maximum."""
    for heads in (4, 40):
        b = Q4Batch([1], [1500], heads, 1, 64, seed=8)
        unit = torch.full((1500, 1, 4), 1.0) * (torch.arange(1500) // 16 / 16.0 + 0.25)[:, None, None]
        unit = unit.to(torch.float8_e4m3fn)
        from tests.rotate_support import packed
        code = torch.full((1500, 1, 64), 2)  # ones
        j = torch.arange(1500)
        b.tensors[0][b.table_cpu[0, j // 16].long(), j % 16] = packed(code, unit.view(torch.uint8)).cuda()
        b.rows[0][0] = unit.double().repeat_interleave(16, -1)
        b.q_cpu = torch.ones_like(b.q_cpu)
        b.q = b.q_cpu.cuda()
        check(b, scale=1.0)


@pytest.mark.parametrize("long", [3, 70])
def test_strides_of_q_and_out(long):
    b = Q4Batch([3, long], [90, 200], 6, 2, 64, seed=2)
    t = 3 + long
    wide = torch.full((t, 9, 96), NAN, dtype=BF, device="cuda")
    wide[:, 2:8, 16:80] = b.q
    b.q = wide[:, 2:8, 16:80]
    base = torch.full((t, 8, 72), 7.0, dtype=BF, device="cuda")
    out, _ = check(b, out=base[:, 1:7, 8:])
    assert out.data_ptr() == base[:, 1:7, 8:].data_ptr()
    assert torch.all(base[:, 0] == 7) and torch.all(base[:, 7] == 7) and torch.all(base[:, :, :8] == 7)
    b.q = b.q_cpu.cuda().permute(1, 0, 2).contiguous().permute(1, 0, 2)
    check(b)


@pytest.mark.parametrize("heads", [4, 64, 96])
def test_rows_behind_the_last_sequence_stay(heads):
    b = Q4Batch([3, 2], [90, 20], heads, 2, 64, seed=2)
    b.q = torch.cat([b.q, torch.full((4, heads, 64), NAN, dtype=BF, device="cuda")])
    out = torch.full((9, heads, 64), 3.0, dtype=BF, device="cuda")
    lse = torch.full((9, heads), 5.0, device="cuda")
    K.kv_get_last_error(clear=True)
    b.run(0.125, out=out, lse=lse)
    assert K.kv_get_last_error(clear=True) == 0
    o, l, to, tl = reference(b.q_cpu, *b.rows, b.q_lens, 0.125)
    close(out[:5], o, to, "out")
    close(lse[:5], l, tl, "lse")
    assert torch.all(out[5:] == 3) and torch.all(lse[5:] == 5)


def test_pages_before_the_window_are_not_read():
    for long in (3, 30, 80):
        b = Q4Batch([1, long], [500, 400], 4, 2, 64, block=16, seed=6)
        b.table[0, : (500 - 64) // 16] = -1
        b.table[1, : (400 - long - 64 + 1) // 16] = 1 << 30
        check(b, window=64)


@pytest.mark.parametrize("heads", [4, 64, 96])
def test_bad_table_entries_read_as_zeros(heads):
    b = Q4Batch([1, 1], [100, 50], heads, 2, 64, block=16, layout="blocks_first", seed=6)
    b.table[0, 2] = -7
    b.table[1, 0] = b.pages
    for r, page in ((0, 2), (1, 0)):
        for rows in b.rows:
            rows[r][page * 16:(page + 1) * 16] = 0
    K.kv_get_last_error(clear=True)
    out, lse = b.run(0.125)
    assert K.kv_get_last_error(clear=True) == K.KV_DERR_TABLE
    o, l, to, tl = reference(b.q_cpu, *b.rows, b.q_lens, 0.125)
    close(out, o, to, "out")
    close(lse, l, tl, "lse")


@pytest.mark.parametrize("heads", [4, 64, 96])
def test_pages_that_only_one_cache_has(heads):
    b = Q4Batch([1], [40], heads, 2, 64, block=16, seed=6)
    have = int(b.table_cpu[0, :3].max())
    if have != int(b.table_cpu[0, 1]):
        at = b.table_cpu[0, :3].tolist().index(have)
    else:
        at = 1
    b.v_cache = K.PagedCache.from_tensors([b.tensors[1][:have]], "separate")  # one page short
    for rows in b.rows:
        rows[0][at * 16:(at + 1) * 16] = 0
    K.kv_get_last_error(clear=True)
    out, lse = b.run(0.125)
    assert K.kv_get_last_error(clear=True) == K.KV_DERR_TABLE
    o, l, to, tl = reference(b.q_cpu, *b.rows, b.q_lens, 0.125)
    close(out, o, to, "out")
    close(lse, l, tl, "lse")


@pytest.mark.parametrize("heads", [4, 64, 96])
def test_lengths_and_offsets_out_of_range_are_clamped(heads):
    b = Q4Batch([1, 1], [64, 64], heads, 2, 64, block=16, seed=6)
    want = [x.clone() for x in check(b)]
    b.table = b.table[:, :4].contiguous()
    b.lens = torch.tensor([1 << 30, -5], dtype=torch.int32, device="cuda")
    out, lse = b.run(64 ** -0.5)
    assert K.kv_get_last_error(clear=True) == K.KV_DERR_TABLE
    assert torch.equal(out[0], want[0][0]) and torch.equal(lse[0], want[1][0])
    assert torch.all(out[1] == 0) and torch.all(lse[1] == float("-inf"))
    b = Q4Batch([2, 2], [64, 64], heads, 2, 64, block=16, seed=6)
    want = b.run(0.125)[0].clone()
    b.offsets = torch.tensor([0, 2, 1 << 20], dtype=torch.int32, device="cuda")
    K.kv_get_last_error(clear=True)
    assert torch.equal(b.run(0.125)[0], want)
    assert K.kv_get_last_error(clear=True) == K.KV_DERR_LIST
    b.offsets = torch.tensor([0, 4, 2], dtype=torch.int32, device="cuda")
    b.run(0.125)
    assert K.kv_get_last_error(clear=True) == K.KV_DERR_LIST


def test_nothing_to_do():
    b = Q4Batch([0, 0], [5, 9], 4, 2, 64, seed=1)
    out, lse = b.run(0.125)
    assert out.shape == (0, 4, 64) and lse.shape == (0, 4)


@pytest.mark.parametrize("heads", [8, 96])
def test_streams_and_graphs(heads):
    b = Q4Batch([1, 3, 2], [3000, 900, 40], heads, 2, 64, seed=1)
    want = [x.clone() for x in b.run(0.1)]
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    got = b.run(0.1, stream=s)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    streams = [torch.cuda.Stream() for _ in range(2)]
    torch.cuda.synchronize()
    runs = []
    for _ in range(10):
        for st in streams:
            with torch.cuda.stream(st):
                runs.append(b.run(0.1))
    torch.cuda.synchronize()
    assert all(torch.equal(x, y) for r in runs for x, y in zip(want, r))
    graphs, outs = [], []
    for _ in range(2):  # two graphs, neither given a workspace: each has its own
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            outs.append(b.run(0.1))
        graphs.append(g)
    for lens in ([3000, 900, 40], [1, 500, 39], [2999, 0, 17]):
        b.lens.copy_(torch.tensor(lens, dtype=torch.int32))
        torch.cuda.synchronize()
        for g, st in zip(graphs, streams):
            with torch.cuda.stream(st):
                g.replay()
        torch.cuda.synchronize()
        o, l, to, tl = reference(b.q_cpu, *[[x[:n] for x, n in zip(rows, lens)] for rows in b.rows], b.q_lens, 0.1)
        for out, lse in outs:
            close(out, o, to, "out")
            close(lse, l, tl, "lse")


_FIRST_CALLS = """
import torch
from paged_kv_cache_81_gb300 import pagedkv as K
from tests.attention_support import Batch
from tests.q4_support import Q4Batch
a, b = Batch([1, 2], [50, 60], 4, 2, 64), Q4Batch([1, 2], [50, 60], 4, 2, 64)
ws = K.kv_attention_workspace()
outs = [torch.empty(3, 4, 64, dtype=torch.bfloat16, device="cuda"), torch.empty(3, 4, device="cuda")]
free = []
for run in (a.run, b.run):
    run(0.1, workspace=ws, out=outs[0], lse=outs[1])
    torch.cuda.synchronize()
    free.append(torch.cuda.mem_get_info()[0])
print(free[0] - free[1])
"""


def test_16_bit_calls_do_not_load_the_kernels_over_4_bits():
    """A process whose first attention call is over 16 bits: the kernels over 4 bits take their memory (and time) with their own first call."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", _FIRST_CALLS], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr
    assert int(r.stdout) > 0


def test_python_refusals():
    b = Q4Batch([1], [20], 4, 2, 64, seed=1)
    args = (b.q, b.cache, b.table, b.offsets, b.lens, 0.125)
    wrong = K.PagedCache.from_tensors([torch.zeros(4, 16, 2, 64, dtype=BF, device="cuda")], "separate")
    for a, kw in (((b.q.float(), *args[1:]), {}), ((b.q, wrong, *args[2:]), {}), (args, dict(v_cache=None)), (args, dict(v_cache=wrong)),
                  (args, dict(kv_heads=1 << 40)), (args, dict(k_tensor=1 << 40)), (args, dict(head_dim_v=-32))):
        with pytest.raises(ValueError):
            K.kv_attention_q4(*a, **{**dict(kv_heads=2, v_cache=b.v_cache), **kw})
    for kw in (dict(kv_heads=4), dict(kv_heads=3), dict(k_scale=0.0), dict(v_scale=float("nan")), dict(head_dim_v=32), dict(causal=False, window=3)):
        with pytest.raises(K.KvError):
            K.kv_attention_q4(*args, **{**dict(kv_heads=2, v_cache=b.v_cache), **kw})


@pytest.mark.parametrize("layout", ["separate", "blocks_first"])
def test_a_requests_life(layout):
    """A prompt is written in 4 bits, its pages move to another pool, tokens are decoded there, the cache is trimmed, decoding goes on."""
    heads, kv_heads, d, block, dtype = 8, 2, 64, 16, BF
    g = torch.Generator().manual_seed(3)
    rope = K.Rope.make(d, 10000.0, scaling="yarn", factor=4.0)
    turns, m = rope.turns.cpu(), rope.desc.magnitude
    scale = d ** -0.5
    total = 100
    qkv = torch.randn(total + 3, heads + 2 * kv_heads, d, generator=g).to(dtype)
    pos = torch.arange(total + 3, dtype=torch.int32)
    keys = rotated(qkv[:, heads:heads + kv_heads], turns, pos, magnitude=m)[0].float().to(dtype)
    k_rows, v_rows = (held(*quantised(x, 1.0), 1.0, torch.float32).double() for x in (keys, qkv[:, heads + kv_heads:]))
    queries = rotated(qkv[:, :heads], turns, pos, magnitude=m)[0].float().to(dtype)
    pools = [q4_pages(layout, 20, block, kv_heads, d, d) for _ in range(2)]
    lists = [[9, 3, 17, 4, 0, 11, 12], [5, 6, 7, 1, 19, 2, 13]]
    tables = [torch.tensor([x], dtype=torch.int32, device="cuda") for x in lists]
    dev = qkv.cuda()

    def parts(a, z):
        return dev[a:z, :heads], dev[a:z, heads:heads + kv_heads], dev[a:z, heads + kv_heads:]

    def step(pool, a, z, at, **kw):
        """Tokens a .. z - 1 written at slots from `at` on and attending there."""
        _, cache, v_cache = pools[pool]
        n = z - a
        slots = torch.arange(at, at + n, dtype=torch.int32, device="cuda")
        q = K.kv_rotate_write_q4(*parts(a, z), cache, tables[pool], torch.zeros(n, dtype=torch.int32, device="cuda"), slots, rope, v_cache=v_cache,
                                 rope_pos=pos[a:z].cuda(), **kw)
        out, lse = K.kv_attention_q4(q, cache, tables[pool], torch.tensor([0, n], dtype=torch.int32, device="cuda"),
                                     torch.tensor([at + n], dtype=torch.int32, device="cuda"), scale, kv_heads=kv_heads, v_cache=v_cache)
        return q, out, lse

    def agree(got, ids, a, z):
        q, out, lse = got
        # the rotated queries may be off by half a step of bf16 here and there: the attention is compared for the ones it got
        o, l, to, tl = reference(q.cpu(), [k_rows[ids]], [v_rows[ids]], [z - a], scale)
        close(out, o, to, "out")
        close(lse, l, tl, "lse")
        assert torch.all((q.cpu().double() - queries[a:z].double()).abs() <= 2.0 ** -7 * queries[a:z].double().abs() + 2.0 ** -20)

    K.kv_get_last_error(clear=True)
    agree(step(0, 0, total, 0), torch.arange(total), 0, total)
    # to the other pool
    off = torch.tensor([0, 7], dtype=torch.int32, device="cuda")
    ids = [torch.tensor(x, dtype=torch.int32, device="cuda") for x in lists]
    for i in range(1 if layout == "blocks_first" else 2):
        src, dst = ((p[1], p[2])[i] for p in pools)
        xfer = K.kv_build_xfer_list(off, *ids)
        K.kv_unpack_blocks(dst, K.kv_pack_blocks(src, xfer, 7), xfer, 7, block)
    agree(step(1, total, total + 1, total), torch.arange(total + 1), total, total + 1)
    # trimmed to 40 tokens by weights that the keys' numbers give; the first 4 and the last 10 stay
    score = ((torch.arange(112) * 37) % 101).float()[None].cuda()
    both = pools[1][1] if layout == "blocks_first" else K.PagedCache.from_tensors(pools[1][0], "separate")
    new_lens, kept, _ = K.kv_evict(both, tables[1], torch.tensor([total + 1], dtype=torch.int32, device="cuda"), score, 40, sinks=4, recent=10)
    kept = kept[0].cpu().long()
    assert int(new_lens[0]) == 40
    agree(step(1, total + 1, total + 3, 40), torch.cat([kept, torch.tensor([total + 1, total + 2])]), total + 1, total + 3)
    assert K.kv_get_last_error(clear=True) == 0


@pytest.mark.parametrize("heads,kv_heads", [(4, 1), (8, 2), (16, 2), (32, 8), (40, 8), (9, 3)])
@pytest.mark.parametrize("long", [2, 90])
@pytest.mark.parametrize("block", [1, 16, 24])
def test_padded_rows(heads, kv_heads, long, block):
    """Rows that do not follow one another without a gap."""
    b = Q4Batch([1, long], [400, 300], heads, kv_heads, 64, block=block, seed=heads)
    want = [x.clone() for x in b.run(0.125)]
    wide = [torch.full((x.shape[0], block, x.shape[2] + 48), 0x7F, dtype=torch.uint8, device="cuda") for x in b.tensors]
    for x, y in zip(b.tensors, wide):
        y[:, :, 16:16 + x.shape[2]] = x
    b.cache, b.v_cache = (K.PagedCache.from_tensors([y[:, :, 16:16 + x.shape[2]]], "separate") for x, y in zip(b.tensors, wide))
    out, lse = check(b, scale=0.125)
    assert torch.allclose(out.float(), want[0].float(), rtol=0, atol=0.02) and torch.allclose(lse, want[1], rtol=0, atol=1e-3)


@pytest.mark.parametrize("long", [2, 90])
def test_pages_past_4_gib(long):
    b = Q4Batch([1, long], [400, 300], 16, 4, 64, seed=3)
    want = [x.clone() for x in b.run(0.125)]
    far = (5 << 30) // (16 * b.tensors[0].shape[2])
    wide = [torch.empty(far + b.pages, 16, x.shape[2], dtype=torch.uint8, device="cuda") for x in b.tensors]
    for x, y in zip(b.tensors, wide):
        y[far:] = x
    b.cache, b.v_cache = (K.PagedCache.from_tensors([y], "separate") for y in wide)
    b.table = torch.where(b.table < 0, b.table, b.table + far)
    assert all(torch.equal(x, y) for x, y in zip(want, b.run(0.125)))
