"""kv_rope_frequencies and what the rotating writes refuse before they touch the GPU (the C ABI, no GPU needed)."""
from __future__ import annotations

import ctypes
import math

import pytest
import torch

from paged_kv_cache_81_gb300 import build
from paged_kv_cache_81_gb300 import pagedkv as K
from tests.test_attention_refusals import cache

OK, ARG, ALIGN, RANGE, UNSUPPORTED = K.KV_OK, K.KV_ERR_INVALID_ARG, K.KV_ERR_ALIGN, K.KV_ERR_RANGE, K.KV_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build.build()
    return K.load()


def radians(turns):
    return [(t % 2 ** 64) / 2.0 ** 64 * 2 * math.pi for t in turns.tolist()]


@pytest.mark.parametrize("d,base", [(2, 10000.0), (64, 10000.0), (128, 500000.0), (80, 1e6), (512, 1.5)])
def test_plain_linear_and_base(lib, d, base):
    plain = [base ** (-2 * i / d) for i in range(d // 2)]
    for how, want in ((dict(), plain), (dict(scaling="linear", factor=4.0), [w / 4 for w in plain])):
        turns, m = K.kv_rope_frequencies(d, base, **how)
        # powers and divisions in 64 bits: some steps of 2^-53
        assert m == 1.0 and radians(turns) == pytest.approx(want, rel=2.0 ** -48)
    if d > 2:
        turns, m = K.kv_rope_frequencies(d, base, scaling="base", factor=8.0)
        got = radians(turns)
        assert got[0] == pytest.approx(1.0, rel=2.0 ** -48)
        assert got[-1] == pytest.approx(plain[-1] / 8.0, rel=2.0 ** -44)  # the slowest pair by the factor


def test_bands_and_yarn(lib):
    d, base, length, f = 128, 10000.0, 4096.0, 16.0
    plain = [base ** (-2 * i / d) for i in range(d // 2)]
    got = radians(K.kv_rope_frequencies(d, base, scaling="bands", factor=f, original_length=length)[0])
    for w, g in zip(plain, got):
        turns = length * w / (2 * math.pi)
        mix = 1.0 if turns >= 4 else 0.0 if turns <= 1 else (turns - 1) / 3
        assert g == pytest.approx(w * mix + w / f * (1 - mix), rel=2.0 ** -44)
    turns, m = K.kv_rope_frequencies(d, base, scaling="yarn", factor=f, original_length=length)
    assert m == pytest.approx(0.1 * math.log(f) + 1, rel=2.0 ** -23)
    at = [d * math.log(length / (n * 2 * math.pi)) / (2 * math.log(base)) for n in (32, 1)]
    low, high = math.floor(at[0]), math.ceil(at[1])
    for i, (w, g) in enumerate(zip(plain, radians(turns))):
        stay = 1 - min(max((i - low) / (high - low), 0), 1)
        assert g == pytest.approx(w * stay + w / f * (1 - stay), rel=2.0 ** -44)
    assert 0 < low < high < d // 2  # both ends and the mix are in the range


def test_frequencies_refused(lib):
    out, m = (ctypes.c_uint64 * 64)(), ctypes.c_float(0)

    def run(d=128, base=10000.0, kind=0, factor=1.0, length=4096.0, fast=32.0, slow=1.0, to=out):
        return lib.kv_rope_frequencies(d, base, ctypes.byref(K.KvRopeScaling(kind, factor, length, fast, slow)), to, ctypes.byref(m))
    assert run() == OK and lib.kv_rope_frequencies(128, 10000.0, None, out, None) == OK
    nan, inf = float("nan"), float("inf")
    assert run(d=0) == ARG and run(d=7) == ARG and run(d=-2) == ARG and run(to=None) == ARG
    assert run(base=1.0) == ARG and run(base=nan) == ARG and run(base=inf) == ARG and run(base=-5.0) == ARG
    assert run(kind=5) == ARG and run(kind=-1) == ARG
    for kind in (1, 2, 3, 4):
        assert run(kind=kind, factor=0.0) == ARG and run(kind=kind, factor=nan) == ARG and run(kind=kind, factor=inf) == ARG
        assert run(kind=kind, factor=2.0) == OK
    for kind in (3, 4):
        assert run(kind=kind, length=0.0) == ARG and run(kind=kind, fast=1.0) == ARG and run(kind=kind, slow=0.0) == ARG and run(kind=kind, fast=inf) == ARG
    assert run(d=2, kind=2, factor=2.0) == ARG
    with pytest.raises(ValueError):
        K.kv_rope_frequencies(64, scaling="other")


def test_frequencies_that_are_no_numbers(lib):
    """Factors so small that a frequency (or the changed base) leaves 64-bit floating point: no such frequency has a fraction of a turn."""
    for kw in (dict(scaling="linear", factor=1e-310), dict(scaling="bands", factor=1e-310), dict(scaling="yarn", factor=1e-310)):
        with pytest.raises(K.KvError):
            K.kv_rope_frequencies(64, 10000.0, **kw)
    with pytest.raises(K.KvError):
        K.kv_rope_frequencies(4, 10000.0, scaling="base", factor=1e-200)
    out = (ctypes.c_uint64 * 2)(7, 7)
    assert lib.kv_rope_frequencies(4, 10000.0, ctypes.byref(K.KvRopeScaling(1, 1e-310, 4096.0, 32.0, 1.0)), out, None) == ARG
    assert list(out) == [7, 7]  # left as they were
    turns, _ = K.kv_rope_frequencies(4, 10000.0, scaling="base", factor=1e200)  # the slowest pair slows down to nothing
    assert turns.tolist()[1] == 0 and radians(turns)[0] == pytest.approx(1.0, rel=2.0 ** -48)


def rope(rot=64, offset=0, inter=0, m=1.0, turns=0x1000):
    return K.KvRope(turns, rot, offset, inter, m)


def test_rotate_arguments(lib):
    def run(dtype=0, heads=4, d=128, x=0x10000, xs=(1024, 256), o=0x20000, os=(1024, 256), n=5, pos=0x3000, r=None, null=False):
        return lib.kv_rotate(dtype, heads, d, x, *xs, o, *os, n, pos, None if null else r or rope(), 0, None)
    assert run(n=0) == OK and run(heads=0) == OK and run(n=0, x=None, o=None, pos=None) == OK
    assert run(dtype=2) == ARG and run(heads=-1) == ARG and run(d=0) == ARG and run(n=-1) == ARG and run(null=True) == ARG
    assert run(x=None) == ARG and run(o=None) == ARG and run(pos=None) == ARG and run(xs=(-16, 256)) == ARG
    assert run(d=100) == ALIGN and run(x=0x10008) == ALIGN and run(xs=(1000, 256)) == ALIGN and run(os=(1024, 8)) == ALIGN
    assert run(r=rope(rot=-2)) == ARG and run(r=rope(offset=-8)) == ARG and run(r=rope(turns=None)) == ARG
    assert run(r=rope(m=float("nan"))) == ARG and run(r=rope(m=float("inf"))) == ARG
    assert run(r=rope(rot=144)) == RANGE and run(r=rope(rot=64, offset=72)) == RANGE and run(r=rope(rot=1 << 30, offset=1 << 30)) == RANGE
    assert run(r=rope(rot=24)) == ALIGN and run(r=rope(rot=20, inter=1)) == ALIGN and run(r=rope(offset=4)) == ALIGN and run(r=rope(turns=0x1004)) == ALIGN
    assert run(d=1024, r=rope(rot=528)) == UNSUPPORTED and run(d=1 << 17) == UNSUPPORTED and run(n=1 << 31) == UNSUPPORTED


def tokens(**kw):
    d = dict(dtype=0, n_heads=8, n_kv_heads=2, head_dim=128, head_dim_v=128, q=0x10000, q_token_stride=2048, q_head_stride=256, q_out=0x20000,
             q_out_token_stride=2048, q_out_head_stride=256, k=0x30000, k_token_stride=512, k_head_stride=256, v=0x40000, v_token_stride=512,
             v_head_stride=256, token_req=0x5000, token_pos=0x6000, rope_pos=None, n_tokens=4, block_table=0x7000, n_reqs=2, max_blocks_per_req=8,
             bt_row_stride=8)
    return K.KvNewTokens(**{**d, **kw})


def test_write_arguments(lib):
    def run(t=None, r=None, k=None, v=None, kt=0, kp=0, vt=0, vp=0):
        return lib.kv_rotate_write(t or tokens(), r or rope(), k or cache(), kt, kp, v or cache(), vt, vp, None)
    assert run(tokens(n_tokens=0, q=None, k=None, v=None, token_req=None, token_pos=None, block_table=None)) == OK
    assert lib.kv_rotate_write(None, rope(), cache(), 0, 0, cache(), 0, 0, None) == ARG
    for bad in (dict(dtype=3), dict(n_heads=-1), dict(n_kv_heads=0), dict(head_dim=0), dict(head_dim_v=-8), dict(n_tokens=-1), dict(n_reqs=-1),
                dict(max_blocks_per_req=-1), dict(bt_row_stride=7), dict(q=None), dict(q_out=None), dict(k=None), dict(v=None), dict(token_req=None),
                dict(token_pos=None), dict(block_table=None), dict(k_token_stride=-512)):
        assert run(tokens(**bad)) == ARG, bad
    for bad in (dict(q=0x10008), dict(q_out=0x20004), dict(k=0x30002), dict(v=0x40008), dict(k_head_stride=250), dict(head_dim=100), dict(head_dim_v=100)):
        assert run(tokens(**bad)) == ALIGN, bad
    assert run(tokens(n_tokens=1 << 31)) == UNSUPPORTED
    assert run(r=rope(rot=144)) == RANGE and run(r=rope(rot=24)) == ALIGN
    assert run(k=cache(row=256)) == ARG and run(v=cache(row=256)) == ARG and run(kt=1) == ARG and run(vp=1) == ARG and run(v=cache(block_size=8)) == ARG
    assert run(k=cache(num_blocks=0)) == ARG


def test_q4_arguments(lib):
    row = K.kv_q4_row_bytes(2, 128)
    assert row == 144
    for (h, d), want in {(1, 32): 32, (1, 64): 48, (1, 128): 80, (8, 128): 576, (3, 96): 176, (8, 64): 288}.items():
        assert K.kv_q4_row_bytes(h, d) == want  # codes and scales, up to a multiple of 16
    out = ctypes.c_int32(0)
    assert lib.kv_q4_row_bytes(2, 128, None) == ARG and lib.kv_q4_row_bytes(0, 128, ctypes.byref(out)) == ARG
    assert lib.kv_q4_row_bytes(2, 48, ctypes.byref(out)) == ALIGN and lib.kv_q4_row_bytes(2, 160, ctypes.byref(out)) == UNSUPPORTED

    def run(t=None, k=None, v=None, ks=1.0, vs=1.0, kh=None, vh=None):
        return lib.kv_rotate_write_q4(t or tokens(), rope(rot=32), k or cache(row=row), 0, 0, v or cache(row=row), 0, 0, ks, vs, kh, vh, None)
    assert run(tokens(n_tokens=0)) == OK
    assert run(k=cache(row=512)) == ARG and run(v=cache(row=512)) == ARG and run(tokens(dtype=7)) == ARG
    assert run(tokens(head_dim_v=0)) == UNSUPPORTED
    assert run(tokens(head_dim=48, k_head_stride=96), k=cache(row=64)) == ALIGN
    assert run(tokens(head_dim=160, k_head_stride=320), k=cache(row=192)) == UNSUPPORTED
    for bad in (0.0, -1.0, float("nan"), float("inf"), 1e-35):
        assert run(ks=bad) == ARG and run(vs=bad) == ARG
    assert run(kh=0x50008) == ALIGN and run(vh=0x50004) == ALIGN


def test_struct_sizes(lib):
    assert ctypes.sizeof(K.KvRope) == 24 and ctypes.sizeof(K.KvRopeScaling) == 40 and ctypes.sizeof(K.KvNewTokens) == 176
