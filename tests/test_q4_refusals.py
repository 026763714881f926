"""What kv_attention_q4 refuses before it touches the GPU (the C ABI, no GPU needed)."""
from __future__ import annotations

import pytest
import torch

from paged_kv_cache_81_gb300 import build
from paged_kv_cache_81_gb300 import pagedkv as K
from tests.test_attention_refusals import batch, cache, desc

OK, ARG, ALIGN, RANGE, UNSUPPORTED = K.KV_OK, K.KV_ERR_INVALID_ARG, K.KV_ERR_ALIGN, K.KV_ERR_RANGE, K.KV_ERR_UNSUPPORTED
ROW = 144  # two heads of 128


@pytest.fixture(scope="module")
def lib():
    build.build()
    return K.load()


def run(lib, d=None, b=None, k=None, v=None, kt=0, kp=0, vt=0, vp=0, ks=1.0, vs=1.0, q=0x50000, qs=(2048, 256), o=0x60000, os=(2048, 256), lse=0x7000,
        ws=0x80000):
    k = cache(row=ROW) if k is None else k
    return lib.kv_attention_q4(d or desc(), b or batch(), k, kt, kp, k if v is None else v, vt, vp, ks, vs, q, *qs, o, *os, lse, ws, 1 << 40, None)


def test_arguments(lib):
    assert run(lib, b=batch(n_reqs=0, tokens=0, table=None, offsets=None, lens=None)) == OK
    assert run(lib, b=batch(tokens=0), q=None) == OK
    for bad in (desc(dtype=2), desc(heads=0), desc(heads=7), desc(kv_heads=0), desc(dk=0), desc(dv=-32), desc(window=-1), desc(scale=0.0), desc(scale=-1.0),
                desc(scale=float("nan")), desc(scale=float("inf"))):
        assert run(lib, d=bad) == ARG
    for bad in (0.0, -1.0, float("nan"), float("inf"), 1e-35):
        assert run(lib, ks=bad) == ARG and run(lib, vs=bad) == ARG
    assert run(lib, d=desc(dk=112)) == ALIGN and run(lib, d=desc(dv=48)) == ALIGN
    assert run(lib, d=desc(dk=160), k=cache(row=192)) == UNSUPPORTED and run(lib, d=desc(dv=160), v=cache(row=192)) == UNSUPPORTED
    assert run(lib, d=desc(window=5, causal=0)) == UNSUPPORTED and run(lib, d=desc(heads=258)) == UNSUPPORTED
    assert run(lib, k=cache(row=512)) == ARG and run(lib, v=cache(row=160)) == ARG  # rows of another width
    assert run(lib, kt=1) == ARG and run(lib, kp=1) == ARG and run(lib, vt=-1) == ARG and run(lib, vp=2) == ARG
    assert run(lib, v=cache(row=ROW, block_size=32)) == ARG and run(lib, k=cache(row=ROW, num_blocks=0)) == ARG
    assert run(lib, k=cache(row=ROW, base=0x10008)) == ALIGN and run(lib, k=cache(row=ROW, block_stride=1 << 41)) == UNSUPPORTED
    for bad in (batch(n_reqs=-1), batch(tokens=-1), batch(pages=-1), batch(table=None), batch(offsets=None), batch(lens=None), batch(stride=5)):
        assert run(lib, b=bad) == ARG
    assert run(lib, b=batch(tokens=1 << 30)) == UNSUPPORTED and run(lib, b=batch(pages=1 << 30)) == UNSUPPORTED
    assert run(lib, q=None) == ARG and run(lib, o=None) == ARG and run(lib, ws=None) == ARG
    assert run(lib, q=0x50008) == ALIGN and run(lib, qs=(2048, 250)) == ALIGN and run(lib, os=(2040, 256)) == ALIGN
    assert run(lib, lse=0x7002) == ALIGN and run(lib, ws=0x80004) == ALIGN
    assert run(lib, d=desc(scale=1e-30), ks=1e-9) == ARG  # the two together are no 32-bit number


def test_binding_refuses(lib):
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises((ValueError, RuntimeError)):
        K.kv_attention_q4(q, None, None, None, None, 0.1, kv_heads=2)
    with pytest.raises(ValueError):
        K.kv_attention_q4(q.float(), None, None, None, None, 0.1, kv_heads=2)
    with pytest.raises(ValueError, match="32-bit"):
        K._attn_desc(K.KV_BF16, 8, 2 ** 32 + 2, 128, 128, True, 0, 0.1)
    with pytest.raises(ValueError, match="32-bit"):
        K._attn_desc(K.KV_BF16, 8, 2, 128, 2 ** 32 + 64, True, 0, 0.1)
