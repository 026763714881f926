"""What the attention entry points refuse before they touch the GPU (the C ABI, no GPU needed)."""
from __future__ import annotations

import ctypes

import pytest
import torch

from paged_kv_cache_81_gb300 import build
from paged_kv_cache_81_gb300 import pagedkv as K

OK, ARG, ALIGN, RANGE, UNSUPPORTED = K.KV_OK, K.KV_ERR_INVALID_ARG, K.KV_ERR_ALIGN, K.KV_ERR_RANGE, K.KV_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build.build()
    return K.load()


def cache(row=512, planes=1, tensors=1, base=0x10000, **kw):
    d = dict(block_size=16, num_blocks=100, block_stride=16 * row * planes, plane_stride=16 * row, token_stride=row)
    d.update(kw)
    arr = (ctypes.c_uint64 * max(1, tensors))(*[base + i * 0x100000 for i in range(tensors)])
    desc = K.KvCacheDesc(tensors, d["block_size"], planes, row, d["num_blocks"], d["block_stride"], d["plane_stride"], d["token_stride"],
                         ctypes.cast(arr, ctypes.POINTER(ctypes.c_uint64)))
    desc._keep = arr
    return desc


def batch(n_reqs=2, pages=8, stride=None, tokens=4, table=0x2000, offsets=0x3000, lens=0x4000):
    return K.KvAttnBatch(table, n_reqs, pages, pages if stride is None else stride, offsets, lens, tokens)


def desc(dtype=K.KV_BF16, heads=8, kv_heads=2, dk=128, dv=128, causal=1, window=0, scale=0.1):
    return K.KvAttnDesc(dtype, heads, kv_heads, dk, dv, causal, window, scale)


def attention(lib, d=None, b=None, k=None, v=None, kt=0, kp=0, vt=0, vp=0, q=0x50000, qs=(2048, 256), o=0x60000, os=(2048, 256), lse=0x7000, ws=0x80000,
              nbytes=1 << 40):
    k = cache() if k is None else k
    return lib.kv_attention(d or desc(), b or batch(), k, kt, kp, k if v is None else v, vt, vp, q, *qs, o, *os, lse, ws, nbytes, None)


def test_attention_arguments(lib):
    none = batch(n_reqs=0, tokens=0, table=None, offsets=None, lens=None)
    assert attention(lib, b=none) == OK  # no requests: nothing is looked at
    assert attention(lib, b=batch(tokens=0), q=None) == OK
    for bad in (desc(dtype=2), desc(heads=0), desc(heads=7), desc(kv_heads=0), desc(dk=0), desc(dv=-8), desc(window=-1), desc(scale=0.0),
                desc(scale=-1.0), desc(scale=float("nan")), desc(scale=float("inf")), desc(scale=1e-35), desc(scale=1e35)):
        assert attention(lib, d=bad) == ARG
    assert attention(lib, d=desc(dk=100)) == ALIGN  # heads of 200 bytes
    assert attention(lib, d=desc(dk=200)) == UNSUPPORTED and attention(lib, d=desc(dv=136)) == UNSUPPORTED
    assert attention(lib, d=desc(window=5, causal=0)) == UNSUPPORTED
    assert attention(lib, d=desc(heads=258), k=cache()) == UNSUPPORTED  # 129 query heads a key head
    assert attention(lib, k=cache(row=256)) == ARG  # rows of another width
    assert attention(lib, kt=1) == ARG and attention(lib, kp=1) == ARG and attention(lib, vt=-1) == ARG
    assert attention(lib, v=cache(block_size=32)) == ARG  # one table, two page sizes
    assert attention(lib, k=cache(num_blocks=0)) == ARG
    assert attention(lib, k=cache(base=0x10008)) == ALIGN
    assert attention(lib, k=cache(block_stride=1 << 41)) == UNSUPPORTED
    for bad in (batch(n_reqs=-1), batch(tokens=-1), batch(pages=-1), batch(table=None), batch(offsets=None), batch(lens=None), batch(stride=5)):
        assert attention(lib, b=bad) == ARG
    assert attention(lib, b=batch(tokens=1 << 30)) == UNSUPPORTED
    assert attention(lib, b=batch(pages=1 << 30)) == UNSUPPORTED
    assert attention(lib, b=batch(pages=1 << 25, tokens=1 << 26)) == UNSUPPORTED  # more steps than 32 bits count
    assert attention(lib, q=None) == ARG and attention(lib, o=None) == ARG and attention(lib, ws=None) == ARG
    assert attention(lib, q=0x50008) == ALIGN and attention(lib, qs=(2048, 250)) == ALIGN and attention(lib, os=(2040, 256)) == ALIGN
    assert attention(lib, lse=0x7002) == ALIGN and attention(lib, ws=0x80004) == ALIGN
    assert lib.kv_attention(None, batch(), cache(), 0, 0, cache(), 0, 0, 0x1000, 16, 16, 0x1000, 16, 16, None, 0x1000, 1, None) == ARG
    assert lib.kv_attention_workspace_bytes(None) == ARG and lib.kv_attention_mass_workspace_bytes(None) == ARG


def test_latent_arguments(lib):
    def run(d=None, c=None, b=None, q=0x50000):
        return lib.kv_latent_attention(d or desc(heads=16, kv_heads=1, dk=576, dv=512), b or batch(), c or cache(row=1152), 0, q, 16 * 1152, 1152,
                                       0x60000, 16 * 1024, 1024, None, 0x80000, 1 << 40, None)
    assert run(b=batch(tokens=0)) == OK
    assert run(d=desc(heads=16, kv_heads=2, dk=576, dv=512)) == ARG
    assert run(d=desc(heads=16, kv_heads=1, dk=512, dv=512)) == UNSUPPORTED
    assert run(d=desc(heads=16, kv_heads=1, dk=576, dv=512, causal=0, window=3)) == UNSUPPORTED
    assert run(c=cache(row=1024)) == ARG and run(q=None) == ARG and run(q=0x50004) == ALIGN


def test_expand_arguments(lib):
    def run(dtype=K.KV_BF16, heads=4, n=2, w=0x90000, src=None, k=None, v=None, table=0x2000, out=0x3000, lens=0x4000, pages=8, stride=8):
        return lib.kv_latent_expand(dtype, heads, src or cache(row=1152), 0, table, n, pages, stride, lens, w, k or cache(row=heads * 384), 0,
                                    v or cache(row=heads * 256), 0, out, 8, 8, None)
    assert run(n=0) == OK and run(pages=0, table=None) == OK
    assert run(dtype=5) == ARG and run(heads=0) == ARG and run(n=-1) == ARG and run(w=None) == ARG and run(table=None) == ARG
    assert run(out=None) == ARG and run(lens=None) == ARG and run(stride=3) == ARG
    assert run(w=0x90008) == ALIGN
    assert run(src=cache(row=1024)) == ARG and run(k=cache(row=1024)) == ARG and run(v=cache(row=4 * 256, block_size=32)) == ARG
    assert run(pages=1 << 30, stride=1 << 30) == UNSUPPORTED


def test_mass_arguments(lib):
    def run(d=None, b=None, q=0x50000, lse=0x7000, prev=None, ps=100, score=0x9000, ss=100, width=100, ws=0x80000):
        return lib.kv_attention_mass(d or desc(), b or batch(), cache(), 0, 0, q, 2048, 256, lse, prev, ps, score, ss, width, ws, 1 << 40, None)
    assert run(b=batch(n_reqs=0)) == OK and run(width=0) == OK
    assert run(width=-1) == ARG and run(lse=None) == ARG and run(score=None) == ARG and run(ws=None) == ARG and run(ss=99) == ARG
    assert run(prev=0x9000, ps=50) == ARG
    assert run(lse=0x7001) == ALIGN and run(prev=0x9001) == ALIGN and run(score=0x9002) == ALIGN and run(q=0x50002) == ALIGN
    assert run(d=desc(heads=258)) == UNSUPPORTED and run(d=desc(dk=200)) == UNSUPPORTED and run(d=desc(window=4, causal=0)) == UNSUPPORTED
    assert run(d=desc(scale=0.0)) == ARG


def test_evict_arguments(lib):
    def run(c=None, n=2, lens=0x4000, score=0x9000, ss=300, width=300, budget=100, sinks=4, recent=20, table=0x2000, out=0x3000, new=0x5000, kept=0x6000,
            ks=100, osc=0x7000, os=100, stride=8):
        return lib.kv_evict(c or cache(), table, n, 8, stride, lens, score, ss, width, budget, sinks, recent, out, 8, 8, new, kept, ks, osc, os, None)
    assert run(n=0) == OK
    for bad in (dict(sinks=90), dict(sinks=-1), dict(recent=-1), dict(budget=-1), dict(width=-1), dict(lens=None), dict(new=None), dict(kept=None),
                dict(score=None), dict(table=None), dict(out=None), dict(ss=10), dict(ks=10), dict(os=10), dict(stride=7), dict(n=-2)):
        assert run(**bad) == ARG, bad
    assert run(score=0x9002) == ALIGN and run(c=cache(token_stride=500)) == ALIGN
    assert run(n=70000) == UNSUPPORTED


def test_binding_refuses_what_is_not_on_the_gpu():
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    with pytest.raises((ValueError, RuntimeError)):
        K.kv_attention(q, None, None, None, None, 0.1)
    with pytest.raises(ValueError):
        K.kv_attention(q.float(), None, None, None, None, 0.1)
    with pytest.raises(ValueError):
        K.kv_latent_attention(q[0], None, None, None, None, 0.1)


def test_binding_refuses_numbers_past_32_bits():
    """They would reach the library cut off: a window of 2^32 + 5 as one of 5."""
    assert K._attn_desc(K.KV_BF16, 8, 2, 128, 128, True, 2 ** 31 - 1, 0.1).window == 2 ** 31 - 1
    for window in (2 ** 31, 2 ** 32 + 5, -2 ** 32):
        with pytest.raises(ValueError):
            K._attn_desc(K.KV_BF16, 8, 2, 128, 128, True, window, 0.1)
    lens = torch.zeros(1, dtype=torch.int32)
    for kw in (dict(budget=2 ** 32 + 4), dict(budget=8, sinks=2 ** 32), dict(budget=8, recent=-2 ** 32)):
        with pytest.raises(ValueError, match="32-bit"):
            K.kv_evict(None, None, lens, None, **kw)


def test_lengths_past_what_is_counted(lib):
    """Columns are counted in 32 bits, in steps of a thousand."""
    big = (1 << 30) + 1
    assert lib.kv_attention_mass(desc(), batch(), cache(), 0, 0, 0x50000, 2048, 256, 0x7000, None, 0, 0x9000, big, big, 0x80000, 1 << 40, None) == UNSUPPORTED
    assert lib.kv_evict(cache(), 0x2000, 2, 8, 8, 0x4000, 0x9000, 300, 300, big, 4, 20, 0x3000, 8, 8, 0x5000, 0x6000, big, 0x7000, big, None) == UNSUPPORTED
    # a product of requests, heads and tiles that would pass 64 bits
    wide, n = 1 << 22, (1 << 31) - 1
    assert lib.kv_latent_expand(K.KV_BF16, wide, cache(row=1152), 0, 0x2000, n, 1 << 20, 1 << 20, 0x4000, 0x90000, cache(row=wide * 384), 0,
                                cache(row=wide * 256), 0, 0x3000, 1 << 20, 1 << 20, None) == UNSUPPORTED
    rows = cache(row=wide * 256)
    assert attention(lib, d=desc(heads=wide, kv_heads=wide), b=batch(n_reqs=n, pages=1 << 20), k=rows) == UNSUPPORTED


def test_binding_refuses_tensor_numbers_past_32_bits():
    """Tensor 2^32 of a cache would be taken for its first."""
    q = torch.zeros(2, 4, 64, dtype=torch.bfloat16)
    for number in (2 ** 31, 2 ** 32, -2 ** 32 + 1):
        for call in (lambda: K.kv_attention(q, None, None, None, None, 0.1, k_tensor=number),
                     lambda: K.kv_attention(q, None, None, None, None, 0.1, v_tensor=number),
                     lambda: K.kv_latent_attention(q, None, None, None, None, 0.1, tensor=number),
                     lambda: K.kv_latent_expand(None, None, None, q, None, None, None, tensor=number),
                     lambda: K.kv_latent_expand(None, None, None, q, None, None, None, k_tensor=number),
                     lambda: K.kv_latent_expand(None, None, None, q, None, None, None, v_tensor=number),
                     lambda: K.kv_attention_mass(q, None, None, None, None, None, 0.1, k_tensor=number)):
            with pytest.raises(ValueError, match="32-bit"):
                call()


def test_binding_refuses_columns_past_32_bits():
    table, score = (torch.empty(1, 2 ** 32 + 5, dtype=t, device="meta") for t in (torch.int32, torch.float32))
    with pytest.raises(ValueError, match="32-bit"):
        K._table(-1, table, 1, "block_table")
    with pytest.raises(ValueError, match="32-bit"):
        K._score_rows(-1, score, 1, 0, "score")
    assert K._score_rows(-1, score[:, :7], 1, 5, "score")[1] == 2 ** 32 + 5


def test_token_counts_whose_product_with_the_heads_passes_64_bits(lib):
    """2^60 tokens of 16 heads would be taken for none."""
    for tokens in (1 << 60, (1 << 61) + 1, (1 << 63) - 1):
        assert attention(lib, d=desc(heads=16, kv_heads=2), b=batch(tokens=tokens)) == UNSUPPORTED
        assert lib.kv_attention_mass(desc(heads=16), batch(tokens=tokens), cache(), 0, 0, 0x50000, 2048, 256, 0x7000, None, 0, 0x9000, 100, 100, 0x80000,
                                     1 << 40, None) == UNSUPPORTED
