"""Batches and 64-bit references for the attention tests.

The references are plain loops over requests in float64 on the CPU; they share nothing with the kernels.
"""
from __future__ import annotations

import math

import torch

from paged_kv_cache_81_gb300 import pagedkv as K

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # half a step, relative
NAN = float("nan")


class Batch:
    """A ragged batch over a scattered page pool.  Slots that no token uses hold NaN."""

    def __init__(self, q_lens, kv_lens, heads, kv_heads, dk, dv=None, *, block=16, layout="separate", dtype=torch.bfloat16, seed=0,
                 spare_pages=3, device="cuda", spread=1.0):
        self.q_lens, self.kv_lens, self.heads, self.kv_heads, self.block, self.layout, self.dtype = \
            list(q_lens), list(kv_lens), heads, kv_heads, block, layout, dtype
        dv = dk if dv is None else dv
        self.dk, self.dv = dk, dv
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // block) for n in kv_lens]
        pages = sum(need) + spare_pages
        ids = torch.randperm(pages, generator=g)
        width = max([1] + need) + 1
        table = torch.full((len(kv_lens), width), -1, dtype=torch.int32)
        at = 0
        for r, n in enumerate(need):
            table[r, :n] = ids[at:at + n].to(torch.int32)
            at += n
        self.pages, self.table_cpu = pages, table
        total = sum(q_lens)
        self.q_cpu = (torch.randn(total, heads, dk, generator=g) * spread).to(dtype)
        self.k_rows = [torch.randn(n, kv_heads, dk, generator=g).to(dtype) for n in kv_lens]
        self.v_rows = [torch.randn(n, kv_heads, dv, generator=g).to(dtype) for n in kv_lens]
        k = torch.full((pages, block, kv_heads, dk), NAN, dtype=dtype)
        v = torch.full((pages, block, kv_heads, dv), NAN, dtype=dtype)
        for r, n in enumerate(kv_lens):
            for j in range(n):
                k[table[r, j // block], j % block] = self.k_rows[r][j]
                v[table[r, j // block], j % block] = self.v_rows[r][j]
        if layout == "separate":
            self.tensors = [k.to(device), v.to(device)]
            self.cache = K.PagedCache.from_tensors(self.tensors[:1], "separate")
            self.v_cache = K.PagedCache.from_tensors(self.tensors[1:], "separate")
        else:
            both = torch.stack([k, v], 1 if layout == "blocks_first" else 0)
            self.tensors = [both.to(device)]
            self.cache, self.v_cache = K.PagedCache.from_tensors(self.tensors, layout), None
        self.table = table.to(device)
        self.offsets = torch.tensor([sum(q_lens[:i]) for i in range(len(q_lens) + 1)], dtype=torch.int32, device=device)
        self.lens = torch.tensor(kv_lens, dtype=torch.int32, device=device)
        self.q = self.q_cpu.to(device)

    def run(self, scale, causal=True, window=0, **kw):
        return K.kv_attention(self.q, self.cache, self.table, self.offsets, self.lens, scale, v_cache=self.v_cache, causal=causal,
                              window=window, **kw)


def hidden(m, n, causal, window):
    """[m, n] of the keys that a token does not see; token i stands at n - m + i."""
    pos = n - m + torch.arange(m)[:, None]
    j = torch.arange(n)[None]
    h = torch.zeros(m, n, dtype=torch.bool)
    if causal:
        h |= j > pos
    if window:
        h |= j <= pos - window
    return h


def reference(q, k_rows, v_rows, q_lens, scale, causal=True, window=0):
    """(out, lse, out tolerance, lse tolerance) in float64 for rows of the given type.

    The kernel's weights are rounded to the element type (half a step u each, against a maximum that has a
    weight of at least 1, so 16-bit floats below 2^-14 lose at most 2^-25), the sum is rounded once more; products and
    sums are in 32 bits, of dk terms."""
    u = U[q.dtype]
    outs, lses, tol_o, tol_l = [], [], [], []
    first = 0
    for k, v, m in zip(k_rows, v_rows, q_lens):
        x = q[first:first + m].double()
        first += m
        n, kv_heads = k.shape[0], k.shape[1]
        group = x.shape[1] // kv_heads
        kd, vd = k.double().repeat_interleave(group, 1), v.double().repeat_interleave(group, 1)
        s = torch.einsum("mhd,nhd->hmn", x, kd) * scale
        size = torch.einsum("mhd,nhd->hmn", x.abs(), kd.abs()) * scale
        h = hidden(m, n, causal, window)
        s = s.masked_fill(h, -math.inf)
        lse = torch.logsumexp(s, -1) if n else torch.full((x.shape[1], m), -math.inf, dtype=torch.float64)
        p = torch.where(h, 0.0, torch.exp(s - lse[..., None]))
        p = torch.where(torch.isfinite(lse)[..., None], p, 0.0)
        o = torch.einsum("hmn,nhd->mhd", p, vd)
        mag = torch.einsum("hmn,nhd->mhd", p, vd.abs())
        big = size.masked_fill(h, 0.0).amax(-1) if n else torch.zeros_like(lse)  # [h, m]
        e32 = ((x.shape[2] + 16) * 2.0 ** -24 * (1 + big)).transpose(0, 1)[..., None]
        vmax = vd.abs().max() if n else torch.tensor(0.0)
        outs.append(o)
        lses.append(lse.transpose(0, 1))
        tol_o.append(u * (o.abs() + mag) * 1.01 + 2 * e32 * mag + n * 2.0 ** -25 * vmax)
        tol_l.append(e32[..., 0] + 2.0 ** -21 + 2.0 ** -22 * lse.transpose(0, 1).abs().nan_to_num(posinf=0.0))
    return torch.cat(outs), torch.cat(lses), torch.cat(tol_o), torch.cat(tol_l)


def close(got, want, tol, what):
    got = got.double().cpu()
    fine = torch.isfinite(want)
    assert torch.equal(fine, torch.isfinite(got)), f"{what}: finite values differ"
    assert torch.equal(got[~fine], want[~fine]), f"{what}: infinities differ"
    off = (got - want).abs()[fine] - tol[fine]
    assert off.numel() == 0 or float(off.max()) <= 0, f"{what}: over its tolerance by {float(off.max()):.3e}"


def check(batch, scale=None, causal=True, window=0, **kw):
    scale = batch.dk ** -0.5 if scale is None else scale
    K.kv_get_last_error(clear=True)
    out, lse = batch.run(scale, causal, window, **kw)
    torch.cuda.synchronize()
    assert K.kv_get_last_error(clear=True) == 0
    o, l, to, tl = reference(batch.q_cpu, batch.k_rows, batch.v_rows, batch.q_lens, scale, causal, window)
    close(out[:o.shape[0]], o, to, "out")
    close(lse[:o.shape[0]], l, tl, "lse")
    return out, lse
