"""Batches over a 4-bit cache and their 64-bit references, in plain steps on the CPU."""
from __future__ import annotations

import math

import torch

from paged_kv_cache_81_gb300 import pagedkv as K
from tests.attention_support import close, hidden
from tests.rotate_support import U, VALUES, packed, plane, q4_pages


class Q4Batch:
    """A ragged batch over a scattered pool of 4-bit pages.  Slots that no token uses hold scales of NaN."""

    def __init__(self, q_lens, kv_lens, heads, kv_heads, dk, dv=None, *, block=16, layout="separate", dtype=torch.bfloat16, seed=0, spare_pages=3,
                 spread=1.0, k_scale=1.0, v_scale=1.0):
        dv = dk if dv is None else dv
        self.q_lens, self.kv_lens, self.heads, self.kv_heads, self.dk, self.dv, self.block, self.layout, self.dtype = \
            list(q_lens), list(kv_lens), heads, kv_heads, dk, dv, block, layout, dtype
        self.k_scale, self.v_scale = k_scale, v_scale
        g = torch.Generator().manual_seed(seed)
        need = [-(-n // block) for n in kv_lens]
        self.pages = sum(need) + spare_pages
        ids = torch.randperm(self.pages, generator=g)
        self.table_cpu = torch.full((len(kv_lens), max([1] + need) + 1), -1, dtype=torch.int32)
        at = 0
        for r, n in enumerate(need):
            self.table_cpu[r, :n] = ids[at:at + n].to(torch.int32)
            at += n
        self.tensors, self.cache, self.v_cache = q4_pages(layout, self.pages, block, kv_heads, dk, dv, fill=0xFF)
        self.q_cpu = (torch.randn(sum(q_lens), heads, dk, generator=g) * spread).to(dtype)
        self.rows = []  # keys and values of every request in float64
        for which, (d, scale) in enumerate(((dk, k_scale), (dv, v_scale))):
            pages, held = plane(self.tensors, layout, which).cpu(), []
            for r, n in enumerate(kv_lens):
                code = torch.randint(0, 16, (n, kv_heads, d), generator=g)
                unit = (torch.rand(n, kv_heads, d // 16, generator=g) * 0.35 + 0.15).to(torch.float8_e4m3fn)
                held.append(VALUES[code] * unit.double().repeat_interleave(16, -1) * float(torch.tensor(scale, dtype=torch.float32)))
                j = torch.arange(n)
                pages[self.table_cpu[r, j // block].long(), j % block] = packed(code, unit.view(torch.uint8))
            plane(self.tensors, layout, which).copy_(pages)
            self.rows.append(held)
        self.q, self.table = self.q_cpu.cuda(), self.table_cpu.cuda()
        self.offsets = torch.tensor([sum(q_lens[:i]) for i in range(len(q_lens) + 1)], dtype=torch.int32, device="cuda")
        self.lens = torch.tensor(kv_lens, dtype=torch.int32, device="cuda")

    def run(self, scale, causal=True, window=0, **kw):
        return K.kv_attention_q4(self.q, self.cache, self.table, self.offsets, self.lens, scale, kv_heads=self.kv_heads, head_dim_v=self.dv,
                                 v_cache=self.v_cache, k_scale=self.k_scale, v_scale=self.v_scale, causal=causal, window=window, **kw)


def reference(q, k_rows, v_rows, q_lens, scale, causal=True, window=0):
    """(out, lse, out tolerance, lse tolerance) in float64.

    The rounding of the output to its type is u of its value.  Weights are rounded to fp16 (u_w; below 2^-25 of the
    largest they may be lost), the queries to 2^-25 of the row's largest; products and sums are in 32 bits, of dk terms."""
    u = U[q.dtype]
    outs, lses, tol_o, tol_l = [], [], [], []
    first = 0
    kv_heads = k_rows[0].shape[1]
    group = q.shape[1] // kv_heads
    u_w = 2.0 ** -11
    for k, v, m in zip(k_rows, v_rows, q_lens):
        x = q[first:first + m].double()
        first += m
        n = k.shape[0]
        kd, vd = k.repeat_interleave(group, 1), v.repeat_interleave(group, 1)
        s = torch.einsum("mhd,nhd->hmn", x, kd) * scale
        h = hidden(m, n, causal, window)
        size = (torch.einsum("mhd,nhd->hmn", x.abs(), kd.abs()) * scale).masked_fill(h, 0.0)
        rest = (torch.einsum("mh,nh->hmn", x.abs().amax(-1), kd.abs().sum(-1)) * scale).masked_fill(h, 0.0)
        s = s.masked_fill(h, -math.inf)
        lse = torch.logsumexp(s, -1) if n else torch.full((x.shape[1], m), -math.inf, dtype=torch.float64)
        p = torch.where(h, 0.0, torch.exp(s - lse[..., None]))
        p = torch.where(torch.isfinite(lse)[..., None], p, 0.0)
        o = torch.einsum("hmn,nhd->mhd", p, vd)
        mag = torch.einsum("hmn,nhd->mhd", p, vd.abs())
        big, off = (z.amax(-1) if n else torch.zeros_like(lse) for z in (size, rest))
        e32 = ((x.shape[2] + 16) * 2.0 ** -24 * (1 + big) + 2.0 ** -25 * off).transpose(0, 1)[..., None]
        vmax = vd.abs().max() if n else torch.tensor(0.0)
        outs.append(o)
        lses.append(lse.transpose(0, 1))
        tol_o.append(u * o.abs() * 1.01 + u_w * mag * 1.01 + 2 * e32 * mag + n * 2.0 ** -25 * vmax)
        tol_l.append(e32[..., 0] + 2.0 ** -21 + 2.0 ** -22 * lse.transpose(0, 1).abs().nan_to_num(posinf=0.0))
    return torch.cat(outs), torch.cat(lses), torch.cat(tol_o), torch.cat(tol_l)


def check(b, scale=None, causal=True, window=0, **kw):
    scale = b.dk ** -0.5 if scale is None else scale
    K.kv_get_last_error(clear=True)
    out, lse = b.run(scale, causal, window, **kw)
    torch.cuda.synchronize()
    assert K.kv_get_last_error(clear=True) == 0
    o, l, to, tl = reference(b.q_cpu, *b.rows, b.q_lens, scale, causal, window)
    close(out[:o.shape[0]], o, to, "out")
    close(lse[:o.shape[0]], l, tl, "lse")
    return out, lse
