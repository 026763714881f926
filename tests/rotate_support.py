"""64-bit references of rotary positions and of rows held in 4 bits, in plain steps on the CPU; they share nothing with the kernels."""
from __future__ import annotations

import math

import torch

from paged_kv_cache_81_gb300 import pagedkv as K

U = {torch.bfloat16: 2.0 ** -8, torch.float16: 2.0 ** -11}  # half a step, relative
GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
VALUES = torch.tensor(GRID + [-x for x in GRID], dtype=torch.float64)


def angles(turns, pos):
    """[tokens, pairs] in float64: whole turns taken off in whole numbers."""
    return torch.tensor([[2 * math.pi * ((int(p) * int(t)) % 2 ** 64) / 2.0 ** 64 for t in turns.tolist()] for p in pos.tolist()],
                        dtype=torch.float64).reshape(len(pos), len(turns))


def pairs(rot, offset, interleaved):
    half = rot // 2
    return [(offset + 2 * i, offset + 2 * i + 1) if interleaved else (offset + i, offset + i + half) for i in range(half)]


def rotated(x, turns, pos, offset=0, interleaved=False, magnitude=1.0, inverse=False):
    """(x rotated, the sizes that its rounding errors go by) in float64."""
    t = angles(turns, pos)
    x = x.double()
    out, size = x.clone(), torch.zeros_like(x)
    m = float(torch.tensor(magnitude, dtype=torch.float32))
    for i, (a, b) in enumerate(pairs(2 * len(turns), offset, interleaved)):
        c, s = m * torch.cos(t[:, i])[:, None], m * torch.sin(t[:, i])[:, None] * (-1 if inverse else 1)
        out[..., a], out[..., b] = x[..., a] * c - x[..., b] * s, x[..., a] * s + x[..., b] * c
        size[..., a] = size[..., b] = m * (x[..., a].abs() + x[..., b].abs())
    return out, size


def tolerance(want, size, dtype):
    """The rounding to the element type (fp16: at least half a step of its smallest numbers), and in 32 bits: each of cosine and
    sine off by half a step (relative), the products and the sum rounded: three halves of a step of the sizes."""
    return want.abs() * U[dtype] * (1 + 2.0 ** -12) + 4 * 2.0 ** -24 * size + (2.0 ** -25 if dtype == torch.float16 else 2.0 ** -134)


def quantised(x, scale):
    """(codes [..., dim], scale bytes [..., dim / 16]) of rows in the element type, from the definition."""
    inv = (torch.tensor(1.0, dtype=torch.float64) / torch.tensor(scale, dtype=torch.float32).double()).float()
    y = (x.float() * inv).double().reshape(*x.shape[:-1], -1, 16)
    most = (y.abs().amax(-1).float() / torch.tensor(6.0)).double()
    # the positive e4m3 numbers in order: byte b stands for e4m3[b]
    e4m3 = torch.arange(1, 127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    near = (most[..., None] - e4m3).abs()
    best = near.amin(-1, keepdim=True)
    # ties go to the even byte
    tied = near == best
    byte = torch.arange(1, 127)
    key = torch.where(tied, (byte % 2) * 1000 + byte, 10 ** 6)
    b = byte[key.argmin(-1)]
    unit = e4m3[b - 1]
    z = y.abs() / unit[..., None]
    grid = torch.tensor(GRID, dtype=torch.float64)
    near = (z[..., None] - grid).abs()
    tied = near == near.amin(-1, keepdim=True)
    code = torch.arange(8)
    code = torch.where(tied, (code % 2) * 100 + code, 10 ** 6).argmin(-1)
    code = torch.where(torch.isinf(z), 7, code)
    code = code + 8 * torch.signbit(y).long()
    return code.reshape(x.shape), b


def held(code, b, scale, dtype):
    """The values that codes and scale bytes stand for, in the element type."""
    unit = b.to(torch.uint8).view(torch.float8_e4m3fn).double().repeat_interleave(16, -1)
    s = torch.tensor(scale, dtype=torch.float32)
    return ((VALUES[code] * unit).float() * s).to(dtype)


def packed(code, b):
    """Rows [tokens, row bytes] as the cache holds them, the bytes that fill it up zero."""
    t, h, d = code.shape
    rows = torch.zeros(t, K.kv_q4_row_bytes(h, d), dtype=torch.uint8)
    flat = code.reshape(t, h * d)
    rows[:, :h * d // 2] = (flat[:, 0::2] | flat[:, 1::2] << 4).to(torch.uint8)
    rows[:, h * d // 2:h * d // 2 + h * d // 16] = b.reshape(t, h * d // 16).to(torch.uint8)
    return rows


def q4_pages(layout, pages, block, heads, dk, dv, tensors=1, fill=0x77, device="cuda"):
    """Tensors of a 4-bit cache filled with a byte, and its one or two descriptions (keys, values)."""
    def make(*shape):
        return torch.full(shape, fill, dtype=torch.uint8, device=device)
    rk, rv = K.kv_q4_row_bytes(heads, dk), K.kv_q4_row_bytes(heads, dv)
    if layout == "separate":
        t = [make(pages, block, rk), make(pages, block, rv)]
        return t, K.PagedCache.from_tensors(t[:1], "separate"), K.PagedCache.from_tensors(t[1:], "separate")
    assert rk == rv
    t = [make(pages, 2, block, rk) if layout == "blocks_first" else make(2, pages, block, rk) for _ in range(tensors)]
    return t, K.PagedCache.from_tensors(t, layout), None


def plane(t, layout, which):
    """[pages, block, ...row] of keys (0) or values (1)."""
    if layout == "separate":
        return t[which]
    return t[0][:, which] if layout == "blocks_first" else t[0][which]
