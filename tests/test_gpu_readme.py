"""The examples of README.md, run one after another on small tensors."""
from __future__ import annotations

import os
import re

import pytest
import torch

from paged_kv_cache_81_gb300 import pagedkv as K

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_examples():
    with open(os.path.join(ROOT, "README.md")) as f:
        blocks = re.findall(r"```python\n(.*?)```", f.read(), re.S)
    assert blocks
    g = torch.Generator(device="cuda").manual_seed(1)
    heads, kv_heads, lens, new = 8, 2, [40, 25], [3, 1]
    n_pages, n_reqs, tokens = 12, len(lens), sum(new)
    pages = torch.randn(n_pages, 2, 16, kv_heads, 128, generator=g, device="cuda", dtype=torch.bfloat16)
    row = torch.randn(tokens, heads + 2 * kv_heads, 128, generator=g, device="cuda", dtype=torch.bfloat16)
    q, k, v = row[:, :heads], row[:, heads:heads + kv_heads], row[:, heads + kv_heads:]
    table = torch.full((n_reqs, 128), -1, dtype=torch.int32)
    table[0, :3], table[1, :2] = torch.tensor([7, 2, 9]), torch.tensor([4, 11])

    def ints(*x):
        return torch.tensor(x, dtype=torch.int32, device="cuda")
    env = dict(torch=torch, pages=pages, n_reqs=n_reqs, n_pages=n_pages, kv_heads=kv_heads, q=q, k=k, v=v, block_table=table.cuda(),
               q_offsets=ints(0, 3, 4), kv_lens=ints(*lens), token_req=ints(0, 0, 0, 1), token_pos=ints(37, 38, 39, 24))
    given = row.clone()
    K.kv_get_last_error(clear=True)
    for block in blocks:
        # what the example over 4 bits reads before the new tokens: any bytes but scales of NaN
        exec(block.replace("torch.empty(", "torch.zeros("), env)
    assert K.kv_get_last_error(clear=True) == 0 and torch.equal(row, given)
    turned = K.kv_rotate(q, env["token_pos"], env["rope"])
    want, lse = K.kv_attention_q4(turned, env["cache4"], env["block_table"], env["q_offsets"], env["kv_lens"], 128 ** -0.5, kv_heads=kv_heads)
    assert torch.equal(env["out"], want) and torch.equal(env["lse"], lse)
