"""After a wait that ran out: the workspaces that the binding keeps are not used again."""
from __future__ import annotations

from types import SimpleNamespace

import pytest
import torch

from paged_kv_cache_81_gb300 import pagedkv as K
from tests.attention_support import Batch


def with_error_word(monkeypatch, bits):
    """The binding over a library whose error word reads `bits`; no GPU."""
    def kv_get_last_error(out, clear, stream):
        out._obj.value = bits
        return K.KV_OK

    monkeypatch.setattr(K, "_lib", SimpleNamespace(kv_get_last_error=kv_get_last_error))
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 0)
    f = K.kv_attention_workspace_bytes
    monkeypatch.setattr(K, "_workspaces", {(f, 0, 0): "a", (f, 0, 77): "b", (K.kv_attention_mass_workspace_bytes, 0, 0): "c", (f, 1, 0): "d"})
    return f


@pytest.mark.parametrize("clear", [False, True])
@pytest.mark.parametrize("bits", [K.KV_DERR_TIMEOUT, K.KV_DERR_TIMEOUT | K.KV_DERR_TABLE])
def test_a_timeout_gives_the_workspaces_up(monkeypatch, bits, clear):
    f = with_error_word(monkeypatch, bits)
    assert K.kv_get_last_error(clear=clear, stream=SimpleNamespace(cuda_stream=0)) == bits
    assert K._workspaces == {(f, 1, 0): "d"}  # another device's calls have not been asked about


def test_other_errors_keep_them(monkeypatch):
    with_error_word(monkeypatch, 0xff & ~K.KV_DERR_TIMEOUT)
    K.kv_get_last_error(stream=SimpleNamespace(cuda_stream=0))
    assert len(K._workspaces) == 4
    K.kv_reset_workspaces(1)
    assert len(K._workspaces) == 3
    K.kv_reset_workspaces()
    assert not K._workspaces


@pytest.mark.gpu
def test_calls_after_a_timeout_are_right():
    b = Batch([1, 200, 1, 7], [9000, 900, 3000, 5000], 8, 2, 128, seed=1)
    want = [x.clone() for x in b.run(0.1)]
    args = (b.q, b.cache, b.table, b.offsets, b.lens, want[1], 0.1)
    score = K.kv_attention_mass(*args)
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    b.run(0.1, stream=s)
    torch.cuda.synchronize()
    assert len(K._workspaces) >= 3
    for ws in K._workspaces.values():  # what a call that broke off would leave
        ws[: K.KV_ATTENTION_ZEROED_BYTES].view(torch.int32).fill_(1)
    K.kv_get_last_error(clear=True)
    K.kv_wait_signal(K.new_signal(), 1, 1000)  # nothing sets it
    assert K.kv_get_last_error(clear=True) == K.KV_DERR_TIMEOUT
    assert all(torch.equal(x, y) for x, y in zip(want, b.run(0.1)))
    assert torch.equal(score, K.kv_attention_mass(*args))
    got = b.run(0.1, stream=s)
    s.synchronize()
    assert all(torch.equal(x, y) for x, y in zip(want, got))
    assert K.kv_get_last_error(clear=True) == 0
