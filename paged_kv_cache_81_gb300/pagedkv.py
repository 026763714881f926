"""ctypes binding of libpagedkv.so (argument marshalling only).

Every function here has the name of the C entry point it calls, takes torch CUDA
tensors, passes their data pointers and the current CUDA stream, and raises
``KvError`` on a non-zero status.  No step of the data path runs in Python or on the
CPU: when the library is missing, the first call raises.
"""
from __future__ import annotations

import ctypes
import functools
import os
import threading
from contextlib import nullcontext as _no_context
from dataclasses import dataclass
from typing import Optional, Sequence

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.environ.get("PAGEDKV_LIB") or os.path.join(_HERE, "libpagedkv.so")

KV_OK, KV_ERR_INVALID_ARG, KV_ERR_ALIGN, KV_ERR_RANGE, KV_ERR_CUDA, KV_ERR_TIMEOUT, KV_ERR_UNSUPPORTED = range(7)
KV_DERR_TABLE, KV_DERR_SLOT, KV_DERR_BLOCK, KV_DERR_LIST = 0x01, 0x02, 0x04, 0x08
KV_DERR_CAPACITY, KV_DERR_STAGE, KV_DERR_DST_TABLE, KV_DERR_TIMEOUT = 0x10, 0x20, 0x40, 0x80

KV_BF16, KV_F16 = 0, 1
KV_ATTENTION_ZEROED_BYTES = 16384
_DTYPES = {torch.bfloat16: KV_BF16, torch.float16: KV_F16}

RUN_WORDS = 6  # a kv_xfer_run is 24 bytes: six int32 words (the last two hold the int64 stage_block)
EXPORTS = ("kv_version", "kv_status_string", "kv_last_cuda_error", "kv_slot_mapping", "kv_reshape_and_cache",
           "kv_xfer_workspace_bytes", "kv_build_xfer_list", "kv_pack_blocks", "kv_unpack_blocks",
           "kv_get_last_error", "kv_build_xfer_list_static", "kv_unpack_blocks_signal", "kv_wait_signal",
           "kv_clip_block_lists", "kv_block_hashes", "kv_block_hashes_workspace_bytes", "kv_write_tokens",
           "kv_attention", "kv_attention_workspace_bytes", "kv_latent_attention", "kv_latent_expand", "kv_attention_mass",
           "kv_attention_mass_workspace_bytes", "kv_evict", "kv_rope_frequencies", "kv_rotate", "kv_rotate_write",
           "kv_q4_row_bytes", "kv_rotate_write_q4", "kv_attention_q4")


class KvError(RuntimeError):
    def __init__(self, fn: str, status: int, detail: str = ""):
        self.status = status
        super().__init__(f"{fn} failed: {_status_name(status)}{(' ' + detail) if detail else ''}")


class KvCacheDesc(ctypes.Structure):
    _fields_ = [
        ("n_tensors", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("n_planes", ctypes.c_int32),
        ("row_bytes", ctypes.c_int32),
        ("num_blocks", ctypes.c_int64),
        ("block_stride", ctypes.c_int64),
        ("plane_stride", ctypes.c_int64),
        ("token_stride", ctypes.c_int64),
        ("base", ctypes.POINTER(ctypes.c_uint64)),
    ]


class KvStageDesc(ctypes.Structure):
    _fields_ = [
        ("n_blocks", ctypes.c_int64),
        ("n_tensors", ctypes.c_int32),
        ("n_planes", ctypes.c_int32),
        ("block_size", ctypes.c_int32),
        ("slice_bytes", ctypes.c_int32),
    ]


class KvAttnBatch(ctypes.Structure):
    _fields_ = [
        ("block_table", ctypes.c_void_p),
        ("n_reqs", ctypes.c_int32),
        ("max_blocks_per_req", ctypes.c_int32),
        ("bt_row_stride", ctypes.c_int64),
        ("q_offsets", ctypes.c_void_p),
        ("kv_lens", ctypes.c_void_p),
        ("n_tokens", ctypes.c_int64),
    ]


class KvAttnDesc(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int32),
        ("n_heads", ctypes.c_int32),
        ("n_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("head_dim_v", ctypes.c_int32),
        ("causal", ctypes.c_int32),
        ("window", ctypes.c_int32),
        ("scale", ctypes.c_float),
    ]


class KvRope(ctypes.Structure):
    _fields_ = [
        ("turns", ctypes.c_void_p),
        ("rot_dim", ctypes.c_int32),
        ("rot_offset", ctypes.c_int32),
        ("interleaved", ctypes.c_int32),
        ("magnitude", ctypes.c_float),
    ]


class KvRopeScaling(ctypes.Structure):
    _fields_ = [
        ("kind", ctypes.c_int32),
        ("factor", ctypes.c_double),
        ("original_length", ctypes.c_double),
        ("fast", ctypes.c_double),
        ("slow", ctypes.c_double),
    ]


class KvNewTokens(ctypes.Structure):
    _fields_ = [
        ("dtype", ctypes.c_int32),
        ("n_heads", ctypes.c_int32),
        ("n_kv_heads", ctypes.c_int32),
        ("head_dim", ctypes.c_int32),
        ("head_dim_v", ctypes.c_int32),
        ("q", ctypes.c_void_p),
        ("q_token_stride", ctypes.c_int64),
        ("q_head_stride", ctypes.c_int64),
        ("q_out", ctypes.c_void_p),
        ("q_out_token_stride", ctypes.c_int64),
        ("q_out_head_stride", ctypes.c_int64),
        ("k", ctypes.c_void_p),
        ("k_token_stride", ctypes.c_int64),
        ("k_head_stride", ctypes.c_int64),
        ("v", ctypes.c_void_p),
        ("v_token_stride", ctypes.c_int64),
        ("v_head_stride", ctypes.c_int64),
        ("token_req", ctypes.c_void_p),
        ("token_pos", ctypes.c_void_p),
        ("rope_pos", ctypes.c_void_p),
        ("n_tokens", ctypes.c_int64),
        ("block_table", ctypes.c_void_p),
        ("n_reqs", ctypes.c_int32),
        ("max_blocks_per_req", ctypes.c_int32),
        ("bt_row_stride", ctypes.c_int64),
    ]


_lock = threading.Lock()
_lib = None


def load(path: str = LIB_PATH) -> ctypes.CDLL:
    """Load and bind libpagedkv.so; raises if it has not been built."""
    global _lib
    with _lock:
        if _lib is not None:
            return _lib
        if not os.path.exists(path):
            raise RuntimeError(f"{path} is missing: build it with `python -c 'import __graft_entry__ as g; g.build()'`")
        lib = ctypes.CDLL(path)
        P, i32, i64 = ctypes.c_void_p, ctypes.c_int32, ctypes.c_int64
        D = ctypes.POINTER(KvCacheDesc)
        S = ctypes.POINTER(KvStageDesc)
        A, B = ctypes.POINTER(KvAttnDesc), ctypes.POINTER(KvAttnBatch)
        R, N = ctypes.POINTER(KvRope), ctypes.POINTER(KvNewTokens)
        f32 = ctypes.c_float
        sig = {
            "kv_version": ([], ctypes.c_char_p),
            "kv_status_string": ([ctypes.c_int], ctypes.c_char_p),
            "kv_last_cuda_error": ([], ctypes.c_int),
            "kv_slot_mapping": ([P, i32, i32, i64, P, P, i64, i32, P, P], ctypes.c_int),
            "kv_reshape_and_cache": ([D, P, i64, P, i64, P], ctypes.c_int),
            "kv_xfer_workspace_bytes": ([i64, ctypes.POINTER(i64)], ctypes.c_int),
            "kv_build_xfer_list": ([P, i32, P, P, i64, i32, P, i64, P, P, i64, P], ctypes.c_int),
            "kv_pack_blocks": ([D, i32, S, P, P, i64, i32, P, i64, P], ctypes.c_int),
            "kv_unpack_blocks": ([D, i32, S, P, P, i64, i32, P, i64, P, P, P, i32, P], ctypes.c_int),
            "kv_get_last_error": ([ctypes.POINTER(i32), i32, P], ctypes.c_int),
            "kv_build_xfer_list_static": ([P, i32, P, P, i64, i32, P, i64, P, P], ctypes.c_int),
            "kv_unpack_blocks_signal": ([D, i32, S, P, P, i64, i32, P, i64, P, P, P, i32, P, ctypes.c_uint64, P],
                                        ctypes.c_int),
            "kv_wait_signal": ([P, ctypes.c_uint64, ctypes.c_uint32, P, P], ctypes.c_int),
            "kv_clip_block_lists": ([P, i32, P, i64, P, i32, i32, P, P, i64, P], ctypes.c_int),
            "kv_block_hashes": ([P, i32, P, i64, i32, ctypes.c_uint64, P, P, i64, P, i64, P], ctypes.c_int),
            "kv_block_hashes_workspace_bytes": ([i64, i32, ctypes.POINTER(ctypes.c_int64)], ctypes.c_int),
            "kv_attention_workspace_bytes": ([ctypes.POINTER(i64)], ctypes.c_int),
            "kv_attention": ([A, B, D, i32, i32, D, i32, i32, P, i64, i64, P, i64, i64, P, P, i64, P], ctypes.c_int),
            "kv_latent_attention": ([A, B, D, i32, P, i64, i64, P, i64, i64, P, P, i64, P], ctypes.c_int),
            "kv_latent_expand": ([i32, i32, D, i32, P, i32, i32, i64, P, P, D, i32, D, i32, P, i32, i64, P], ctypes.c_int),
            "kv_attention_mass_workspace_bytes": ([ctypes.POINTER(i64)], ctypes.c_int),
            "kv_attention_mass": ([A, B, D, i32, i32, P, i64, i64, P, P, i64, P, i64, i32, P, i64, P], ctypes.c_int),
            "kv_evict": ([D, P, i32, i32, i64, P, P, i64, i32, i32, i32, i32, P, i32, i64, P, P, i64, P, i64, P],
                         ctypes.c_int),
            "kv_write_tokens": ([D, P, i64, P, i32, i32, i64, P, P, i64, P, P], ctypes.c_int),
            "kv_rope_frequencies": ([i32, ctypes.c_double, ctypes.POINTER(KvRopeScaling), P, ctypes.POINTER(f32)], ctypes.c_int),
            "kv_rotate": ([i32, i32, i32, P, i64, i64, P, i64, i64, i64, P, R, i32, P], ctypes.c_int),
            "kv_rotate_write": ([N, R, D, i32, i32, D, i32, i32, P], ctypes.c_int),
            "kv_q4_row_bytes": ([i32, i32, ctypes.POINTER(i32)], ctypes.c_int),
            "kv_rotate_write_q4": ([N, R, D, i32, i32, D, i32, i32, f32, f32, P, P, P], ctypes.c_int),
            "kv_attention_q4": ([A, B, D, i32, i32, D, i32, i32, f32, f32, P, i64, i64, P, i64, i64, P, P, i64, P], ctypes.c_int),
        }
        for name, (args, res) in sig.items():
            f = getattr(lib, name)
            f.argtypes, f.restype = args, res
        _lib = lib
        return lib


def _status_name(status: int) -> str:
    try:
        return load().kv_status_string(status).decode()
    except Exception:  # the library may be what is missing
        return f"status {status}"


def _check(fn: str, status: int):
    if status != KV_OK:
        detail = f"(cuda error {load().kv_last_cuda_error()})" if status == KV_ERR_CUDA else ""
        raise KvError(fn, status, detail)


def _stream(stream=None) -> ctypes.c_void_p:
    s = stream if stream is not None else torch.cuda.current_stream()
    return ctypes.c_void_p(s.cuda_stream)


def _ptr(t: Optional[torch.Tensor]) -> Optional[ctypes.c_void_p]:
    if t is None:
        return None
    if not t.is_cuda:
        raise ValueError("libpagedkv takes CUDA tensors")
    return ctypes.c_void_p(t.data_ptr())


def _stage_ptr(t: torch.Tensor) -> ctypes.c_void_p:
    """Staging may live in device memory or in pinned host memory (reached over the host link)."""
    if not (t.is_cuda or t.is_pinned()):
        raise ValueError("the staging buffer must be a CUDA tensor or pinned host memory")
    return ctypes.c_void_p(t.data_ptr())


def _i32(t: torch.Tensor, name: str) -> torch.Tensor:
    if t.dtype != torch.int32 or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 CUDA tensor")
    return t


def version() -> str:
    return load().kv_version().decode()


# ---------------------------------------------------------------------------
# cache geometry
# ---------------------------------------------------------------------------
@dataclass
class PagedCache:
    """A paged cache: equal-shaped device tensors plus their byte geometry (kv_cache_desc)."""

    tensors: list
    num_blocks: int
    block_size: int
    n_planes: int
    row_bytes: int
    block_stride: int
    plane_stride: int
    token_stride: int

    @classmethod
    def from_tensors(cls, tensors: Sequence[torch.Tensor], layout: str) -> "PagedCache":
        """layout: "separate" / "mla" ([num_blocks, bs, ...row]), "blocks_first"
        ([num_blocks, 2, bs, ...row]) or "kv_first" ([2, num_blocks, bs, ...row])."""
        tensors = list(tensors)
        t = tensors[0]
        e = t.element_size()
        st = [s * e for s in t.stride()]
        if layout in ("separate", "mla"):
            nb, bs, planes = t.shape[0], t.shape[1], 1
            block, plane, token, rest = st[0], st[0], st[1], t.shape[2:]
        elif layout == "blocks_first":
            nb, bs, planes = t.shape[0], t.shape[2], 2
            block, plane, token, rest = st[0], st[1], st[2], t.shape[3:]
            assert t.shape[1] == 2
        elif layout == "kv_first":
            nb, bs, planes = t.shape[1], t.shape[2], 2
            block, plane, token, rest = st[1], st[0], st[2], t.shape[3:]
            assert t.shape[0] == 2
        else:
            raise ValueError(layout)
        row = e
        for d in rest:
            row *= d
        for x in tensors:
            if x.shape != t.shape or x.stride() != t.stride() or x.dtype != t.dtype or not x.is_cuda:
                raise ValueError("cache tensors must share shape, strides and dtype and live on the GPU")
        return cls(tensors, int(nb), int(bs), planes, int(row), int(block), int(plane), int(token))

    def desc(self) -> KvCacheDesc:
        """The kv_cache_desc of these tensors, built once and rebuilt only if a tensor moved."""
        ptrs = [x.data_ptr() for x in self.tensors]
        if getattr(self, "_desc_ptrs", None) != ptrs:
            n = len(ptrs)
            self._bases = (ctypes.c_uint64 * max(1, n))(*ptrs)
            self._desc = KvCacheDesc(n, self.block_size, self.n_planes, self.row_bytes, self.num_blocks,
                                     self.block_stride, self.plane_stride, self.token_stride,
                                     ctypes.cast(self._bases, ctypes.POINTER(ctypes.c_uint64)))
            self._desc_ptrs = ptrs
        return self._desc


def stage_desc(n_blocks: int, n_tensors: int, n_planes: int, block_size: int, slice_bytes: int) -> KvStageDesc:
    return KvStageDesc(int(n_blocks), int(n_tensors), int(n_planes), int(block_size), int(slice_bytes))


def stage_nbytes(sd: KvStageDesc) -> int:
    return sd.n_blocks * sd.n_tensors * sd.n_planes * sd.block_size * sd.slice_bytes


# ---------------------------------------------------------------------------
# entry points
# ---------------------------------------------------------------------------
def kv_slot_mapping(block_table: torch.Tensor, token_req: torch.Tensor, token_pos: torch.Tensor, block_size: int,
                    slot_out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    _i32(token_req, "token_req"), _i32(token_pos, "token_pos")
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.stride(1) != 1:
        raise ValueError("block_table must be a row-major int32 [n_reqs, max_blocks] CUDA tensor")
    n = token_req.shape[0]
    if slot_out is None:
        slot_out = torch.empty(n, dtype=torch.int64, device=token_req.device)
    _check("kv_slot_mapping", load().kv_slot_mapping(
        _ptr(block_table), block_table.shape[0], block_table.shape[1], block_table.stride(0), _ptr(token_req),
        _ptr(token_pos), n, int(block_size), _ptr(slot_out), _stream(stream)))
    return slot_out


def kv_reshape_and_cache(cache: PagedCache, new_kv: Sequence[torch.Tensor], slot: torch.Tensor, stream=None):
    """new_kv: n_tensors * n_planes tensors [T, ...row] (tensor-major, plane-minor), equal strides."""
    if slot.dtype != torch.int64:
        raise ValueError("slot must be int64")
    new_kv = list(new_kv)
    stride = new_kv[0].stride(0) * new_kv[0].element_size() if new_kv else cache.row_bytes
    ptrs = (ctypes.c_uint64 * max(1, len(new_kv)))(*[x.data_ptr() for x in new_kv])
    d = cache.desc()
    _check("kv_reshape_and_cache", load().kv_reshape_and_cache(
        ctypes.byref(d), ctypes.cast(ptrs, ctypes.c_void_p), stride, _ptr(slot), slot.shape[0], _stream(stream)))


def kv_write_tokens(cache: PagedCache, new_kv: Sequence[torch.Tensor], block_table: torch.Tensor,
                    token_req: torch.Tensor, token_pos: torch.Tensor, slot_out: Optional[torch.Tensor] = None,
                    stream=None):
    """kv_slot_mapping + kv_reshape_and_cache in one call: the row copy looks each token's slot up in
    the block table (one launch per 128 tensors); slot_out (int64 [T]) optionally gets the slots."""
    _i32(token_req, "token_req"), _i32(token_pos, "token_pos")
    if block_table.dtype != torch.int32 or block_table.dim() != 2 or block_table.stride(1) != 1:
        raise ValueError("block_table must be a row-major int32 [n_reqs, max_blocks] CUDA tensor")
    new_kv = list(new_kv)
    stride = new_kv[0].stride(0) * new_kv[0].element_size() if new_kv else cache.row_bytes
    ptrs = (ctypes.c_uint64 * max(1, len(new_kv)))(*[x.data_ptr() for x in new_kv])
    _check("kv_write_tokens", load().kv_write_tokens(
        ctypes.byref(cache.desc()), ctypes.cast(ptrs, ctypes.c_void_p), stride, _ptr(block_table),
        block_table.shape[0], block_table.shape[1], block_table.stride(0), _ptr(token_req), _ptr(token_pos),
        token_req.shape[0], _ptr(slot_out), _stream(stream)))


def kv_xfer_workspace_bytes(n_blocks: int) -> int:
    out = ctypes.c_int64(0)
    _check("kv_xfer_workspace_bytes", load().kv_xfer_workspace_bytes(int(n_blocks), ctypes.byref(out)))
    return out.value


class XferList:
    """Device output of kv_build_xfer_list: run records [capacity, 6] int32 and the run count."""

    def __init__(self, capacity: int, device, max_run_blocks: int):
        self.capacity = int(capacity)
        self.max_run_blocks = int(max_run_blocks)
        self.runs = torch.empty((max(1, self.capacity), RUN_WORDS), dtype=torch.int32, device=device)
        self.n_runs = torch.zeros(1, dtype=torch.int32, device=device)
        self._ws = None
        self._ws_blocks = -1

    def workspace(self, n_blocks: int) -> torch.Tensor:
        """A builder workspace for lists of n_blocks entries, kept with this list for reuse."""
        if self._ws is None or self._ws_blocks < n_blocks:
            self._ws = torch.empty(kv_xfer_workspace_bytes(n_blocks), dtype=torch.uint8, device=self.runs.device)
            self._ws_blocks = n_blocks
        return self._ws

    def host(self) -> dict:
        """Copy the runs to the host as numpy columns (synchronises)."""
        n = min(int(self.n_runs.item()), self.capacity)
        r = self.runs[:n].cpu()
        return dict(req=r[:, 0].numpy(), src_block=r[:, 1].numpy(), dst_block=r[:, 2].numpy(),
                    n_blocks=r[:, 3].numpy(), stage_block=r[:, 4:6].contiguous().view(torch.int64)[:, 0].numpy(),
                    count=int(self.n_runs.item()))


def kv_build_xfer_list(req_offsets: torch.Tensor, src_ids: torch.Tensor, dst_ids: Optional[torch.Tensor] = None,
                       max_run_blocks: int = 0, out: Optional[XferList] = None,
                       workspace: Optional[torch.Tensor] = None, stream=None) -> XferList:
    _i32(req_offsets, "req_offsets"), _i32(src_ids, "src_ids")
    if dst_ids is not None:
        _i32(dst_ids, "dst_ids")
    n = src_ids.shape[0]
    if out is None:
        out = XferList(n, src_ids.device, max_run_blocks)
    if workspace is None:
        workspace = out.workspace(n)
    _check("kv_build_xfer_list", load().kv_build_xfer_list(
        _ptr(req_offsets), req_offsets.shape[0] - 1, _ptr(src_ids), _ptr(dst_ids), n, int(max_run_blocks),
        _ptr(out.runs), out.capacity, _ptr(out.n_runs), _ptr(workspace), workspace.numel(), _stream(stream)))
    out.max_run_blocks = int(max_run_blocks)
    return out


def kv_clip_block_lists(req_offsets: torch.Tensor, ids: torch.Tensor, n_tokens: torch.Tensor, window: int,
                        block_size: int, out_offsets: Optional[torch.Tensor] = None,
                        out_ids: Optional[torch.Tensor] = None, stream=None):
    """Sliding-window clip of per-request block lists; returns device (out_offsets, out_ids)
    where out_ids has room for every input entry and out_offsets[-1] is the kept count."""
    _i32(req_offsets, "req_offsets"), _i32(ids, "ids"), _i32(n_tokens, "n_tokens")
    if out_offsets is None:
        out_offsets = torch.empty_like(req_offsets)
    if out_ids is None:
        out_ids = torch.empty(max(1, ids.shape[0]), dtype=torch.int32, device=ids.device)
    _check("kv_clip_block_lists", load().kv_clip_block_lists(
        _ptr(req_offsets), req_offsets.shape[0] - 1, _ptr(ids), ids.shape[0], _ptr(n_tokens), int(window),
        int(block_size), _ptr(out_offsets), _ptr(out_ids), out_ids.shape[0], _stream(stream)))
    return out_offsets, out_ids


def kv_block_hashes_workspace_bytes(n_tokens: int, block_size: int) -> int:
    out = ctypes.c_int64(0)
    _check("kv_block_hashes_workspace_bytes", load().kv_block_hashes_workspace_bytes(int(n_tokens), int(block_size),
                                                                                     ctypes.byref(out)))
    return out.value


def kv_block_hashes(tok_offsets: torch.Tensor, tokens: torch.Tensor, block_size: int, seed: int,
                    out_offsets: Optional[torch.Tensor] = None, out_hashes: Optional[torch.Tensor] = None,
                    workspace="auto", stream=None):
    """Prefix hash chain of every request's full token blocks; returns device (out_offsets int32,
    out_hashes int64 holding the uint64 bit patterns).  workspace: "auto" (a uint8 device tensor
    of kv_block_hashes_workspace_bytes is allocated here, for the table path), None (the plain
    per-request chain) or a caller's uint8 tensor."""
    _i32(tok_offsets, "tok_offsets"), _i32(tokens, "tokens")
    cap = max(1, tokens.shape[0] // int(block_size))
    if out_offsets is None:
        out_offsets = torch.empty_like(tok_offsets)
    if out_hashes is None:
        out_hashes = torch.empty(cap, dtype=torch.int64, device=tokens.device)
    if isinstance(workspace, str):
        if workspace != "auto":
            raise ValueError(f"workspace must be 'auto', None or a tensor, not {workspace!r}")
        need = kv_block_hashes_workspace_bytes(tokens.shape[0], block_size)
        workspace = torch.empty(max(need, 16), dtype=torch.uint8, device=tokens.device)
    ws_ptr = _ptr(workspace) if workspace is not None else None
    ws_bytes = workspace.numel() * workspace.element_size() if workspace is not None else 0
    _check("kv_block_hashes", load().kv_block_hashes(
        _ptr(tok_offsets), tok_offsets.shape[0] - 1, _ptr(tokens), tokens.shape[0], int(block_size),
        int(seed) & 0xFFFFFFFFFFFFFFFF, _ptr(out_offsets), _ptr(out_hashes), out_hashes.shape[0], ws_ptr, ws_bytes,
        _stream(stream)))
    return out_offsets, out_hashes


KV_XFER_STATIC_MAX_BLOCKS = 4177920


def kv_build_xfer_list_static(req_offsets: torch.Tensor, src_ids: torch.Tensor,
                              dst_ids: Optional[torch.Tensor] = None, max_run_blocks: int = 0,
                              out: Optional[XferList] = None, stream=None) -> XferList:
    """kv_build_xfer_list without a workspace: the library's own fixed scratch array is used,
    so the call itself allocates nothing (the outputs are still the caller's)."""
    _i32(req_offsets, "req_offsets"), _i32(src_ids, "src_ids")
    if dst_ids is not None:
        _i32(dst_ids, "dst_ids")
    n = src_ids.shape[0]
    if out is None:
        out = XferList(n, src_ids.device, max_run_blocks)
    _check("kv_build_xfer_list_static", load().kv_build_xfer_list_static(
        _ptr(req_offsets), req_offsets.shape[0] - 1, _ptr(src_ids), _ptr(dst_ids), n, int(max_run_blocks),
        _ptr(out.runs), out.capacity, _ptr(out.n_runs), _stream(stream)))
    out.max_run_blocks = int(max_run_blocks)
    return out


def kv_pack_blocks(cache: PagedCache, xfer: XferList, n_blocks: int, stage: Optional[torch.Tensor] = None,
                   slice_off: int = 0, slice_bytes: Optional[int] = None, stream=None) -> torch.Tensor:
    sb = cache.row_bytes if slice_bytes is None else int(slice_bytes)
    sd = stage_desc(n_blocks, len(cache.tensors), cache.n_planes, cache.block_size, sb)
    if stage is None:
        stage = torch.empty(stage_nbytes(sd), dtype=torch.uint8, device=xfer.runs.device)
    d = cache.desc()
    _check("kv_pack_blocks", load().kv_pack_blocks(
        ctypes.byref(d), int(slice_off), ctypes.byref(sd), _ptr(xfer.runs), _ptr(xfer.n_runs), xfer.capacity,
        xfer.max_run_blocks, _stage_ptr(stage), stage.numel() * stage.element_size(), _stream(stream)))
    return stage


def kv_unpack_blocks(cache: PagedCache, stage: torch.Tensor, xfer: XferList, n_blocks: int, src_block_size: int,
                     slice_bytes: Optional[int] = None, dst_slice_off: int = 0,
                     src_req_offsets: Optional[torch.Tensor] = None, dst_req_offsets: Optional[torch.Tensor] = None,
                     dst_ids: Optional[torch.Tensor] = None, stream=None, signal: Optional[torch.Tensor] = None,
                     signal_add: int = 1):
    """Whole-block mode when dst_ids is None (runs carry destination ids), remap mode otherwise.
    With `signal` (see new_signal) the call is kv_unpack_blocks_signal: signal value += signal_add
    once every row has landed."""
    sb = cache.row_bytes if slice_bytes is None else int(slice_bytes)
    sd = stage_desc(n_blocks, len(cache.tensors), cache.n_planes, src_block_size, sb)
    n_reqs = 0 if dst_req_offsets is None else dst_req_offsets.shape[0] - 1
    d = cache.desc()
    args = [ctypes.byref(d), int(dst_slice_off), ctypes.byref(sd), _ptr(xfer.runs), _ptr(xfer.n_runs), xfer.capacity,
            xfer.max_run_blocks, _stage_ptr(stage), stage.numel() * stage.element_size(), _ptr(src_req_offsets),
            _ptr(dst_req_offsets), _ptr(dst_ids), n_reqs]
    if signal is None:
        _check("kv_unpack_blocks", load().kv_unpack_blocks(*args, _stream(stream)))
    else:
        _check("kv_unpack_blocks_signal", load().kv_unpack_blocks_signal(*args, _ptr(signal), int(signal_add),
                                                                         _stream(stream)))


def new_signal(device="cuda") -> torch.Tensor:
    """A zeroed kv_signal (16 bytes: value int64, arrived + reserved) in device memory."""
    return torch.zeros(2, dtype=torch.int64, device=device)


def signal_value(signal: torch.Tensor) -> int:
    return int(signal[0].item())


def kv_wait_signal(signal: torch.Tensor, expected: int, timeout_us: int, status: Optional[torch.Tensor] = None,
                   stream=None) -> torch.Tensor:
    """Queue a bounded device-side wait until signal value >= expected; returns the device status word."""
    if status is None:
        status = torch.full((1,), -1, dtype=torch.int32, device=signal.device)
    _check("kv_wait_signal", load().kv_wait_signal(_ptr(signal), int(expected), int(timeout_us), _ptr(status),
                                                   _stream(stream)))
    return status


def kv_get_last_error(clear: bool = True, stream=None) -> int:
    """The sticky error word (KV_DERR_* bits).  Where it reports KV_DERR_TIMEOUT, the workspaces that the attention
    calls without one keep on this device are given up: a call that broke off leaves its counters in them."""
    out = ctypes.c_int32(0)
    _check("kv_get_last_error", load().kv_get_last_error(ctypes.byref(out), 1 if clear else 0, _stream(stream)))
    if out.value & KV_DERR_TIMEOUT:
        kv_reset_workspaces()
    return out.value


# ---------------------------------------------------------------------------
# attention over the paged cache
# ---------------------------------------------------------------------------
# These calls run once a layer and step, so the marshalling is kept short: plain integers for pointers, the
# raw stream handle, one device check a tensor.
LATENT_DIM, LATENT_RANK = 576, 512  # elements of a latent row, and of its latent part


def kv_attention_workspace_bytes() -> int:
    out = ctypes.c_int64(0)
    _check("kv_attention_workspace_bytes", load().kv_attention_workspace_bytes(ctypes.byref(out)))
    return out.value


def kv_attention_mass_workspace_bytes() -> int:
    out = ctypes.c_int64(0)
    _check("kv_attention_mass_workspace_bytes", load().kv_attention_mass_workspace_bytes(ctypes.byref(out)))
    return out.value


def kv_attention_workspace(device="cuda") -> torch.Tensor:
    """A workspace for kv_attention, kv_latent_attention and kv_attention_mass calls of any size on `device`,
    zeroed on the current stream; calls that share one must be ordered."""
    with torch.cuda.device(device):
        return torch.zeros(kv_attention_workspace_bytes(), dtype=torch.uint8, device=device)


_workspaces = {}  # (bytes function, device, stream handle) -> the workspace of calls without one on that stream


def kv_reset_workspaces(device: Optional[int] = None):
    """Gives up the workspaces that calls without one keep, one a stream, on a device (default: the current one).  The
    next such call makes a zeroed one.  Done by kv_get_last_error after a timeout; also frees those of streams that are no longer used."""
    dev = torch.cuda.current_device() if device is None else device
    for key in list(_workspaces):
        if key[1] == dev:
            _workspaces.pop(key, None)


def _workspace(nbytes, dev: int, handle: int, given: Optional[torch.Tensor], stream) -> torch.Tensor:
    """The workspace of a call.  Calls that bring none share one a stream, whose calls are in order.  A call that is being
    captured gets one of its own, in the graph's memory and zeroed by the graph, as replays are not in that order."""
    if given is not None:
        if given.get_device() != dev or not given.is_contiguous():
            raise ValueError(f"the workspace must be a contiguous tensor on cuda:{dev}")
        return given
    with _no_context() if stream is None else torch.cuda.stream(stream):
        if torch.cuda.is_current_stream_capturing():
            ws = torch.empty(nbytes(), dtype=torch.uint8, device=f"cuda:{dev}")
            ws[:KV_ATTENTION_ZEROED_BYTES].zero_()
            return ws
        key = (nbytes, dev, handle)
        ws = _workspaces.get(key)
        if ws is None:
            ws = _workspaces[key] = torch.zeros(nbytes(), dtype=torch.uint8, device=f"cuda:{dev}")
        return ws


def _begin(dev: int, stream) -> int:
    """The raw stream handle of a call whose tensors are on device `dev`."""
    if dev != torch._C._cuda_getDevice():
        raise ValueError("libpagedkv takes CUDA tensors" if dev < 0 else f"the tensors are on cuda:{dev}, which is not the current device")
    return torch._C._cuda_getCurrentRawStream(dev) if stream is None else stream.cuda_stream


def _on(dev: int, *tensors):
    for t in tensors:
        if t is not None and t.get_device() != dev:
            raise ValueError(f"every tensor must be on cuda:{dev}")


def _empty(like: torch.Tensor, shape, dtype: torch.dtype, stream) -> torch.Tensor:
    """An output, which belongs to the stream that writes it."""
    if stream is None:
        return torch.empty(shape, dtype=dtype, device=like.device)
    with torch.cuda.stream(stream):
        return torch.empty(shape, dtype=dtype, device=like.device)


def _table(dev: int, t: torch.Tensor, n: int, name: str):
    """(pointer, pages of a row, row stride) of a block table of n requests."""
    if t.dtype is not torch.int32 or t.dim() != 2 or t.shape[0] != n or t.get_device() != dev:
        raise ValueError(f"{name} must be an int32 [n_reqs, max_blocks] tensor on cuda:{dev}, with the batch's requests")
    row, one = t.stride()
    if one != 1:
        raise ValueError(f"{name} must be row-major")
    pages = t.shape[1]
    if pages >= 2 ** 31:
        raise ValueError(f"{name}'s columns must be a 32-bit number")
    return t.data_ptr(), pages, row


def _i32_on(dev: int, t: torch.Tensor, n: int, name: str) -> int:
    if t.dtype is not torch.int32 or t.get_device() != dev or t.shape != (n,) or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous int32 [{n}] tensor on cuda:{dev}")
    return t.data_ptr()


def _attn_batch(dev: int, block_table: torch.Tensor, q_offsets: torch.Tensor, kv_lens: torch.Tensor, n_tokens: int) -> KvAttnBatch:
    n = kv_lens.numel()
    table, pages, row = _table(dev, block_table, n, "block_table")
    return KvAttnBatch(table, n, pages, row, _i32_on(dev, q_offsets, n + 1, "q_offsets"), _i32_on(dev, kv_lens, n, "kv_lens"), n_tokens)


def _rows3(t: torch.Tensor, name: str):
    """(KV_BF16 or KV_F16, byte strides of tokens and heads) of [tokens, heads, dim] rows."""
    code = _DTYPES.get(t.dtype)
    if code is None or t.dim() != 3:
        raise ValueError(f"{name} must be a bf16 or fp16 CUDA tensor [tokens, heads, dim]")
    token, head, one = t.stride()
    if one != 1 and t.shape[2] > 1:
        raise ValueError(f"{name} must have contiguous rows")
    return code, token * 2, head * 2


def _like_cache(dev: int, cache: PagedCache, dtype: torch.dtype, name: str) -> KvCacheDesc:
    t = cache.tensors[0]
    if t.dtype is not dtype or t.get_device() != dev:
        raise ValueError(f"{name} must hold {dtype} on cuda:{dev}")
    return cache.desc()


def _attn_outputs(dev: int, q: torch.Tensor, T: int, H: int, dv: int, out: Optional[torch.Tensor], lse: Optional[torch.Tensor], stream):
    """(out, its token and head strides in bytes, lse)."""
    if out is None and lse is None and stream is None:
        device = q.device
        return (torch.empty((T, H, dv), dtype=q.dtype, device=device), H * dv * 2, dv * 2,
                torch.empty((T, H), dtype=torch.float32, device=device))
    if out is None:
        out = _empty(q, (T, H, dv), q.dtype, stream)
    elif out.shape != (T, H, dv) or out.dtype is not q.dtype or out.get_device() != dev:
        raise ValueError("out must be [tokens, heads, value dim] of q's type, on its device")
    if lse is None:
        lse = _empty(q, (T, H), torch.float32, stream)
    elif lse.shape != (T, H) or lse.dtype is not torch.float32 or not lse.is_contiguous() or lse.get_device() != dev:
        raise ValueError("lse must be a contiguous float32 [tokens, heads] tensor on q's device")
    _, token, head = _rows3(out, "out")
    return out, token, head, lse


def _int32(**values):
    """ctypes would cut a number off to 32 bits without a word."""
    for name, x in values.items():
        if not -2 ** 31 <= x < 2 ** 31:
            raise ValueError(f"{name} must be a 32-bit number")


def _tensor_numbers(*numbers):
    """Short of _int32's names: these are checked at every call."""
    for x in numbers:
        if not -2 ** 31 <= x < 2 ** 31:
            raise ValueError("a tensor's number must be a 32-bit number")


@functools.lru_cache(maxsize=256)
def _attn_desc(*fields) -> KvAttnDesc:
    """Descriptions repeat from layer to layer; the library only reads them."""
    _int32(n_kv_heads=fields[2], head_dim_v=fields[4], window=fields[6])
    return KvAttnDesc(*fields)


def kv_attention(q: torch.Tensor, cache: PagedCache, block_table: torch.Tensor, q_offsets: torch.Tensor,
                 kv_lens: torch.Tensor, scale: float, *, v_cache: Optional[PagedCache] = None, k_tensor: int = 0,
                 v_tensor: Optional[int] = None, causal: bool = True, window: int = 0, out: Optional[torch.Tensor] = None,
                 lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """Attention of new tokens q [tokens, heads, dim] over the paged cache; returns (out, lse float32 [tokens, heads]).

    Keys are tensor `k_tensor` of `cache` (plane 0).  Values are tensor `v_tensor` of `v_cache`, or, without a
    `v_cache`, plane 1 of the same tensor (two-plane caches) or tensor `v_tensor` of `cache`."""
    _tensor_numbers(k_tensor, v_tensor or 0)
    code, q_token, q_head = _rows3(q, "q")
    dev = q.get_device()
    handle = _begin(dev, stream)
    k_desc = _like_cache(dev, cache, q.dtype, "cache")
    if v_cache is None:
        values, v_desc = cache, k_desc
        if v_tensor is None:
            if cache.n_planes == 1:
                raise ValueError("a one-plane cache holds the values in another tensor: give v_tensor or v_cache")
            v_tensor = k_tensor
    else:
        values, v_desc, v_tensor = v_cache, _like_cache(dev, v_cache, q.dtype, "v_cache"), v_tensor or 0
    T, H, dk = q.shape
    kv_heads, left = divmod(cache.row_bytes, dk * 2) if dk else (0, 0)
    if left or not kv_heads or values.row_bytes % (kv_heads * 2):
        raise ValueError("the cache's rows are not whole heads of q's width")
    dv = values.row_bytes // (kv_heads * 2)
    batch = _attn_batch(dev, block_table, q_offsets, kv_lens, T)
    out, o_token, o_head, lse = _attn_outputs(dev, q, T, H, dv, out, lse, stream)
    workspace = _workspace(kv_attention_workspace_bytes, dev, handle, workspace, stream)
    _check("kv_attention", (_lib or load()).kv_attention(
        _attn_desc(code, H, kv_heads, dk, dv, causal, window, float(scale)), batch, k_desc, k_tensor, 0, v_desc, v_tensor, values.n_planes - 1,
        q.data_ptr(), q_token, q_head, out.data_ptr(), o_token, o_head, lse.data_ptr(), workspace.data_ptr(), workspace.nbytes, handle))
    return out, lse


def kv_latent_attention(q: torch.Tensor, cache: PagedCache, block_table: torch.Tensor, q_offsets: torch.Tensor,
                        kv_lens: torch.Tensor, scale: float, *, tensor: int = 0, causal: bool = True, window: int = 0,
                        out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                        workspace: Optional[torch.Tensor] = None, stream=None):
    """Attention of new tokens q [tokens, heads, 576] over a latent cache (the absorbed form); returns
    (out [tokens, heads, 512], lse float32 [tokens, heads])."""
    _tensor_numbers(tensor)
    code, q_token, q_head = _rows3(q, "q")
    dev = q.get_device()
    handle = _begin(dev, stream)
    c_desc = _like_cache(dev, cache, q.dtype, "cache")
    T, H, dk = q.shape
    batch = _attn_batch(dev, block_table, q_offsets, kv_lens, T)
    out, o_token, o_head, lse = _attn_outputs(dev, q, T, H, LATENT_RANK, out, lse, stream)
    workspace = _workspace(kv_attention_workspace_bytes, dev, handle, workspace, stream)
    _check("kv_latent_attention", (_lib or load()).kv_latent_attention(
        _attn_desc(code, H, 1, dk, LATENT_RANK, causal, window, float(scale)), batch, c_desc, tensor, q.data_ptr(), q_token, q_head,
        out.data_ptr(), o_token, o_head, lse.data_ptr(), workspace.data_ptr(), workspace.nbytes, handle))
    return out, lse


def kv_latent_expand(cache: PagedCache, block_table: torch.Tensor, kv_lens: torch.Tensor, weight: torch.Tensor,
                     k_out: PagedCache, v_out: PagedCache, out_table: torch.Tensor, *, tensor: int = 0, k_tensor: int = 0,
                     v_tensor: int = 0, stream=None):
    """The latent rows of every request multiplied out by weight [heads, 256, 512] into per-head keys (192) and
    values (128) of the caches k_out and v_out, at the same tokens of out_table."""
    _tensor_numbers(tensor, k_tensor, v_tensor)
    code = _DTYPES.get(weight.dtype)
    if code is None or weight.dim() != 3 or tuple(weight.shape[1:]) != (256, LATENT_RANK) or not weight.is_contiguous():
        raise ValueError("weight must be a contiguous bf16 or fp16 [heads, 256, 512] CUDA tensor")
    dev = weight.get_device()
    handle = _begin(dev, stream)
    n = kv_lens.numel()
    table, pages, row = _table(dev, block_table, n, "block_table")
    out, out_pages, out_row = _table(dev, out_table, n, "out_table")
    dtype = weight.dtype
    _check("kv_latent_expand", (_lib or load()).kv_latent_expand(
        code, weight.shape[0], _like_cache(dev, cache, dtype, "cache"), tensor, table, n, pages, row, _i32_on(dev, kv_lens, n, "kv_lens"),
        weight.data_ptr(), _like_cache(dev, k_out, dtype, "k_out"), k_tensor, _like_cache(dev, v_out, dtype, "v_out"), v_tensor, out,
        out_pages, out_row, handle))


def _score_rows(dev: int, t: torch.Tensor, n: int, width: int, name: str):
    """(pointer, row stride) of scores."""
    if t.dtype is not torch.float32 or t.dim() != 2 or t.shape[0] != n or t.shape[1] < width or t.get_device() != dev:
        raise ValueError(f"{name} must be a float32 [n_reqs, {width} or more] tensor on cuda:{dev}")
    row, one = t.stride()
    if one != 1 and t.shape[1] > 1:
        raise ValueError(f"{name} must be row-major")
    if t.shape[1] >= 2 ** 31:
        raise ValueError(f"{name}'s columns must be a 32-bit number")
    return t.data_ptr(), row


def kv_attention_mass(q: torch.Tensor, cache: PagedCache, block_table: torch.Tensor, q_offsets: torch.Tensor,
                      kv_lens: torch.Tensor, lse: torch.Tensor, scale: float, *, k_tensor: int = 0, causal: bool = True,
                      window: int = 0, prev: Optional[torch.Tensor] = None, score: Optional[torch.Tensor] = None,
                      width: Optional[int] = None, workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The attention weight every cached token receives from q, added to prev (float32 [n_reqs, width], or None);
    returns score [n_reqs, width].  width: prev's or score's columns, else a table row's slots."""
    _tensor_numbers(k_tensor)
    code, q_token, q_head = _rows3(q, "q")
    dev = q.get_device()
    handle = _begin(dev, stream)
    k_desc = _like_cache(dev, cache, q.dtype, "cache")
    T, H, dk = q.shape
    kv_heads, left = divmod(cache.row_bytes, dk * 2) if dk else (0, 0)
    if left or not kv_heads:
        raise ValueError("the cache's rows are not whole heads of q's width")
    batch = _attn_batch(dev, block_table, q_offsets, kv_lens, T)
    if lse.shape != (T, H) or lse.dtype is not torch.float32 or not lse.is_contiguous() or lse.get_device() != dev:
        raise ValueError("lse must be a contiguous float32 [tokens, heads] tensor on q's device")
    n = batch.n_reqs
    if width is None:
        width = prev.shape[1] if prev is not None else score.shape[1] if score is not None else batch.max_blocks_per_req * cache.block_size
    if score is None:
        score = _empty(q, (n, width), torch.float32, stream)
    to, to_row = _score_rows(dev, score, n, width, "score")
    before, before_row = (None, 0) if prev is None else _score_rows(dev, prev, n, width, "prev")
    workspace = _workspace(kv_attention_mass_workspace_bytes, dev, handle, workspace, stream)
    _check("kv_attention_mass", (_lib or load()).kv_attention_mass(
        _attn_desc(code, H, kv_heads, dk, dk, causal, window, float(scale)), batch, k_desc, k_tensor, 0, q.data_ptr(), q_token, q_head,
        lse.data_ptr(), before, before_row, to, to_row, width, workspace.data_ptr(), workspace.nbytes, handle))
    return score


def kv_evict(cache: PagedCache, block_table: torch.Tensor, kv_lens: torch.Tensor, score: torch.Tensor, budget: int, *,
             sinks: int = 0, recent: int = 0, out_table: Optional[torch.Tensor] = None, new_lens: Optional[torch.Tensor] = None,
             kept: Optional[torch.Tensor] = None, out_score: Optional[torch.Tensor] = None, stream=None):
    """Trims every request to `budget` tokens: the first `sinks`, the last `recent` and the highest scores between, in
    their order; rows of every tensor and plane are gathered to out_table's pages (None: in place).  Returns
    (new_lens int32 [n_reqs], kept int32 [n_reqs, budget], out_score float32 [n_reqs, budget]).

    Tokens past score's columns count as 0.  Of out_score only `budget` columns are written: to go on adding weights,
    keep a score of a table row's slots, clear it and copy out_score to its first columns."""
    _int32(budget=budget, sinks=sinks, recent=recent)
    dev = kv_lens.get_device()
    handle = _begin(dev, stream)
    n = kv_lens.numel()
    table, pages, row = _table(dev, block_table, n, "block_table")
    out, out_pages, out_row = (table, pages, row) if out_table is None else _table(dev, out_table, n, "out_table")
    if budget < 0:
        raise ValueError("budget must not be negative")
    if new_lens is None:
        new_lens = _empty(kv_lens, (n,), torch.int32, stream)
    if kept is None:
        kept = _empty(kv_lens, (n, budget), torch.int32, stream)
    elif kept.dtype is not torch.int32 or kept.shape != (n, budget) or kept.get_device() != dev or (budget > 1 and kept.stride(1) != 1):
        raise ValueError("kept must be a row-major int32 [n_reqs, budget] tensor on the requests' device")
    if out_score is None:
        out_score = _empty(kv_lens, (n, budget), torch.float32, stream)
    from_score, from_row = _score_rows(dev, score, n, 0, "score")
    to_score, to_row = _score_rows(dev, out_score, n, budget, "out_score")
    _on(dev, *cache.tensors[:1])
    _check("kv_evict", (_lib or load()).kv_evict(
        cache.desc(), table, n, pages, row, _i32_on(dev, kv_lens, n, "kv_lens"), from_score, from_row, score.shape[1], budget, sinks, recent,
        out, out_pages, out_row, _i32_on(dev, new_lens, n, "new_lens"), kept.data_ptr(), kept.stride(0), to_score, to_row, handle))
    return new_lens, kept, out_score


# ---------------------------------------------------------------------------
# rotary positions, and the writes that apply them
# ---------------------------------------------------------------------------
_ROPE_KINDS = {"none": 0, "linear": 1, "base": 2, "bands": 3, "yarn": 4}


def kv_rope_frequencies(rot_dim: int, base: float = 10000.0, *, scaling: str = "none", factor: float = 1.0,
                        original_length: float = 8192.0, fast: Optional[float] = None, slow: float = 1.0):
    """(frequencies as 64-bit fractions of a turn, int64 [rot_dim / 2] on the CPU; magnitude), see kv_rope_scaling.

    scaling: "none", "linear", "base", "bands" or "yarn"; fast: turns over original_length from which a pair stays as it
    is (default 4 for "bands", 32 for "yarn")."""
    if scaling not in _ROPE_KINDS:
        raise ValueError(f"scaling must be one of {', '.join(_ROPE_KINDS)}")
    _int32(rot_dim=rot_dim)
    turns = torch.empty(max(rot_dim, 0) // 2, dtype=torch.int64)
    magnitude = ctypes.c_float(0)
    how = KvRopeScaling(_ROPE_KINDS[scaling], factor, original_length, fast if fast is not None else 32.0 if scaling == "yarn" else 4.0, slow)
    _check("kv_rope_frequencies", load().kv_rope_frequencies(rot_dim, base, ctypes.byref(how), turns.data_ptr(), ctypes.byref(magnitude)))
    return turns, magnitude.value


class Rope:
    """What rotates of a head (kv_rope): the frequencies on the GPU, the part of the head, the order of its pairs."""

    def __init__(self, turns: torch.Tensor, *, offset: int = 0, interleaved: bool = False, magnitude: float = 1.0):
        if turns.dtype is not torch.int64 or turns.dim() != 1 or not turns.is_contiguous() or not turns.is_cuda:
            raise ValueError("turns must be a contiguous int64 CUDA tensor, one frequency a pair")
        _int32(rot_dim=2 * turns.numel(), offset=offset)
        self.turns, self.device = turns, turns.get_device()
        self.desc = KvRope(turns.data_ptr(), 2 * turns.numel(), offset, 1 if interleaved else 0, magnitude)

    @classmethod
    def make(cls, rot_dim: int, base: float = 10000.0, *, offset: int = 0, interleaved: bool = False, device="cuda", **scaling) -> "Rope":
        """The rotation of rot_dim elements; scaling: the keywords of kv_rope_frequencies."""
        turns, magnitude = kv_rope_frequencies(rot_dim, base, **scaling)
        return cls(turns.to(device), offset=offset, interleaved=interleaved, magnitude=magnitude)


def _rope_on(dev: int, rope: Optional[Rope]) -> Optional[KvRope]:
    if rope is None:
        return None
    if rope.device != dev:
        raise ValueError(f"the rotation's frequencies must be on cuda:{dev}")
    return rope.desc


def _rotated_out(dev: int, x: torch.Tensor, shape, out: Optional[torch.Tensor], name: str, stream):
    """(out, its token and head strides in bytes) for x [tokens, heads, dim] rotated."""
    if out is None:
        _, H, d = shape
        return _empty(x, shape, x.dtype, stream), H * d * 2, d * 2
    if out.shape != shape or out.dtype is not x.dtype or out.get_device() != dev:
        raise ValueError(f"the output of {name} must have its shape and type, on its device")
    _, token, head = _rows3(out, f"the output of {name}")
    return out, token, head


def kv_rotate(x: torch.Tensor, token_pos: torch.Tensor, rope: Rope, *, inverse: bool = False, out: Optional[torch.Tensor] = None,
              stream=None) -> torch.Tensor:
    """Heads x [tokens, heads, dim] rotated by their tokens' positions (int32 [tokens]); out may be x itself.  inverse: the
    transposed map, which takes the output's gradient to x's."""
    dev = x.get_device()
    handle = _begin(dev, stream)
    code, token, head = _rows3(x, "x")
    T, H, d = shape = x.shape
    out, to_token, to_head = _rotated_out(dev, x, shape, out, "x", stream)
    _check("kv_rotate", (_lib or load()).kv_rotate(code, H, d, x.data_ptr(), token, head, out.data_ptr(), to_token, to_head, T,
                                                   _i32_on(dev, token_pos, T, "token_pos"), _rope_on(dev, rope), 1 if inverse else 0, handle))
    return out


def _new_tokens(q, k, v, block_table, token_req, token_pos, rope_pos, q_out, stream):
    """(kv_new_tokens, device, stream handle, q_out)."""
    code, k_token, k_head = _rows3(k, "k")
    dev = k.get_device()
    handle = _begin(dev, stream)
    T, G, dk = k.shape
    H = q_at = q_token = q_head = to_at = to_token = to_head = v_at = v_token = v_head = dv = 0
    if q is not None:
        q_code, q_token, q_head = _rows3(q, "q")
        tokens, H, d = shape = q.shape
        if q_code != code or tokens != T or d != dk or q.get_device() != dev:
            raise ValueError("q must have k's tokens, width, type and device")
        q_out, to_token, to_head = _rotated_out(dev, q, shape, q_out, "q", stream)
        q_at, to_at = q.data_ptr(), q_out.data_ptr()
    elif q_out is not None:
        raise ValueError("q_out without q")
    if v is not None:
        v_code, v_token, v_head = _rows3(v, "v")
        tokens, heads, dv = v.shape
        if v_code != code or tokens != T or heads != G or v.get_device() != dev:
            raise ValueError("v must have k's tokens, heads, type and device")
        v_at = v.data_ptr()
    if block_table.dim() != 2:
        raise ValueError("block_table must be an int32 [n_reqs, max_blocks] tensor")
    n = block_table.shape[0]
    table, pages, row = _table(dev, block_table, n, "block_table")
    d = KvNewTokens(code, H, G, dk, dv, q_at, q_token, q_head, to_at, to_token, to_head, k.data_ptr(), k_token, k_head, v_at, v_token, v_head,
                    _i32_on(dev, token_req, T, "token_req"), _i32_on(dev, token_pos, T, "token_pos"),
                    None if rope_pos is None else _i32_on(dev, rope_pos, T, "rope_pos"), T, table, n, pages, row)
    return d, dev, handle, q_out


def _key_and_value_planes(dev: int, cache: PagedCache, v_cache: Optional[PagedCache], k_tensor: int, v_tensor: Optional[int], dtype, values: bool = True):
    """(descriptions of the keys' and values' caches, the values' tensor, their plane), as kv_attention finds them."""
    k_desc = _like_cache(dev, cache, dtype, "cache")
    if v_cache is not None:
        return k_desc, _like_cache(dev, v_cache, dtype, "v_cache"), v_tensor or 0, v_cache.n_planes - 1
    if v_tensor is None:
        if cache.n_planes == 1 and values:
            raise ValueError("a one-plane cache holds the values in another tensor: give v_tensor or v_cache")
        v_tensor = k_tensor
    return k_desc, k_desc, v_tensor, cache.n_planes - 1


def kv_rotate_write(q: Optional[torch.Tensor], k: torch.Tensor, v: Optional[torch.Tensor], cache: PagedCache, block_table: torch.Tensor,
                    token_req: torch.Tensor, token_pos: torch.Tensor, rope: Optional[Rope], *, v_cache: Optional[PagedCache] = None,
                    k_tensor: int = 0, v_tensor: Optional[int] = None, rope_pos: Optional[torch.Tensor] = None,
                    q_out: Optional[torch.Tensor] = None, stream=None) -> Optional[torch.Tensor]:
    """One layer's new tokens: keys k [tokens, key heads, dim] rotated and values v as they are written to the pages that the
    block table gives, queries q [tokens, heads, dim] rotated into q_out (may be q), which is returned.  v None: rows
    without values (latent ones).  Keys and values are placed as kv_attention finds them.  rope_pos: positions to rotate by, where
    they are not token_pos."""
    _tensor_numbers(k_tensor, v_tensor or 0)
    d, dev, handle, q_out = _new_tokens(q, k, v, block_table, token_req, token_pos, rope_pos, q_out, stream)
    k_desc, v_desc, v_tensor, v_plane = _key_and_value_planes(dev, cache, v_cache, k_tensor, v_tensor, k.dtype, v is not None)
    _check("kv_rotate_write", (_lib or load()).kv_rotate_write(d, _rope_on(dev, rope), k_desc, k_tensor, 0, v_desc, v_tensor, v_plane, handle))
    return q_out


def kv_q4_row_bytes(heads: int, head_dim: int) -> int:
    """Bytes of a 4-bit cache's row; such a cache is a PagedCache of uint8 tensors [.., block, row bytes]."""
    _int32(heads=heads, head_dim=head_dim)
    out = ctypes.c_int32(0)
    _check("kv_q4_row_bytes", load().kv_q4_row_bytes(heads, head_dim, ctypes.byref(out)))
    return out.value


def kv_rotate_write_q4(q: Optional[torch.Tensor], k: torch.Tensor, v: torch.Tensor, cache: PagedCache, block_table: torch.Tensor,
                       token_req: torch.Tensor, token_pos: torch.Tensor, rope: Optional[Rope], *, v_cache: Optional[PagedCache] = None,
                       k_tensor: int = 0, v_tensor: Optional[int] = None, rope_pos: Optional[torch.Tensor] = None, k_scale: float = 1.0,
                       v_scale: float = 1.0, q_out: Optional[torch.Tensor] = None, held: bool = False, stream=None):
    """kv_rotate_write into a 4-bit cache; k_scale and v_scale are the tensors' scales, which kv_attention_q4 takes too.  Returns
    q_out, or (q_out, keys, values) with what the cache now stands for when `held`."""
    _tensor_numbers(k_tensor, v_tensor or 0)
    d, dev, handle, q_out = _new_tokens(q, k, v, block_table, token_req, token_pos, rope_pos, q_out, stream)
    k_desc, v_desc, v_tensor, v_plane = _key_and_value_planes(dev, cache, v_cache, k_tensor, v_tensor, torch.uint8)
    k_held = _empty(k, k.shape, k.dtype, stream) if held else None
    v_held = _empty(k, v.shape, v.dtype, stream) if held else None
    _check("kv_rotate_write_q4", (_lib or load()).kv_rotate_write_q4(
        d, _rope_on(dev, rope), k_desc, k_tensor, 0, v_desc, v_tensor, v_plane, k_scale, v_scale, k_held.data_ptr() if held else None,
        v_held.data_ptr() if held else None, handle))
    return (q_out, k_held, v_held) if held else q_out


def kv_attention_q4(q: torch.Tensor, cache: PagedCache, block_table: torch.Tensor, q_offsets: torch.Tensor, kv_lens: torch.Tensor,
                    scale: float, *, kv_heads: int, head_dim_v: Optional[int] = None, v_cache: Optional[PagedCache] = None, k_tensor: int = 0,
                    v_tensor: Optional[int] = None, k_scale: float = 1.0, v_scale: float = 1.0, causal: bool = True, window: int = 0,
                    out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None, workspace: Optional[torch.Tensor] = None, stream=None):
    """kv_attention over a 4-bit cache that kv_rotate_write_q4 filled; returns (out, lse float32 [tokens, heads]).  kv_heads and
    head_dim_v (default: q's width) say what a row holds; k_scale and v_scale are the tensors' scales."""
    _tensor_numbers(k_tensor, v_tensor or 0)
    code, q_token, q_head = _rows3(q, "q")
    dev = q.get_device()
    handle = _begin(dev, stream)
    k_desc, v_desc, v_tensor, v_plane = _key_and_value_planes(dev, cache, v_cache, k_tensor, v_tensor, torch.uint8)
    T, H, dk = q.shape
    dv = dk if head_dim_v is None else head_dim_v
    if dv < 0:
        raise ValueError("head_dim_v must not be negative")
    attn = _attn_desc(code, H, kv_heads, dk, dv, causal, window, float(scale))
    batch = _attn_batch(dev, block_table, q_offsets, kv_lens, T)
    out, o_token, o_head, lse = _attn_outputs(dev, q, T, H, dv, out, lse, stream)
    workspace = _workspace(kv_attention_workspace_bytes, dev, handle, workspace, stream)
    _check("kv_attention_q4", (_lib or load()).kv_attention_q4(
        attn, batch, k_desc, k_tensor, 0, v_desc, v_tensor, v_plane, k_scale, v_scale,
        q.data_ptr(), q_token, q_head, out.data_ptr(), o_token, o_head, lse.data_ptr(), workspace.data_ptr(), workspace.nbytes, handle))
    return out, lse


def default_max_run_blocks(stage_block_bytes: int, target_bytes: int = 16 * 1024) -> int:
    """A run cap that keeps one run at or under target_bytes per tensor (at least one block).

    16 KiB is the piece a copy kernel hands to one warp, so a capped run is never split."""
    return max(1, int(target_bytes) // max(1, int(stage_block_bytes)))
