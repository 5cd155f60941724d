"""The attention side of a decode layer, on torch tensors: residual addition +
RMSNorm + MXFP8, the 8-bit paged key/value cache, and the attention over it.

Argument marshalling only, like :mod:`.api`: tensor shapes, dtypes, devices and
strides are checked here (the kernels' loads are unbounded), the work runs in
the library's CUDA kernels on the current stream. Nothing synchronises: what
the kernels find in device data (page ids, lengths) is reported in the bits of
an int32 ``status`` tensor if one is passed (``KV_STATUS_*`` of :mod:`._lib`).
"""

from __future__ import annotations

import ctypes
import math
import struct

import torch

from . import _lib
from ._lib import ATTN_X8_WORKSPACE_BYTES, KV_PAGE_TOKENS, check


def _rows(name: str, t: torch.Tensor, shape: tuple, device) -> int:
    """Checks bf16 rows of contiguous values (any row stride); returns the stride."""
    if t.dtype != torch.bfloat16 or t.shape != shape or t.device != device:
        raise ValueError(f"{name} must be bf16 {tuple(shape)} on {device}, got {t.dtype} {tuple(t.shape)} {t.device}")
    stride = t.stride()
    if len(shape) == 3:
        width = shape[1] * shape[2]
        dense = (stride[2] == 1 or shape[2] == 1) and (stride[1] == shape[2] or shape[1] == 1)
    else:
        width = shape[1]
        dense = stride[1] == 1 or width == 1
    if not dense and shape[0] > 0:
        raise ValueError(f"{name}: the values of a row must be contiguous")
    return stride[0] if shape[0] > 1 else width  # (one row or none: any stride)


def _dense(name: str, t, shape: tuple, dtype, device) -> None:
    if t.shape != shape or t.dtype != dtype or t.device != device or not t.is_contiguous():
        raise ValueError(f"{name} must be a contiguous {dtype} {tuple(shape)} tensor on {device}, "
                         f"got {t.dtype} {tuple(t.shape)} {t.device}")


# The decode step's calls are a few microseconds of GPU work each, so the way to
# the launch is kept short: torch's own accessors behind current_device() and
# current_stream(), without their argument handling.
_current_device = getattr(torch._C, "_cuda_getDevice", torch.cuda.current_device)
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream",
                      lambda index: torch.cuda.current_stream(index).cuda_stream)


# moe_kv_cache and moe_kv_seqs as bytes in C layout
_CACHE = struct.Struct("@PPiii")
_SEQS = struct.Struct("@PPPiiii")
_entry_points = None


def _entries():
    """The cache's two entry points with their structs passed as bytes."""
    global _entry_points
    if _entry_points is None:
        L = _lib.lib()
        append, attn = L["moe_kv_append_x8"], L["moe_attn_x8"]
        for fn, ref in ((append, L.moe_kv_append_x8), (attn, L.moe_attn_x8)):
            fn.argtypes = [ctypes.c_char_p, ctypes.c_char_p, *ref.argtypes[2:]]
            fn.restype = ref.restype
        _entry_points = append, attn
    return _entry_points


def _call(name: str, fn, index: int, *args) -> None:
    """fn(*args, stream) on the device's current stream, with the device current."""
    if _current_device() == index:
        code = fn(*args, _raw_stream(index))
    else:
        with torch.cuda.device(index):
            code = fn(*args, _raw_stream(index))
    if code:
        check(code, name)


def add_norm_x8(x: torch.Tensor, residual: torch.Tensor, norm_w: torch.Tensor, eps: float = 1e-6,
                res_out: torch.Tensor | None = None, x8: torch.Tensor | None = None,
                codes: torch.Tensor | None = None, normed: torch.Tensor | None = None):
    """res_out = bf16(x + residual), its RMSNorm with ``norm_w``, and the norm's
    MXFP8 (``moe_add_norm_x8``) for rows [M, H], M any.

    x and residual: bf16 [M, H], rows may be strided. Returns (res_out bf16
    [M, H], x8 uint8 [M, H], codes uint8 [M, H/32], normed): outputs not passed
    are allocated here, except ``normed`` (the norm in bf16), which is written
    only if a tensor is passed. ``res_out`` may be ``residual`` (or ``x``) itself
    if that is contiguous.
    """
    if x.dim() != 2 or not x.is_cuda:
        raise ValueError("x must be a CUDA bf16 [M, H] tensor")
    shape = x.shape
    M, H = shape
    dev = x.device
    if H % 32:
        raise ValueError("H must be a multiple of 32")
    ldx = _rows("x", x, shape, dev)
    ldr = _rows("residual", residual, shape, dev)
    _dense("norm_w", norm_w, (H,), torch.bfloat16, dev)
    if res_out is None:
        res_out = torch.empty(shape, dtype=torch.bfloat16, device=dev)
    else:
        _dense("res_out", res_out, shape, torch.bfloat16, dev)
    if x8 is None:
        x8 = torch.empty(shape, dtype=torch.uint8, device=dev)
    else:
        _dense("x8", x8, shape, torch.uint8, dev)
    if codes is None:
        codes = torch.empty((M, H // 32), dtype=torch.uint8, device=dev)
    else:
        _dense("codes", codes, (M, H // 32), torch.uint8, dev)
    if normed is not None:
        _dense("normed", normed, shape, torch.bfloat16, dev)
    _call("moe_add_norm_x8", _lib.lib().moe_add_norm_x8, dev.index, x.data_ptr(), ldx,
          residual.data_ptr(), ldr, norm_w.data_ptr(), M, H, eps, res_out.data_ptr(), x8.data_ptr(),
          codes.data_ptr(), None if normed is None else normed.data_ptr())
    return res_out, x8, codes, normed


# ---------------------------------------------------------------- the cache
def kv_cache_x8(pages: int, kv_heads: int, head_dim: int, device="cuda"):
    """(blocks uint8 [pages, kv_heads, 2, 64 * head_dim], codes uint8 [pages,
    kv_heads, 2]) of an empty cache; a page needs no initial value."""
    blocks = torch.empty((pages, kv_heads, 2, KV_PAGE_TOKENS * head_dim), dtype=torch.uint8, device=device)
    codes = torch.zeros((pages, kv_heads, 2), dtype=torch.uint8, device=device)
    return blocks, codes


def kv_dequant_x8(blocks: torch.Tensor, codes: torch.Tensor) -> torch.Tensor:
    """The values the cache stands for, fp32 [pages, kv_heads, 2, 64, head_dim]
    (for tests and inspection: torch indexing, any device)."""
    pages, heads, _, size = blocks.shape
    d = size // KV_PAGE_TOKENS
    t = torch.arange(KV_PAGE_TOKENS, device=blocks.device)[:, None]
    c = torch.arange(d, device=blocks.device)[None, :]
    s = t % 8 if d >= 128 else t // 2 % 4
    key = t * d + 16 * ((c // 16) ^ s) + c % 16
    value = c * KV_PAGE_TOKENS + 16 * ((t // 16) ^ (c // 2 % 4)) + 4 * (t % 8 // 2) + 2 * (t % 16 // 8) + t % 2
    index = torch.stack((key, value)).reshape(2, -1)
    byte = torch.gather(blocks, 3, index.expand(pages, heads, 2, size))
    scale = torch.exp2(codes.double() - 127).float()
    return (byte.view(torch.float8_e4m3fn).float() * scale[..., None]).view(pages, heads, 2, KV_PAGE_TOKENS, d)


def _cache(blocks: torch.Tensor, codes: torch.Tensor):
    """(packed moe_kv_cache, kv_heads, head_dim, device)"""
    shape, dev = blocks.shape, blocks.device
    if len(shape) != 4 or not blocks.is_cuda or blocks.dtype != torch.uint8 or not blocks.is_contiguous() \
            or shape[2] != 2 or shape[3] % KV_PAGE_TOKENS:
        raise ValueError("blocks must be a contiguous CUDA uint8 [pages, kv_heads, 2, 64 * head_dim] tensor")
    pages, heads, _, size = shape
    _dense("codes", codes, (pages, heads, 2), torch.uint8, dev)
    d = size // KV_PAGE_TOKENS
    return _CACHE.pack(blocks.data_ptr(), codes.data_ptr(), pages, heads, d), heads, d, dev


def _seqs(page_table, lens, cu_q, tokens: int, max_q: int, device) -> bytes:
    """Packed moe_kv_seqs."""
    shape = page_table.shape
    if len(shape) != 2:
        raise ValueError("page_table must be an int32 [seqs, max_pages] tensor")
    n = shape[0]
    _dense("page_table", page_table, shape, torch.int32, device)
    _dense("lens", lens, (n,), torch.int32, device)
    if cu_q is None:
        if tokens != n:
            raise ValueError(f"{tokens} rows for {n} sequences: without cu_q each has one")
        starts = 0
    else:
        _dense("cu_q", cu_q, (n + 1,), torch.int32, device)
        starts = cu_q.data_ptr()
    return _SEQS.pack(page_table.data_ptr(), lens.data_ptr(), starts, n, tokens, shape[1], max_q)


def _status(status, device):
    _dense("status", status, (1,), torch.int32, device)
    return status.data_ptr()


def kv_append_x8(blocks: torch.Tensor, codes: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                 page_table: torch.Tensor, start: torch.Tensor, cu_q: torch.Tensor | None = None,
                 status: torch.Tensor | None = None):
    """Writes new keys and values into the cache (``moe_kv_append_x8``).

    k, v: bf16 [tokens, kv_heads, head_dim], rows may be strided (parts of a
    projection's output). page_table int32 [seqs, max_pages], start int32 [seqs]
    (tokens each sequence has already), cu_q int32 [seqs + 1] (rows of each
    sequence; None: one each). Changes blocks and codes in place and returns them.
    """
    cache, heads, d, dev = _cache(blocks, codes)
    if k.dim() != 3:
        raise ValueError("k must be a bf16 [tokens, kv_heads, head_dim] tensor")
    tokens = k.shape[0]
    shape = (tokens, heads, d)
    ldk, ldv = _rows("k", k, shape, dev), _rows("v", v, shape, dev)
    seqs = _seqs(page_table, start, cu_q, tokens, 1, dev)
    st = None if status is None else _status(status, dev)
    _call("moe_kv_append_x8", _entries()[0], dev.index, cache, seqs, k.data_ptr(), ldk,
          v.data_ptr(), ldv, st)
    return blocks, codes


def attn_x8_workspace(device="cuda") -> torch.Tensor:
    """A workspace for :func:`attn_x8` (zeroed; enough for every call)."""
    return torch.zeros(ATTN_X8_WORKSPACE_BYTES, dtype=torch.uint8, device=device)


def attn_x8(q: torch.Tensor, blocks: torch.Tensor, codes: torch.Tensor, page_table: torch.Tensor,
            kv_len: torch.Tensor, cu_q: torch.Tensor | None = None, max_q: int | None = None,
            scale: float | None = None, window: int = 0, sinks: int = 0,
            out: torch.Tensor | None = None, lse: torch.Tensor | None = None,
            workspace: torch.Tensor | None = None, status: torch.Tensor | None = None):
    """Attention of query rows over the cache (``moe_attn_x8``).

    q: bf16 [tokens, q_heads, head_dim], rows may be strided; row i of a
    sequence's n sits at position kv_len - n + i and sees the tokens up to it,
    with ``window`` > 0 only the last ``window`` of them and the first ``sinks``
    tokens. kv_len int32 [seqs] counts the tokens in the cache, the query
    tokens' own included; cu_q as in :func:`kv_append_x8`. max_q: the largest
    number of rows of one sequence, by which the kernel is chosen (default: all
    of them). scale defaults to head_dim ** -0.5.

    Returns (out bf16 [tokens, q_heads, head_dim], lse): ``lse`` (float32
    [tokens, q_heads]) is written only if a tensor is passed. A program that
    calls this often keeps a ``workspace`` (:func:`attn_x8_workspace`), one for
    each stream; without one, a zeroed one is allocated for the call.
    """
    cache, _, d, dev = _cache(blocks, codes)
    if q.dim() != 3:
        raise ValueError("q must be a bf16 [tokens, q_heads, head_dim] tensor")
    tokens, heads, _ = q.shape
    ldq = _rows("q", q, (tokens, heads, d), dev)
    if cu_q is None:
        max_q = 1
    elif max_q is None:
        max_q = max(tokens, 1)
    seqs = _seqs(page_table, kv_len, cu_q, tokens, max_q, dev)
    st = None if status is None else _status(status, dev)
    if out is None:
        out = torch.empty((tokens, heads, d), dtype=torch.bfloat16, device=dev)
    else:
        _dense("out", out, (tokens, heads, d), torch.bfloat16, dev)
    if lse is not None:
        _dense("lse", lse, (tokens, heads), torch.float32, dev)
    if workspace is None:
        workspace = attn_x8_workspace(dev)
    elif workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    _call("moe_attn_x8", _entries()[1], dev.index, cache, seqs, q.data_ptr(), ldq, heads,
          1.0 / math.sqrt(d) if scale is None else scale, window, sinks, out.data_ptr(),
          None if lse is None else lse.data_ptr(), workspace.data_ptr(),
          workspace.numel() * workspace.element_size(), st)
    return out, lse
