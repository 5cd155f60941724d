"""The attention side of a decode layer, on torch tensors: residual addition +
RMSNorm + MXFP8, the 8-bit paged key/value cache, and the attention over it.

Argument marshalling only, like :mod:`.api`, and in compiled code (csrc/host.cpp):
tensor shapes, dtypes, devices and strides are checked there (the kernels'
loads are unbounded) and refused with ValueError, the work runs in the library's
CUDA kernels on the current stream. Nothing synchronises: what the kernels find
in device data (page ids, lengths) is reported in the bits of an int32
``status`` tensor if one is passed (``KV_STATUS_*`` of :mod:`._lib`).
"""

from __future__ import annotations

import ctypes

import torch

from . import _lib
from ._lib import ATTN_X8_WORKSPACE_BYTES, KV_PAGE_TOKENS, check

_bound = None


def _host():
    """The compiled marshalling, bound to the library's entry points."""
    global _bound
    if _bound is None:
        L = _lib.lib()
        try:
            from . import _host as host
        except ImportError as e:
            raise ImportError(f"mxfp8_moe_decode_gb300._host: {e} (build it with "
                              "`python -m mxfp8_moe_decode_gb300.build`)") from e
        host.bind(*(ctypes.cast(fn, ctypes.c_void_p).value
                    for fn in (L.moe_add_norm_x8, L.moe_kv_append_x8, L.moe_attn_x8)))
        _bound = host
    return _bound


def _result(r, name: str):
    if r.__class__ is int:
        check(r, name)
    return r


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
    return _result((_bound or _host()).add_norm_x8(x, residual, norm_w, eps, res_out, x8, codes, normed),
                   "moe_add_norm_x8")


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


def kv_append_x8(blocks: torch.Tensor, codes: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                 page_table: torch.Tensor, start: torch.Tensor, cu_q: torch.Tensor | None = None,
                 status: torch.Tensor | None = None):
    """Writes new keys and values into the cache (``moe_kv_append_x8``).

    k, v: bf16 [tokens, kv_heads, head_dim], rows may be strided (parts of a
    projection's output). page_table int32 [seqs, max_pages], start int32 [seqs]
    (tokens each sequence has already), cu_q int32 [seqs + 1] (rows of each
    sequence; None: one each). Changes blocks and codes in place and returns them.
    """
    return _result((_bound or _host()).kv_append_x8(blocks, codes, k, v, page_table, start, cu_q, status),
                   "moe_kv_append_x8")


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
    return _result((_bound or _host()).attn_x8(q, blocks, codes, page_table, kv_len, cu_q, max_q, scale, window, sinks,
                                               out, lse, workspace, status), "moe_attn_x8")
