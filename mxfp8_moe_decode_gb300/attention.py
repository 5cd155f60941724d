"""The attention side of a decode layer, on torch tensors: residual addition +
RMSNorm + MXFP8 (also with a norm, gate and scales in front), rotary positions,
the 8-bit paged key/value cache, and the attention over it.

Argument marshalling only, like :mod:`.api`, and in compiled code (csrc/host.cpp):
tensor shapes, dtypes, devices and strides are checked there (the kernels'
loads are unbounded) and refused with ValueError, the work runs in the library's
CUDA kernels on the current stream. Nothing synchronises: what the kernels find
in device data (page ids, lengths) is reported in the bits of an int32
``status`` tensor if one is passed (``KV_STATUS_*`` of :mod:`._lib`).
"""

from __future__ import annotations

import ctypes
import math

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
                    for fn in (L.moe_add_norm_x8, L.moe_kv_append_x8, L.moe_attn_x8, L.moe_norm_add_norm_x8,
                               L.moe_rope, L.moe_rope_kv_append_x8, L.moe_linear_x4,
                               L.moe_linear_x4_workspace_bytes)))
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


def norm_add_norm_x8(x: torch.Tensor, residual: torch.Tensor, post_w: torch.Tensor | None, norm_w: torch.Tensor,
                     gate: torch.Tensor | None = None, res_scale: float = 1.0, block_scale: float = 1.0,
                     eps: float = 1e-6, res_out: torch.Tensor | None = None, x8: torch.Tensor | None = None,
                     codes: torch.Tensor | None = None, normed: torch.Tensor | None = None):
    """The norms behind and before a block with its gate (``moe_norm_add_norm_x8``):
    res_out = bf16(res_scale * residual + block_scale * gate * RMSNorm(x) * post_w),
    its RMSNorm with ``norm_w``, and the norm's MXFP8, for rows [M, H], M any.

    ``post_w`` None: the block's output x is not normed; ``gate``: bf16 [M, H]
    (rows may be strided, expanded ones included), [H], or None. The rest, and
    what is returned, as :func:`add_norm_x8`.
    """
    return _result((_bound or _host()).norm_add_norm_x8(x, residual, post_w, norm_w, gate, res_scale, block_scale, eps,
                                                        res_out, x8, codes, normed), "moe_norm_add_norm_x8")


# ---------------------------------------------------------------- rotary positions
def rope_freqs(rot: int, base: float = 10000.0, factor: float = 1.0, trained: int | None = None,
               fast: float = 32.0, slow: float = 1.0, inv_freq=None, device="cuda") -> torch.Tensor:
    """The frequencies of :func:`rope`: int64 [rot / 2], in 2^-64 turns per position
    (bits of unsigned numbers).

    Pair i turns by base^(-2 i / rot) radians per position, or by ``inv_freq[i]``
    where that is given. ``factor`` stretches a context: every frequency is
    divided by it, or with ``trained`` (the length the model was trained on) by
    parts: pairs that turn ``fast`` times or more within that length keep their
    frequency, those that turn ``slow`` times or less are divided, the pairs
    between them are mixed linearly by their number. (Given frequencies must fall
    for that, and are positive; where the two borders lie among them goes by the
    line of their logarithms. The factor of cos and sin that goes with it is
    :func:`rope`'s ``scale``.)
    """
    if rot < 2 or rot % 2:
        raise ValueError(f"rot must be even and positive, got {rot}")
    n = rot // 2
    if inv_freq is None and not 0 < base < math.inf:
        raise ValueError(f"base must be finite and positive, got {base}")
    f = [base ** (-2.0 * i / rot) for i in range(n)] if inv_freq is None else [float(v) for v in inv_freq]
    if len(f) != n:
        raise ValueError(f"inv_freq must have {n} values, got {len(f)}")
    if not factor > 0 or not all(map(math.isfinite, [factor, *f])):
        raise ValueError("frequencies must be finite, and the factor positive")
    if trained is None:
        f = [v / factor for v in f]
    else:
        if not 0 < trained < math.inf or not 0 < slow <= fast < math.inf:
            raise ValueError("trained must be positive, and 0 < slow <= fast")
        if inv_freq is None and base <= 1:
            raise ValueError(f"base must be above 1 to scale by parts, got {base}")
        if inv_freq is not None and (n < 2 or f[-1] <= 0 or any(a <= b for a, b in zip(f, f[1:]))):
            raise ValueError("inv_freq must be positive and fall from pair to pair to be scaled by parts")

        def pair(turns):  # the pair (not whole) that turns so often within the trained length
            if inv_freq is None:
                return n * math.log(trained / (turns * 2 * math.pi)) / math.log(base)
            border = turns * 2 * math.pi / trained
            i = min(max(sum(v > border for v in f) - 1, 0), n - 2)  # (beyond the ends the last two's line goes on)
            return i + math.log(f[i] / border) / math.log(f[i] / f[i + 1])

        low, high = max(math.floor(pair(fast)), 0), min(math.ceil(pair(slow)), rot - 1)
        for i in range(n):
            keep = 1.0 - min(max((i - low) / max(high - low, 1e-3), 0.0), 1.0)
            f[i] *= keep + (1.0 - keep) / factor
    if not all(map(math.isfinite, f)):
        raise ValueError("frequencies divided by the factor must be finite")
    turns = [round(math.ldexp(v / (2 * math.pi), 64)) % (1 << 64) for v in f]
    return torch.tensor([t - (1 << 64) if t >> 63 else t for t in turns], dtype=torch.int64, device=device)


def rope(x: torch.Tensor, positions: torch.Tensor, freqs: torch.Tensor, first: int = 0, interleaved: bool = False,
         scale: float = 1.0, out: torch.Tensor | None = None) -> torch.Tensor:
    """Rotary positions (``moe_rope``) of x, bf16 [tokens, heads, head_dim], rows may be strided.

    The 2 * len(freqs) dims from ``first`` on turn by positions int32 [tokens]
    (any values) times freqs (:func:`rope_freqs`); the others are copied. Pairs
    are (i, i + rot / 2), ``interleaved``: (2 i, 2 i + 1). ``scale`` is a factor of
    cos and sin. ``out``: rows may be strided; x itself turns in place.
    """
    return _result((_bound or _host()).rope(x, positions, freqs, first, interleaved, scale, out), "moe_rope")


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


def rope_kv_append_x8(blocks: torch.Tensor, codes: torch.Tensor, q: torch.Tensor, k: torch.Tensor, v: torch.Tensor,
                      page_table: torch.Tensor, start: torch.Tensor, freqs: torch.Tensor,
                      cu_q: torch.Tensor | None = None, positions: torch.Tensor | None = None, first: int = 0,
                      interleaved: bool = False, scale: float = 1.0, q_out: torch.Tensor | None = None,
                      status: torch.Tensor | None = None):
    """:func:`rope` of q and k and :func:`kv_append_x8` of k and v in one kernel
    (``moe_rope_kv_append_x8``), bit for bit what they give one after the other.

    q: bf16 [tokens, q_heads, head_dim], k and v as :func:`kv_append_x8`'s, all
    rows may be strided (parts of one projection's output). ``positions`` int32
    [tokens]; None: a token's place in the cache. Changes blocks and codes in
    place; returns (q_out, blocks, codes). ``q_out`` may be q itself.
    """
    return _result((_bound or _host()).rope_kv_append_x8(blocks, codes, q, k, v, page_table, start, freqs, cu_q,
                                                         positions, first, interleaved, scale, q_out, status),
                   "moe_rope_kv_append_x8")


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
