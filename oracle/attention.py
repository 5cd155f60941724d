"""The attention side in float64: residual addition, the 8-bit paged cache and
the attention over it.

TEST INFRASTRUCTURE ONLY (see the package header).

The source pages name the attention seam's norm and quantisation (layer page,
``store_x8``: :mod:`oracle.moe` ``attn_norm`` / ``attn_seam_quant``) and a
sliding-window width (``MonoBuild``'s ``swa_width``) but show no attention
body, so the formulas here are the operators' own definitions:

* ``add``: bf16(x + residual), one rounding;
* ``image_bytes``: where a page's (token, dim) bytes lie, found by walking the
  images in byte order (the library computes byte from position; this is the
  inverse, so the two pin each other);
* ``append``: per page, head and kind, token by token on plain arrays;
* ``attention``: softmax over the visible set, one row at a time.

Pins: tests/test_oracle_attention.py (hand-worked cases).
"""

from __future__ import annotations

import math

import numpy as np

from .mx import mx_code, mx_mul, mx_scale
from .numerics import bf16_rne, e4m3_decode, e4m3_encode_rne

PAGE = 64


def add(x, residual):
    """bf16_RNE(x + residual) of bf16-exact float64 arrays (the float64 sum of
    two bf16 values is exact or rounds far below the bf16 border)."""
    return bf16_rne(np.asarray(x, np.float64) + np.asarray(residual, np.float64))


def image_bytes(d: int):
    """(key, value): int arrays [64, d] of the byte of (token, dim) in a page's
    key and value image, by walking the bytes in order."""
    key = np.full((PAGE, d), -1, dtype=np.int64)
    for at in range(PAGE * d):
        token, rest = divmod(at, d)
        chunk, low = divmod(rest, 16)
        turn = token % 8 if d >= 128 else (token // 2) % 4
        key[token, (chunk ^ turn) * 16 + low] = at
    value = np.full((PAGE, d), -1, dtype=np.int64)
    for at in range(PAGE * d):
        dim, rest = divmod(at, PAGE)
        chunk, low = divmod(rest, 16)
        word, byte = divmod(low, 4)
        token = (chunk ^ ((dim // 2) % 4)) * 16 + 2 * word + (byte % 2) + 8 * (byte // 2)
        value[token, dim] = at
    return key, value


def encode(v):
    """float64 -> E4M3 bytes: saturating, NaN -> 0x7F, ties to even."""
    v = np.asarray(v, np.float64)
    b = e4m3_encode_rne(np.where(np.isnan(v), 0.0, np.clip(v, -448.0, 448.0)))
    return np.where(np.isnan(v), np.uint8(0x7F), b)


def append(blocks, codes, k, v, page_table, start, cu_q):
    """New (blocks, codes) after the append; k, v float64 [tokens, heads, d]."""
    blocks, codes = blocks.copy(), codes.copy()
    heads, d = k.shape[1:]
    where = image_bytes(d)
    for b in range(len(start)):
        n = cu_q[b + 1] - cu_q[b]
        for p in range(start[b] // PAGE, -(-(start[b] + n) // PAGE) if n else 0):
            t0, t1 = max(start[b], p * PAGE), min(start[b] + n, (p + 1) * PAGE)
            page = page_table[b][p]
            for h in range(heads):
                for kind, x in ((0, k), (1, v)):
                    new = x[cu_q[b] + t0 - start[b]:cu_q[b] + t1 - start[b], h]
                    finite = np.abs(new[np.isfinite(new)])
                    code = int(mx_code(finite.max() if finite.size else 0.0))
                    old = np.arange(0, t0 - p * PAGE)
                    if old.size:
                        had = int(codes[page, h, kind])
                        code = max(code, had)
                        if code > had:
                            at = where[kind][old].reshape(-1)
                            val = e4m3_decode(blocks[page, h, kind, at])
                            blocks[page, h, kind, at] = encode(np.ldexp(val, had - code))
                    at = where[kind][t0 - p * PAGE:t1 - p * PAGE].reshape(-1)
                    with np.errstate(invalid="ignore"):
                        blocks[page, h, kind, at] = encode(new * mx_mul(code)).reshape(-1)
                    codes[page, h, kind] = code
    return blocks, codes


def cache_values(blocks, codes):
    """float64 [pages, heads, 2, 64, d]: what the bytes stand for."""
    d = blocks.shape[3] // PAGE
    val = e4m3_decode(blocks) * mx_scale(codes)[..., None]
    key, value = image_bytes(d)
    return np.stack((val[:, :, 0][..., key], val[:, :, 1][..., value]), axis=2)


def visible(pos: int, kv: int, window: int, sinks: int):
    """Positions the row at `pos` sees, ascending."""
    return [j for j in range(min(pos + 1, kv))
            if window == 0 or j > pos - window or j < sinks]


def attention(q, values, page_table, kv_len, cu_q, scale, window=0, sinks=0):
    """(out [tokens, heads, d], lse [tokens, heads], spread [tokens, heads, d],
    slack [tokens, heads]) in float64. spread = sum_j w_j |v_j| and slack = the
    largest over the visible j of scale * (sum_d |q_d k_jd| eps_acc + 2^-17
    max|q| sum_d |k_jd|): what error bounds are made of."""
    tokens, heads, d = q.shape
    group = heads // values.shape[1]
    out = np.zeros((tokens, heads, d))
    spread = np.zeros((tokens, heads, d))
    lse = np.full((tokens, heads), -math.inf)
    slack = np.zeros((tokens, heads))
    for b in range(len(kv_len)):
        n, kv = cu_q[b + 1] - cu_q[b], kv_len[b]
        for i in range(n):
            js = np.array(visible(kv - n + i, kv, window, sinks), dtype=np.int64)
            if js.size == 0:
                continue
            pages = np.asarray(page_table[b])[js // PAGE]
            for h in range(heads):
                r = cu_q[b] + i
                k = values[pages, h // group, 0, js % PAGE]
                v = values[pages, h // group, 1, js % PAGE]
                s = scale * (k @ q[r, h])
                top = s.max()
                e = np.exp(s - top)
                w = e / e.sum()
                out[r, h] = w @ v
                spread[r, h] = w @ np.abs(v)
                lse[r, h] = top + math.log(e.sum())
                slack[r, h] = scale * ((np.abs(k) @ np.abs(q[r, h])) * (2 * d + 4) * 2.0 ** -24
                                       + 2.0 ** -17 * np.abs(q[r, h]).max() * np.abs(k).sum(1)).max()
    return out, lse, spread, slack
