"""The rest of a decoder layer in float64: the norms around a block with its
gate, rotary positions, and products with MXFP4 weights.

TEST INFRASTRUCTURE ONLY (see the package header).

The source pages show none of these bodies; the formulas are the operators' own
definitions:

* ``block_residual``: res_scale * residual + block_scale * gate * RMSNorm(x) * post_w,
  unrounded (the norm of the rounded sum is :mod:`oracle.moe` ``attn_norm``);
* ``turns``: the angle of a position from whole numbers, position * frequency
  modulo 2^64, one Python integer at a time;
* ``rope``: pairs of a head turned one after the other, unrounded;
* ``linear``: x times the dequantised rows (:mod:`oracle.mx` ``dequant_fp4_rows``).

Pins: tests/test_oracle_layer.py (hand-worked cases).
"""

from __future__ import annotations

import math

import numpy as np

from .mx import dequant_fp4_rows, mx_scale
from .numerics import e4m3_decode


def block_residual(x, residual, post_w=None, gate=None, res_scale=1.0, block_scale=1.0, eps=1e-6):
    """(the unrounded new residual rows, the block's part of them), float64 [rows, hidden]."""
    x = np.asarray(x, np.float64)
    b = x
    if post_w is not None:
        power = np.array([math.fsum(v * v for v in row) / len(row) for row in x])
        b = x / np.sqrt(power + eps)[:, None] * np.asarray(post_w, np.float64)
    if gate is not None:
        b = b * np.asarray(gate, np.float64)
    b = block_scale * b
    return res_scale * np.asarray(residual, np.float64) + b, b


def turns(position: int, freq: int) -> float:
    """position * freq * 2^-64 turns, without the whole ones."""
    return ((position * freq) % (1 << 64)) / float(1 << 64)


def rope(x, positions, freqs, first=0, interleaved=False, scale=1.0):
    """float64 [tokens, heads, d] turned; freqs: whole numbers (unsigned 64 bits)."""
    out = np.array(x, np.float64)
    n = len(freqs)
    for t, pos in enumerate(positions):
        for i, f in enumerate(freqs):
            a = 2.0 * math.pi * turns(int(pos), int(f))
            c, s = scale * math.cos(a), scale * math.sin(a)
            u, v = (first + 2 * i, first + 2 * i + 1) if interleaved else (first + i, first + n + i)
            p, q = np.asarray(x, np.float64)[t, :, u], np.asarray(x, np.float64)[t, :, v]
            out[t, :, u] = p * c - q * s
            out[t, :, v] = q * c + p * s
    return out


def mxfp8_rows(b, codes):
    """E4M3 bytes [rows, k] with a code per 32 columns -> float64."""
    return e4m3_decode(b) * np.repeat(mx_scale(codes), 32, axis=1)


def linear(x, w, w_codes):
    """(x w^T, |x| |w|^T) in float64; x float64 [m, k], w packed E2M1 [n, k / 2]."""
    d = dequant_fp4_rows(w, w_codes)
    return np.asarray(x, np.float64) @ d.T, np.abs(np.asarray(x, np.float64)) @ np.abs(d).T
