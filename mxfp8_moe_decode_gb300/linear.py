"""Products with 4-bit weights, on torch tensors: a layer's projections in MXFP4.

Argument marshalling only, in compiled code, as :mod:`.attention`.
"""

from __future__ import annotations

import math

import torch

from . import attention, _lib
from .attention import _result


def linear_x4(x: torch.Tensor, w: torch.Tensor, w_codes: torch.Tensor, x_codes: torch.Tensor | None = None,
              out: torch.Tensor | None = None, workspace: torch.Tensor | None = None,
              status: torch.Tensor | None = None) -> torch.Tensor:
    """out = x w^T in bf16 [M, N] (``moe_linear_x4``), for any number of rows.

    w: uint8 [N, K / 2], two E2M1 codes a byte (column 2 j in the low nibble of
    byte j), w_codes uint8 [N, K / 32], one E8M0 code per row per 32 columns (the
    form of ``MoeDecode(routed="e2m1")``'s experts). x: bf16 [M, K], or with
    x_codes (uint8 [M, K / 32]) MXFP8 rows, uint8 [M, K], as :func:`add_norm_x8`
    returns them. Rows of x and out may be strided. ``workspace``: a uint8 tensor
    of at least :func:`linear_x4_workspace_bytes` (None: allocated for the call),
    ``status``: int32 [1], ``LINEAR_STATUS_TIMEOUT`` of :mod:`._lib`.
    """
    return _result((attention._bound or attention._host()).linear_x4(x, w, w_codes, x_codes, out, workspace, status),
                   "moe_linear_x4")


def quant_x4(w: torch.Tensor) -> tuple[torch.Tensor, torch.Tensor]:
    """(uint8 [N, K / 2], uint8 [N, K / 32]) of weights [N, K] in MXFP4 (torch
    operations, any device): per 32 columns the smallest scale 2^(code - 127) under
    which no value passes E2M1's largest, 6, and the nearest E2M1 values, ties to
    the even code. For finite weights; K a multiple of 32."""
    if w.dim() != 2 or w.shape[1] % 32:
        raise ValueError(f"w must be [N, K] with K a multiple of 32, got {tuple(w.shape)}")
    n, k = w.shape
    packed = torch.empty(n, k // 2, dtype=torch.uint8, device=w.device)
    codes = torch.empty(n, k // 32, dtype=torch.uint8, device=w.device)
    # the borders between E2M1's values; at .75, 1.75 and 3.5 the even code is the upper one
    border = [0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0]
    border = [math.nextafter(b, 0.0) if b in (0.75, 1.75, 3.5) else b for b in border]
    border = torch.tensor(border, dtype=torch.float64, device=w.device)
    step = max(1, (1 << 24) // max(k, 1))  # (rows at a time: what 64 bits take stays below a GB)
    for lo in range(0, n, step):
        groups = w[lo:lo + step].double().reshape(-1, k // 32, 32)
        m, e = torch.frexp(groups.abs().amax(-1) / 6.0)
        code = (torch.where(m == 0.5, e - 1, e) + 127).clamp(0, 254) * (m > 0)  # a group of zeros: 0
        v = groups * torch.exp2(127.0 - code.double())[..., None]
        nibble = torch.bucketize(v.abs().contiguous(), border)
        nibble = (nibble + 8 * torch.signbit(v)).to(torch.uint8).view(-1, k // 2, 2)
        packed[lo:lo + step] = nibble[..., 0] | (nibble[..., 1] << 4)
        codes[lo:lo + step] = code.to(torch.uint8)
    return packed, codes


def dequant_x4(w: torch.Tensor, w_codes: torch.Tensor) -> torch.Tensor:
    """The values that MXFP4 rows stand for, fp32 [N, K], NaN under the code 255
    (for tests and inspection: torch operations, any device)."""
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], device=w.device)
    table = torch.cat((table, -table))
    v = torch.stack((table[(w & 15).long()], table[(w >> 4).long()]), -1).view(*w_codes.shape, 32)
    scale = torch.exp2(w_codes.double() - 127).masked_fill(w_codes == 255, math.nan)
    return (v.double() * scale[..., None]).float().flatten(1)


def linear_x4_workspace_bytes(rows: int, cols: int, mxfp8: bool) -> int:
    """Bytes of workspace that :func:`linear_x4` needs for x [rows, cols]."""
    return _lib.lib().moe_linear_x4_workspace_bytes(rows, cols, _lib.LINEAR_MXFP8 if mxfp8 else _lib.LINEAR_BF16)


def linear_x4_shape(rows: int, cols: int, out: int, mxfp8: bool, device="cuda") -> dict:
    """How :func:`linear_x4` lays out x [rows, cols] onto ``out`` columns on a
    device (``moe_linear_shape``; for tests and inspection)."""
    shape = _lib.LinearShape()
    with torch.cuda.device(device):
        rc = _lib.lib().moe_linear_x4_shape(rows, out, cols, _lib.LINEAR_MXFP8 if mxfp8 else _lib.LINEAR_BF16, shape)
    _result(rc, "moe_linear_x4_shape")
    return {name: getattr(shape, name) for name, _ in shape._fields_}
