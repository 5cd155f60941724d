"""Products with 4-bit weights, on torch tensors: a layer's projections in MXFP4.

Argument marshalling only, in compiled code, as :mod:`.attention`.
"""

from __future__ import annotations

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


def linear_x4_workspace_bytes(rows: int, cols: int, mxfp8: bool) -> int:
    """Bytes of workspace that :func:`linear_x4` needs for x [rows, cols]."""
    return _lib.lib().moe_linear_x4_workspace_bytes(rows, cols, _lib.LINEAR_MXFP8 if mxfp8 else _lib.LINEAR_BF16)
