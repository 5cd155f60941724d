"""GB300 (sm_103a) MXFP8 MoE decode step: the FFN half of one decode step.

``MoeDecode`` and ``attn_seam_x8`` (mxfp8_moe_decode_gb300.api) wrap the C ABI of
libmoe_decode.so (include/moe_decode.h), as do the attention side's operators
``add_norm_x8``, ``norm_add_norm_x8``, ``rope``, ``kv_append_x8``, ``rope_kv_append_x8`` and
``attn_x8`` (mxfp8_moe_decode_gb300.attention) and the products with MXFP4 weights
``linear_x4`` (mxfp8_moe_decode_gb300.linear);
``workloads`` draws seeded synthetic inputs; ``build`` compiles the library and the
attention side's argument marshalling (csrc/host.cpp) in-tree.
"""

from .api import MoeDecode, attn_seam_x8, expected_shapes, kernel_names  # noqa: F401
from .attention import (add_norm_x8, attn_x8, attn_x8_workspace, kv_append_x8,  # noqa: F401
                        kv_cache_x8, kv_dequant_x8, norm_add_norm_x8, rope, rope_freqs, rope_kv_append_x8)
from .linear import dequant_x4, linear_x4, linear_x4_workspace_bytes, quant_x4  # noqa: F401
