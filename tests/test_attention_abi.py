"""Refusals of the attention side's entry points (CPU only: every check comes
before anything is enqueued) and of the Python binding."""

import ctypes

import pytest
import torch

import mxfp8_moe_decode_gb300 as M
from mxfp8_moe_decode_gb300 import _lib
from mxfp8_moe_decode_gb300._lib import (MOE_ERR_ALIGN, MOE_ERR_ARG, MOE_ERR_RANGE,
                                         MOE_ERR_UNSUPPORTED, MOE_OK, KvCache, KvSeqs)

P = [0x100000 * (i + 1) for i in range(12)]  # stand-ins for device pointers, never read


@pytest.fixture(scope="module")
def L():
    from mxfp8_moe_decode_gb300 import build
    build.build()
    return _lib.lib()


def test_constants_match_the_header():
    import os
    import re
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))),
                            "include", "moe_decode.h")).read()
    val = dict(re.findall(r"#define (MOE_\w+) \(?(\d+)", src))
    assert int(val["MOE_KV_PAGE_TOKENS"]) == _lib.KV_PAGE_TOKENS
    assert int(val["MOE_ATTN_X8_WORKSPACE_BYTES"]) << 20 == _lib.ATTN_X8_WORKSPACE_BYTES
    for bit in ("TIMEOUT", "PAGE", "LENGTH"):
        assert int(val["MOE_KV_STATUS_" + bit]) == getattr(_lib, "KV_STATUS_" + bit)


def test_add_norm_refusals(L):
    def call(x=P[0], ldx=256, r=P[1], ldr=256, w=P[2], m=4, h=256, eps=1e-6, res=P[3], x8=P[4],
             c=P[5], n=P[6]):
        return L.moe_add_norm_x8(x, ldx, r, ldr, w, m, h, eps, res, x8, c, n, None)

    assert call(m=-1) == MOE_ERR_RANGE
    assert call(m=0, x=None) == MOE_OK  # no rows: nothing is looked at
    for h in (0, 16, 100, 8224):
        assert call(h=h, ldx=9000, ldr=9000) == MOE_ERR_UNSUPPORTED
    for eps in (-1e-6, float("nan")):
        assert call(eps=eps) == MOE_ERR_ARG
    for name in ("x", "r", "w", "res", "x8", "c"):
        assert call(**{name: None}) == MOE_ERR_ARG, name
    for name in ("x", "r", "w", "res", "x8", "n"):
        assert call(**{name: P[7] + 8}) == MOE_ERR_ALIGN, name
    assert call(ldx=248) == MOE_ERR_ARG and call(ldr=248) == MOE_ERR_ARG
    assert call(ldx=260) == MOE_ERR_ALIGN and call(ldr=260) == MOE_ERR_ALIGN
    assert call(res=P[1], ldr=512) == MOE_ERR_ARG and call(res=P[0], ldx=512) == MOE_ERR_ARG


def _cache(**kw):
    a = dict(blocks=P[0], codes=P[1], pages=10, kv_heads=2, head_dim=128)
    a.update(kw)
    return KvCache(*a.values())


def _seqs(**kw):
    a = dict(page_table=P[2], lens=P[3], cu_q=P[4], seqs=3, tokens=5, max_pages=4, max_q=2)
    a.update(kw)
    return KvSeqs(*a.values())


SHARED = [
    (dict(head_dim=96), {}, MOE_ERR_UNSUPPORTED), (dict(head_dim=0), {}, MOE_ERR_UNSUPPORTED),
    (dict(kv_heads=0), {}, MOE_ERR_UNSUPPORTED), (dict(kv_heads=1025), {}, MOE_ERR_UNSUPPORTED),
    (dict(pages=0), {}, MOE_ERR_ARG), ({}, dict(max_pages=0), MOE_ERR_ARG),
    ({}, dict(tokens=-1), MOE_ERR_RANGE), ({}, dict(seqs=-1), MOE_ERR_RANGE),
    ({}, dict(tokens=(1 << 24) + 1), MOE_ERR_RANGE), ({}, dict(seqs=(1 << 20) + 1), MOE_ERR_RANGE),
    ({}, dict(cu_q=None), MOE_ERR_ARG),  # 5 rows for 3 sequences of one token each
    ({}, dict(seqs=0), MOE_ERR_ARG),
    (dict(blocks=None), {}, MOE_ERR_ARG), (dict(codes=None), {}, MOE_ERR_ARG),
    ({}, dict(page_table=None), MOE_ERR_ARG), ({}, dict(lens=None), MOE_ERR_ARG),
    (dict(blocks=P[0] + 8), {}, MOE_ERR_ALIGN), (dict(codes=P[1] + 1), {}, MOE_ERR_ALIGN),
    ({}, dict(page_table=P[2] + 2), MOE_ERR_ALIGN), ({}, dict(lens=P[3] + 1), MOE_ERR_ALIGN),
    ({}, dict(cu_q=P[4] + 2), MOE_ERR_ALIGN),
]


@pytest.mark.parametrize("cache,seqs,code", SHARED)
def test_cache_refusals(L, cache, seqs, code):
    c, s = _cache(**cache), _seqs(**seqs)
    assert L.moe_kv_append_x8(c, s, P[5], 256, P[6], 256, None, None) == code
    assert L.moe_attn_x8(c, s, P[5], 1024, 8, 0.1, 0, 0, P[6], None, P[7], 48 << 20, None, None) == code


def test_append_refusals(L):
    def call(k=P[5], ldk=256, v=P[6], ldv=256, status=None, c=None, s=None):
        return L.moe_kv_append_x8(c or _cache(), s or _seqs(), k, ldk, v, ldv, status, None)

    assert L.moe_kv_append_x8(None, _seqs(), P[5], 256, P[6], 256, None, None) == MOE_ERR_ARG
    assert L.moe_kv_append_x8(_cache(), None, P[5], 256, P[6], 256, None, None) == MOE_ERR_ARG
    assert call(s=_seqs(tokens=0), k=None) == MOE_OK
    assert call(k=None) == MOE_ERR_ARG and call(v=None) == MOE_ERR_ARG
    assert call(k=P[5] + 8) == MOE_ERR_ALIGN and call(v=P[6] + 2) == MOE_ERR_ALIGN
    assert call(ldk=260) == MOE_ERR_ALIGN and call(ldv=260) == MOE_ERR_ALIGN
    assert call(status=P[8] + 2) == MOE_ERR_ALIGN
    assert call(ldk=248) == MOE_ERR_ARG and call(ldv=248) == MOE_ERR_ARG


def test_attention_refusals(L):
    def call(q=P[5], ldq=1024, heads=8, scale=0.1, window=0, sinks=0, out=P[6], lse=None, ws=P[7],
             size=48 << 20, status=None, s=None):
        return L.moe_attn_x8(_cache(), s or _seqs(), q, ldq, heads, scale, window, sinks, out, lse,
                             ws, size, status, None)

    assert call(s=_seqs(tokens=0), q=None) == MOE_OK
    assert call(heads=0) == MOE_ERR_ARG and call(heads=7) == MOE_ERR_ARG
    assert call(heads=514, ldq=514 * 128) == MOE_ERR_UNSUPPORTED
    for scale in (0.0, -1.0, float("nan"), float("inf")):
        assert call(scale=scale) == MOE_ERR_ARG
    assert call(window=-1) == MOE_ERR_ARG and call(sinks=-1) == MOE_ERR_ARG
    assert call(s=_seqs(max_q=0)) == MOE_ERR_ARG
    for name in ("q", "out", "ws"):
        assert call(**{name: None}) == MOE_ERR_ARG, name
    for name in ("q", "out", "ws"):
        assert call(**{name: P[9] + 8}) == MOE_ERR_ALIGN, name
    assert call(ldq=1028) == MOE_ERR_ALIGN
    assert call(lse=P[8] + 2) == MOE_ERR_ALIGN and call(status=P[8] + 2) == MOE_ERR_ALIGN
    assert call(ldq=1016) == MOE_ERR_ARG


@pytest.mark.parametrize("kv_heads,group,max_pages,seqs,max_q,refused", [
    # one row a sequence: an item of 1 page takes 1 + 10 positions, (2^20 / 8 + 2^20) * kv_heads items at most
    (200, 1, 1, 1 << 20, 1, True), (166, 1, 1, 1 << 20, 1, True), (165, 1, 1, 1 << 20, 1, False),
    (108, 1, 7, 1 << 20, 1, True), (107, 1, 7, 1 << 20, 1, False),
    (16, 1, 100, 1 << 20, 1, False), (17, 1, 100, 1 << 20, 1, True),
    (1, 256, 1, 1 << 16, 1, True), (1, 256, 1, (1 << 16) - 1, 1, False),  # tokens * group^2 beside it
])
def test_attention_work_list_fits_32_bits(L, kv_heads, group, max_pages, seqs, max_q, refused):
    c = _cache(kv_heads=kv_heads, head_dim=64)
    s = _seqs(cu_q=None, seqs=seqs, tokens=seqs, max_pages=max_pages, max_q=max_q)
    heads = kv_heads * group
    # (a workspace of no bytes: what is not refused here is refused for that, or for want of a GPU)
    rc = L.moe_attn_x8(c, s, P[5], heads * 64, heads, 0.1, 0, 0, P[6], None, P[7], 0, None, None)
    assert (rc == MOE_ERR_UNSUPPORTED) == refused, rc


def test_attention_scale_is_finite_in_log2_units(L):
    """Scores are computed times log2 e: a scale that is infinite there is refused
    (it made NaN of scores of 0). No rows: nothing else is looked at."""
    def call(scale):
        return L.moe_attn_x8(_cache(), _seqs(tokens=0), None, 1024, 8, scale, 0, 0, None, None, None, 0, None, None)

    assert call(3e38) == MOE_ERR_ARG and call(2.4e38) == MOE_ERR_ARG
    assert call(2.3e38) == MOE_OK


def test_binding_refuses_host_tensors_and_shapes():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        M.add_norm_x8(x, x, x[0])
    blocks, codes = torch.zeros(1, 1, 2, 64 * 64, dtype=torch.uint8), torch.zeros(1, 1, 2, dtype=torch.uint8)
    k = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    i = torch.zeros(1, 1, dtype=torch.int32)
    with pytest.raises(ValueError):
        M.kv_append_x8(blocks, codes, k, k, i, i[0])
    with pytest.raises(ValueError):
        M.attn_x8(k, blocks, codes, i, i[0])
