"""Refusals of the layer's operators (norms around a block, rotary positions,
products with 4-bit weights): CPU only, every check comes before anything is
enqueued; and of the Python bindings."""

import os
import re

import pytest
import torch

import mxfp8_moe_decode_gb300 as M
from mxfp8_moe_decode_gb300 import _lib
from mxfp8_moe_decode_gb300._lib import (MOE_ERR_ALIGN, MOE_ERR_ARG, MOE_ERR_RANGE, MOE_ERR_UNSUPPORTED, MOE_OK,
                                         KvCache, KvSeqs, RopeSpec)

P = [0x100000 * (i + 1) for i in range(12)]  # stand-ins for device pointers, never read
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def L():
    from mxfp8_moe_decode_gb300 import build
    build.build()
    return _lib.lib()


def test_constants_match_the_header():
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe_decode.h")).read()
    val = dict(re.findall(r"#define (MOE_LINEAR_\w+) (\d+)", src))
    for name in ("LINEAR_BF16", "LINEAR_MXFP8", "LINEAR_STATUS_TIMEOUT"):
        assert int(val["MOE_" + name]) == getattr(_lib, name)


def test_norm_add_norm_refusals(L):
    def call(x=P[0], ldx=256, r=P[1], ldr=256, g=P[2], ldg=256, pw=P[3], w=P[4], m=4, h=256, rs=1.0, bs=1.0, eps=1e-6,
             res=P[5], x8=P[6], c=P[7], n=P[8]):
        return L.moe_norm_add_norm_x8(x, ldx, r, ldr, g, ldg, pw, w, m, h, rs, bs, eps, res, x8, c, n, None)

    assert call(m=-1) == MOE_ERR_RANGE
    assert call(m=0, x=None) == MOE_OK
    for h in (0, 16, 100, 8224):
        assert call(h=h, ldx=9000, ldr=9000, ldg=9000) == MOE_ERR_UNSUPPORTED
    for v in (-1e-6, NAN):
        assert call(eps=v) == MOE_ERR_ARG
    for v in (NAN, INF, -INF):
        assert call(rs=v) == MOE_ERR_ARG and call(bs=v) == MOE_ERR_ARG
    for name in ("x", "r", "w", "res", "x8", "c"):
        assert call(**{name: None}) == MOE_ERR_ARG, name
    for name in ("x", "r", "g", "pw", "w", "res", "x8", "n"):
        assert call(**{name: P[9] + 8}) == MOE_ERR_ALIGN, name
    for name in ("ldx", "ldr", "ldg"):
        assert call(**{name: 248}) == MOE_ERR_ARG, name
        assert call(**{name: 260}) == MOE_ERR_ALIGN, name
    assert call(res=P[1], ldr=512) == MOE_ERR_ARG and call(res=P[0], ldx=512) == MOE_ERR_ARG


def _spec(**kw):
    a = dict(freqs=P[9], first=0, rot=64, interleaved=0, scale=1.0)
    a.update(kw)
    return RopeSpec(*a.values())


SPECS = [(dict(rot=0), MOE_ERR_UNSUPPORTED), (dict(rot=24), MOE_ERR_UNSUPPORTED), (dict(rot=144), MOE_ERR_UNSUPPORTED),
         (dict(rot=-16), MOE_ERR_UNSUPPORTED), (dict(first=-8), MOE_ERR_UNSUPPORTED), (dict(first=4), MOE_ERR_UNSUPPORTED),
         (dict(first=72), MOE_ERR_UNSUPPORTED), (dict(first=2 ** 31 - 8), MOE_ERR_UNSUPPORTED),
         (dict(scale=NAN), MOE_ERR_ARG), (dict(scale=INF), MOE_ERR_ARG), (dict(freqs=None), MOE_ERR_ARG),
         (dict(freqs=P[9] + 8), MOE_ERR_ALIGN)]


def test_rope_refusals(L):
    def call(spec=None, x=P[0], ldx=512, tokens=3, heads=4, dim=128, pos=P[1], out=P[2], ldo=512):
        return L.moe_rope(spec or _spec(), x, ldx, tokens, heads, dim, pos, out, ldo, None)

    for kw, code in SPECS:
        assert call(spec=_spec(**kw)) == code, kw
    assert L.moe_rope(None, P[0], 512, 3, 4, 128, P[1], P[2], 512, None) == MOE_ERR_ARG
    assert call(tokens=0, x=None) == MOE_OK
    assert call(tokens=-1) == MOE_ERR_RANGE and call(tokens=(1 << 24) + 1) == MOE_ERR_RANGE
    for dim in (0, 8, 120, 1040):
        assert call(dim=dim, spec=_spec(rot=16)) == MOE_ERR_UNSUPPORTED
    assert call(heads=0) == MOE_ERR_UNSUPPORTED and call(heads=4097, ldx=1 << 20, ldo=1 << 20) == MOE_ERR_UNSUPPORTED
    for name in ("x", "pos", "out"):
        assert call(**{name: None}) == MOE_ERR_ARG, name
    assert call(x=P[0] + 8) == MOE_ERR_ALIGN and call(out=P[2] + 2) == MOE_ERR_ALIGN and call(pos=P[1] + 2) == MOE_ERR_ALIGN
    for name in ("ldx", "ldo"):
        assert call(**{name: 504}) == MOE_ERR_ARG and call(**{name: 516}) == MOE_ERR_ALIGN
    assert call(out=P[0], ldo=1024) == MOE_ERR_ARG  # in place only with one stride
    # more CTAs than a grid holds
    assert call(tokens=1 << 24, heads=4096, dim=1024, ldx=1 << 22, ldo=1 << 22) == MOE_ERR_UNSUPPORTED


def _cache(**kw):
    a = dict(blocks=P[0], codes=P[1], pages=10, kv_heads=2, head_dim=128)
    a.update(kw)
    return KvCache(*a.values())


def _seqs(**kw):
    a = dict(page_table=P[2], lens=P[3], cu_q=P[4], seqs=3, tokens=5, max_pages=4, max_q=1)
    a.update(kw)
    return KvSeqs(*a.values())


def test_rope_append_refusals(L):
    def call(c=None, s=None, spec=None, pos=P[5], q=P[6], ldq=1024, heads=8, out=P[7], ldo=1024, k=P[8], ldk=256,
             v=P[10], ldv=256, status=None):
        return L.moe_rope_kv_append_x8(c or _cache(), s or _seqs(), spec or _spec(), pos, q, ldq, heads, out, ldo, k, ldk,
                                       v, ldv, status, None)

    for kw, code in SPECS:
        assert call(spec=_spec(**kw)) == code, kw
    assert L.moe_rope_kv_append_x8(_cache(), _seqs(), None, P[5], P[6], 1024, 8, P[7], 1024, P[8], 256, P[10], 256, None,
                                   None) == MOE_ERR_ARG
    assert call(c=_cache(head_dim=96)) == MOE_ERR_UNSUPPORTED and call(c=_cache(blocks=None)) == MOE_ERR_ARG
    assert call(s=_seqs(tokens=-1)) == MOE_ERR_RANGE and call(s=_seqs(cu_q=None)) == MOE_ERR_ARG
    assert call(s=_seqs(tokens=0), q=None, k=None) == MOE_OK
    assert call(heads=0) == MOE_ERR_UNSUPPORTED and call(heads=4097, ldq=1 << 20, ldo=1 << 20) == MOE_ERR_UNSUPPORTED
    for name in ("q", "out", "k", "v"):
        assert call(**{name: None}) == MOE_ERR_ARG, name
        assert call(**{name: P[11] + 8}) == MOE_ERR_ALIGN, name
    assert call(pos=P[5] + 2) == MOE_ERR_ALIGN and call(status=P[5] + 2) == MOE_ERR_ALIGN
    for name, low, odd in (("ldq", 1016, 1028), ("ldo", 1016, 1028), ("ldk", 248, 260), ("ldv", 248, 260)):
        assert call(**{name: low}) == MOE_ERR_ARG and call(**{name: odd}) == MOE_ERR_ALIGN
    assert call(out=P[6], ldo=2048) == MOE_ERR_ARG


def test_linear_refusals(L):
    def call(x=P[0], ldx=256, xc=P[1], m=4, w=P[2], wc=P[3], n=100, k=256, out=P[4], ldo=100, ws=P[5], size=1 << 30,
             status=None):
        return L.moe_linear_x4(x, ldx, xc, m, w, wc, n, k, out, ldo, ws, size, status, None)

    assert call(m=-1) == MOE_ERR_RANGE and call(m=(1 << 20) + 1) == MOE_ERR_RANGE
    assert call(n=-1) == MOE_ERR_RANGE and call(n=(1 << 24) + 1) == MOE_ERR_RANGE
    for k in (0, 32, 64, 192, -128, (1 << 16) + 128):
        assert call(k=k, ldx=1 << 20) == MOE_ERR_UNSUPPORTED
    assert call(m=0, x=None) == MOE_OK and call(n=0, w=None) == MOE_OK
    for name in ("x", "w", "wc", "out"):
        assert call(**{name: None}) == MOE_ERR_ARG, name
    for name, by in (("x", 8), ("w", 16), ("wc", 2), ("out", 1), ("xc", 2), ("ws", 8), ("status", 2)):
        assert call(**{name: P[9] + by}) == MOE_ERR_ALIGN, name
    assert call(ldx=240) == MOE_ERR_ARG and call(ldo=99) == MOE_ERR_ARG
    assert call(out=P[0]) == MOE_ERR_ARG  # in place
    assert call(ldx=264) == MOE_ERR_ALIGN           # bytes: 16 at a time
    assert call(xc=None, ldx=260) == MOE_ERR_ALIGN  # bf16: 8 values at a time
    # bf16 rows need a workspace, MXFP8 rows none
    need = L.moe_linear_x4_workspace_bytes(4, 256, _lib.LINEAR_BF16)
    assert need >= 2 * 4 * (256 + 8) and L.moe_linear_x4_workspace_bytes(4, 256, _lib.LINEAR_MXFP8) == 0
    assert L.moe_linear_x4_workspace_bytes(0, 256, _lib.LINEAR_BF16) == 0
    assert L.moe_linear_x4_workspace_bytes(-1, 256, _lib.LINEAR_BF16) == 0
    assert call(xc=None, ws=None) == MOE_ERR_ARG and call(xc=None, size=need - 1) == MOE_ERR_ARG
    assert M.linear_x4_workspace_bytes(4, 256, mxfp8=False) == need


def test_linear_shape_refusals(L):
    def call(m=4, n=100, k=256, form=_lib.LINEAR_BF16, shape=None):
        return L.moe_linear_x4_shape(m, n, k, form, shape or _lib.LinearShape())

    for v in (0, -1, (1 << 20) + 1):
        assert call(m=v) == MOE_ERR_RANGE
    for v in (0, -1, (1 << 24) + 1):
        assert call(n=v) == MOE_ERR_RANGE
    for v in (0, 64, 192, -128, (1 << 16) + 128):
        assert call(k=v) == MOE_ERR_UNSUPPORTED
    assert call(form=2) == MOE_ERR_ARG and call(form=-1) == MOE_ERR_ARG
    assert L.moe_linear_x4_shape(4, 100, 256, 0, None) == MOE_ERR_ARG
    src = open(os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "include", "moe_decode.h")).read()
    body = re.search(r"typedef struct moe_linear_shape \{(.*?)\} moe_linear_shape;", src, re.S)[1]
    assert re.findall(r"int (\w+);", body) == [name for name, _ in _lib.LinearShape._fields_]


def test_bindings_refuse_host_tensors_and_shapes():
    x = torch.zeros(2, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        M.norm_add_norm_x8(x, x, x[0], x[0])
    f, i = torch.zeros(8, dtype=torch.int64), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):
        M.rope(x.view(2, 1, 64), i, f)
    with pytest.raises(ValueError):
        M.linear_x4(x, torch.zeros(4, 32, dtype=torch.uint8), torch.zeros(4, 2, dtype=torch.uint8))
    blocks, codes = torch.zeros(1, 1, 2, 64 * 64, dtype=torch.uint8), torch.zeros(1, 1, 2, dtype=torch.uint8)
    k = torch.zeros(1, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError):
        M.rope_kv_append_x8(blocks, codes, k, k, k, i.view(1, 2), i[:1], f)
