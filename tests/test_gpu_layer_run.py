"""The layer's operators run together (examples/decode_layer.py, DecoderLayerX4):
prompt chunks and single tokens, every operator's result against the float64
oracle over what it was given (bounds as tests/test_gpu_layer.py and
tests/test_gpu_attention.py), and the captured step bit for bit the eager one."""

import importlib.util
import os

import numpy as np
import pytest
import torch

import mxfp8_moe_decode_gb300 as M
from mxfp8_moe_decode_gb300 import kv_dequant_x8
from oracle import attention as A
from oracle import layer as L

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("decode_layer", os.path.join(ROOT, "examples", "decode_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _f64(t):
    return t.detach().cpu().double().numpy()


class Seen:
    """The operators' arguments and results, as the step passes them on."""

    def __init__(self, ex, monkeypatch):
        self.calls = []
        for name in ("norm_add_norm_x8", "linear_x4", "rope_kv_append_x8", "attn_x8"):
            monkeypatch.setattr(ex, name, self._wrap(name, getattr(M, name)))

    def _wrap(self, name, fn):
        def call(*a, **kw):
            kept = [t.clone() if torch.is_tensor(t) else t for t in a]
            r = fn(*a, **kw)
            self.calls.append((name, kept, kw, r.clone() if torch.is_tensor(r) else [t.clone() if torch.is_tensor(t) else t for t in r]))
            return r

        return call


def _check_norm(a, kw, r):
    want, block = L.block_residual(_f64(a[0]), _f64(a[1]), _f64(a[2]), _f64(kw["gate"]))
    assert (np.abs(_f64(r[0]) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -17 * (np.abs(block) + np.abs(_f64(a[1])))).all()
    s8, sc, _ = M.attn_seam_x8(r[0], a[3])
    assert torch.equal(r[1], s8) and torch.equal(r[2], sc)


def _check_linear(a, kw, r):
    xc = kw.get("x_codes")
    v = _f64(a[0]) if xc is None else L.mxfp8_rows(a[0].cpu().numpy(), xc.cpu().numpy())
    want, size = L.linear(v, a[1].cpu().numpy(), a[2].cpu().numpy())
    slack = (v.shape[1] / 32 * 2.0 ** -23 + 2.0 ** -19) * size
    if xc is None:
        top = np.abs(v).reshape(len(v), -1, 32).max(-1).repeat(32, 1)
        slack = slack + 2.0 ** -21 * L.linear(top, a[1].cpu().numpy(), a[2].cpu().numpy())[1]
    assert (np.abs(_f64(r) - want) <= 2.0 ** -8 * np.abs(want) + slack).all()


@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3)])
def test_layer_steps(window, sinks, monkeypatch):
    ex = _example()
    dev = torch.device("cuda:0")
    moe = ex.small_moe(dev)
    layer = ex.DecoderLayerX4(moe, heads=10, kv_heads=2, head_dim=128, pages=8, window=window, sinks=sinks)
    freqs = [int(v) % (1 << 64) for v in layer.freqs.tolist()]
    seen = Seen(ex, monkeypatch)
    table = torch.tensor([[5, 0, 3], [1, 7, 2]], dtype=torch.int32, device=dev)
    had = torch.zeros(2, dtype=torch.int32, device=dev)
    g = torch.Generator(device=dev).manual_seed(3)
    for n in (20, 24, 1, 24, 1, 1, 24):
        seen.calls.clear()
        x, r = (torch.randn(2 * n, moe.hidden, generator=g, device=dev).bfloat16() for _ in range(2))
        cu = None if n == 1 else torch.tensor([0, n, 2 * n], dtype=torch.int32, device=dev)
        out, res, attn = layer.step(x, r, table, had, cu_q=cu, max_q=n)
        torch.cuda.synchronize()
        names = [c[0] for c in seen.calls]
        assert names == ["norm_add_norm_x8", "linear_x4", "rope_kv_append_x8", "attn_x8", "linear_x4", "norm_add_norm_x8"]
        norm, qkv, rope, at, o, last = (c[1:] for c in seen.calls)
        _check_norm(*norm)
        _check_linear(*qkv)
        # the turned queries, and the keys' bytes that are those of kv_append_x8
        q, k, v = rope[0][2:5]
        place = [int(h) + i for h in had.tolist() for i in range(n)]
        want = L.rope(_f64(q), place, freqs)
        size = np.abs(_f64(q)) + np.abs(np.roll(_f64(q), 64, -1))
        assert (np.abs(_f64(rope[2][0]) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -21 * size).all()
        b, c = rope[0][0], rope[0][1]
        M.kv_append_x8(b, c, M.rope(k, torch.tensor(place, dtype=torch.int32, device=dev), layer.freqs), v, table, had, cu_q=cu)
        assert torch.equal(b, layer.blocks) and torch.equal(c, layer.codes)
        had += n
        vals = _f64(kv_dequant_x8(layer.blocks, layer.codes))
        want, _, spread, slack = A.attention(_f64(at[0][0]), vals, table.cpu().numpy(), had.tolist(), [0, n, 2 * n],
                                             128 ** -0.5, window, sinks)
        bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -20 + 2 * slack[..., None]) * spread
        assert (np.abs(_f64(attn) - want) <= bound).all()
        _check_linear(*o)
        _check_norm(*last)
        assert torch.equal(res, last[2][0]) and torch.equal(out, moe.step(res)) and torch.isfinite(out).all()
    assert layer.status.item() == 0 and moe.status() == 0


def test_captured_steps():
    """The step captured once and replayed as the cache grows gives the eager steps' bits."""
    ex = _example()
    dev = torch.device("cuda:0")
    moe = ex.small_moe(dev)
    table = torch.arange(8, dtype=torch.int32, device=dev).view(4, 2)
    g = torch.Generator(device=dev).manual_seed(5)
    rows = [[torch.randn(4, moe.hidden, generator=g, device=dev).bfloat16() for _ in range(2)] for _ in range(70)]
    eager, layer = [], ex.DecoderLayerX4(moe, heads=8, kv_heads=2, head_dim=64, pages=8)
    had = torch.zeros(4, dtype=torch.int32, device=dev)
    for x, r in rows:
        eager.append([t.clone() for t in layer.step(x, r, table, had)])
        had += 1
    blocks, codes = layer.blocks.clone(), layer.codes.clone()
    layer = ex.DecoderLayerX4(moe, heads=8, kv_heads=2, head_dim=64, pages=8)
    had.zero_()
    x, r = (t.clone() for t in rows[0])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        layer.step(x, r, table, had)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = layer.step(x, r, table, had)
        had += 1
    had.zero_()
    for (a, b), want in zip(rows, eager):
        x.copy_(a), r.copy_(b)
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(got, want))
    # (what no sequence holds of a page is unspecified)
    assert torch.equal(codes, layer.codes)
    held = lambda t, c: kv_dequant_x8(t, c).view(4, 2, 2, 2, 64, 64).permute(0, 2, 3, 1, 4, 5).reshape(4, 2, 2, 128, 64)[:, :, :, :70]  # noqa: E731
    assert torch.equal(held(blocks, codes), held(layer.blocks, layer.codes))
    assert layer.status.item() == 0 and moe.status() == 0


def test_example_runs(monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["decode_layer.py", "--steps", "40", "--x4"])
    _example().main()
    assert "us a step" in capsys.readouterr().out
