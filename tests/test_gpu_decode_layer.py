"""The decoder layer's step (examples/decode_layer.py): prompt chunks, then
single tokens, each step's attention rows against the float64 oracle over the
cache as it stands (bounds as tests/test_gpu_attention.py), the residual
additions and the FFN half as the operators alone give them."""

import importlib.util
import os

import numpy as np
import pytest
import torch

from mxfp8_moe_decode_gb300 import kv_dequant_x8
from oracle import attention as A

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("decode_layer", os.path.join(ROOT, "examples", "decode_layer.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _f64(t):
    return t.detach().cpu().double().numpy()


@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 3)])
def test_layer_steps(window, sinks):
    ex = _example()
    dev = torch.device("cuda:0")
    moe = ex.small_moe(dev)
    layer = ex.DecoderLayer(moe, heads=10, kv_heads=2, head_dim=128, pages=8, window=window, sinks=sinks)
    table = torch.tensor([[5, 0, 3], [1, 7, 2]], dtype=torch.int32, device=dev)
    had = torch.zeros(2, dtype=torch.int32, device=dev)
    g = torch.Generator(device=dev).manual_seed(3)
    for n in (20, 24, 1, 24, 1, 1, 24):
        x, r = (torch.randn(2 * n, moe.hidden, generator=g, device=dev).bfloat16() for _ in range(2))
        cu = None if n == 1 else torch.tensor([0, n, 2 * n], dtype=torch.int32, device=dev)
        out, res, attn = layer.step(x, r, table, had, cu_q=cu, max_q=n)
        had += n
        torch.cuda.synchronize()
        # the rows of q as the step made them, over the cache after the append
        normed = torch.empty_like(x)
        res1, _, _, _ = ex.add_norm_x8(x, r, layer.norm_w, normed=normed)
        assert np.array_equal(_f64(res1), A.add(_f64(x), _f64(r)))
        q = (normed @ layer.w_qkv).view(2 * n, -1, 128)[:, :10]
        lens = had.tolist()
        vals = _f64(kv_dequant_x8(layer.blocks, layer.codes))
        want, _, spread, slack = A.attention(_f64(q), vals, table.cpu().numpy(), lens, [0, n, 2 * n], 128 ** -0.5,
                                             window, sinks)
        bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -20 + 2 * slack[..., None]) * spread
        assert (np.abs(_f64(attn) - want) <= bound).all()
        assert torch.equal(res, res1 + attn.view(2 * n, -1) @ layer.w_o)
        assert torch.equal(out, moe.step(res))
        assert torch.isfinite(out).all()
    assert layer.status.item() == 0 and moe.status() == 0


def test_example_runs(monkeypatch, capsys):
    monkeypatch.setattr("sys.argv", ["decode_layer.py", "--steps", "40"])
    _example().main()
    assert "us a step" in capsys.readouterr().out
