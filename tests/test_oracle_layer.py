"""Hand-worked pins of oracle.layer, and of the frequencies a program makes for
the rotary positions (CPU)."""

import math

import numpy as np
import pytest

import torch

from mxfp8_moe_decode_gb300 import dequant_x4, quant_x4, rope_freqs
from oracle import layer as L
from oracle.mx import dequant_fp4_rows


def test_block_residual():
    x, r = np.array([[3.0, 4.0]]), np.array([[1.0, -1.0]])
    # rms = sqrt((9 + 16) / 2) = 5 / sqrt 2
    res, b = L.block_residual(x, r, np.array([2.0, 1.0]), np.array([0.5, 3.0]), 0.5, 2.0, eps=0.0)
    want = 2.0 * np.array([[0.5 * 2.0 * 3.0, 3.0 * 4.0]]) * math.sqrt(2) / 5
    assert np.allclose(b, want, rtol=1e-15) and np.allclose(res, 0.5 * r + want, rtol=1e-15)
    res, b = L.block_residual(x, r)
    assert np.array_equal(b, x) and np.array_equal(res, x + r)


def test_turns_are_whole_numbers():
    assert L.turns(3, 1 << 62) == 0.75
    assert L.turns(5, 1 << 62) == 0.25
    assert L.turns(-1, 1 << 62) == 0.75
    assert L.turns((1 << 31) - 1, (1 << 33) + 1) == (((1 << 31) - 1) * ((1 << 33) + 1) % (1 << 64)) / 2.0 ** 64


@pytest.mark.parametrize("interleaved", [False, True])
def test_rope_by_quarter_turns(interleaved):
    x = np.arange(1.0, 9.0).reshape(1, 1, 8)
    # pair 0 by a quarter turn, pair 1 by a half turn; the last four dims stay
    out = L.rope(x, [1], [1 << 62, 1 << 63], 0, interleaved, 2.0)[0, 0]
    u, v = ([0, 2], [1, 3]) if interleaved else ([0, 1], [2, 3])
    want = x[0, 0].copy()
    want[u[0]], want[v[0]] = -2 * x[0, 0, v[0]], 2 * x[0, 0, u[0]]
    want[u[1]], want[v[1]] = -2 * x[0, 0, u[1]], -2 * x[0, 0, v[1]]
    assert np.allclose(out, want, atol=1e-14)


def test_linear_by_hand():
    # one row of 32 columns: 1.5 at column 0, -6 at column 1, 0.5 at column 31, scale 2
    w = np.zeros((1, 16), np.uint8)
    w[0, 0], w[0, 15] = 0x3 | (0xF << 4), 0x1 << 4
    x = np.zeros((1, 32))
    x[0, 0], x[0, 1], x[0, 31] = 1.0, 10.0, 4.0
    out, size = L.linear(x, w, np.array([[128]], np.uint8))
    assert out[0, 0] == 2 * (1.5 - 60.0 + 2.0) and size[0, 0] == 2 * (1.5 + 60.0 + 2.0)


def unsigned(t):
    return [int(v) % (1 << 64) for v in t.tolist()]


def test_rope_freqs():
    f = unsigned(rope_freqs(8, base=16.0, device="cpu"))
    want = [16.0 ** (-i / 4) / (2 * math.pi) * 2.0 ** 64 for i in range(4)]
    assert all(abs(a - b) <= 2.0 ** -52 * b for a, b in zip(f, want))
    slow = unsigned(rope_freqs(8, base=16.0, factor=4.0, device="cpu"))  # (whole numbers again)
    assert all(abs(a - b / 4) <= 1 for a, b in zip(slow, f))
    # radians beyond half a turn wrap; the given ones are taken as they are
    assert unsigned(rope_freqs(4, inv_freq=[math.pi, 1.5 * math.pi], device="cpu")) == [1 << 63, 3 << 62]


def test_rope_freqs_by_parts():
    """Fast pairs keep their frequency, slow ones are divided, between them a line."""
    plain = unsigned(rope_freqs(64, base=10000.0, device="cpu"))
    got = unsigned(rope_freqs(64, base=10000.0, factor=8.0, trained=4096, device="cpu"))

    def pair(turns):
        return 32 * math.log(4096 / (turns * 2 * math.pi)) / math.log(10000.0)

    low, high = math.floor(pair(32.0)), math.ceil(pair(1.0))
    assert 0 < low < high < 32
    for i in range(32):
        mix = min(max((i - low) / (high - low), 0.0), 1.0)
        want = plain[i] * (1 - mix + mix / 8.0)
        # (both are rounded to whole numbers: half of one each)
        assert abs(got[i] - want) <= 2.0 ** -50 * want + 1


@pytest.mark.parametrize("kw", [dict(rot=0), dict(rot=7), dict(rot=8, factor=0.0), dict(rot=8, factor=float("nan")),
                                dict(rot=8, inv_freq=[1.0]), dict(rot=4, inv_freq=[1.0, float("inf")])])
def test_rope_freqs_refusals(kw):
    with pytest.raises(ValueError):
        rope_freqs(device="cpu", **kw)


def test_quant_x4_rounds_to_the_nearest():
    """Every E2M1 border from both sides and on it, under scales far apart, and groups of zeros."""
    values = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    tie = {0.25: 0.0, 0.75: 1.0, 1.25: 1.0, 1.75: 2.0, 2.5: 2.0, 3.5: 4.0, 5.0: 4.0}
    row, want = [], []
    for b, t in tie.items():
        lo, hi = max(v for v in values if v < b), min(v for v in values if v > b)
        for x, y in ((b - 1e-6, lo), (b, t), (b + 1e-6, hi)):
            row += [x, -x]
            want += [y, -y]
    row, want = row[:31] + [6.0], want[:31] + [6.0]
    rows = torch.tensor([row, row, [0.0] * 32], dtype=torch.float64) * torch.tensor([[1.0], [2.0 ** -60], [1.0]], dtype=torch.float64)
    w, c = quant_x4(rows)
    assert c.tolist() == [[127], [67], [0]]
    got = dequant_x4(w, c).double()
    assert got[0].tolist() == want and (got[1] * 2.0 ** 60).tolist() == want and not got[2].any()
    assert np.array_equal(dequant_fp4_rows(w.numpy(), c.numpy()), got.numpy())


def test_quant_x4_takes_the_smallest_scale():
    w = torch.zeros(3, 64, dtype=torch.bfloat16)
    w[0, 3], w[0, 40], w[1, 0], w[2, 63] = 6.0, -6.03125, 3.0, 1e-30
    packed, c = quant_x4(w)
    assert c.tolist()[0] == [127, 128] and c.tolist()[1] == [126, 0]
    d = dequant_x4(packed, c)
    assert d[0, 3] == 6.0 and d[0, 40] == -6.0 and d[1, 0] == 3.0 and abs(d[2, 63].item() / 1e-30 - 1) < 0.25
    assert packed.shape == (3, 32)
    with pytest.raises(ValueError):
        quant_x4(w[:, :40])


def test_quant_x4_in_parts():
    """Rows that are taken a few at a time come out as each by itself, strided ones and none at all too."""
    k = 1 << 23
    w = torch.randn(5, 64).repeat(1, k // 64)
    packed, c = quant_x4(w)
    one, one_c = quant_x4(w[:, :64].t().contiguous().t())
    assert torch.equal(packed.view(5, -1, 32)[:, 7], one) and torch.equal(c.view(5, -1, 2)[:, -1], one_c)
    assert quant_x4(w[:0, :64])[0].shape == (0, 32)


@pytest.mark.parametrize("code", [0, 1, 127, 254, 255])
def test_dequant_x4_takes_every_code(code):
    """The code 255 makes every value of its group NaN, zeros among them; all others are powers of two."""
    w = torch.arange(16, dtype=torch.uint8)[None]  # (low nibbles 0 .. 15, high nibbles 0)
    w = torch.cat((w, w), 1)
    got = dequant_x4(w, torch.tensor([[code, 127]], dtype=torch.uint8))
    values = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0])
    plain = torch.stack((values, torch.zeros(16)), -1).view(1, 32)
    assert torch.equal(got[:, 32:], plain)
    if code == 255:
        assert torch.isnan(got[:, :32]).all()
    else:  # (2^127 times 4 and 6 lie beyond fp32)
        assert torch.equal(got[:, :32], (plain.double() * 2.0 ** (code - 127)).float())


def test_dequant_x4_of_no_rows():
    """What quant_x4 makes of no rows goes back as it came."""
    assert dequant_x4(*quant_x4(torch.zeros(0, 64))).shape == (0, 64)
    assert dequant_x4(*quant_x4(torch.ones(2, 64))).equal(torch.ones(2, 64))


@pytest.mark.parametrize("base", [100.0, 10000.0, 500000.0, 1e7])
@pytest.mark.parametrize("rot,trained", [(16, 500), (128, 8192), (128, 40), (256, 1000000)])
def test_rope_freqs_by_parts_of_given_frequencies(rot, trained, base):
    """Frequencies that are given are kept, mixed and divided by what they turn themselves: a base's own series gives
    that base's numbers (the borders of fast and slow pairs also beyond the first and the last pair)."""
    kw = dict(rot=rot, factor=8.0, trained=trained, device="cpu")
    want = unsigned(rope_freqs(base=base, **kw))
    got = unsigned(rope_freqs(inv_freq=[base ** (-2.0 * i / rot) for i in range(rot // 2)], **kw))
    # (the line between two borders that lie at least a pair apart moves with their last bits only)
    assert all(abs(a - b) <= 2.0 ** -40 * b + 1 for a, b in zip(got, want))


def test_rope_freqs_by_parts_of_an_uneven_series():
    """By hand: turns within the trained length 64, 32, 8, 4, 1, 1/4."""
    trained, turns = 1000, [64.0, 32.0, 8.0, 4.0, 1.0, 0.25]
    f = [t * 2 * math.pi / trained for t in turns]
    got = unsigned(rope_freqs(12, inv_freq=f, factor=4.0, trained=trained, fast=30.0, slow=1.5, device="cpu"))
    # 30 turns lie behind pair 1, 1.5 turns before pair 4: a line from pair 1 to pair 4
    for g, t, mix in zip(got, turns, [0.0, 0.0, 1 / 3, 2 / 3, 1.0, 1.0]):
        want = t / trained * (1 - mix + mix / 4.0) * 2.0 ** 64
        assert abs(g - want) <= 2.0 ** -45 * want + 1


@pytest.mark.parametrize("f", [[1.0, 1.0, 0.5, 0.1], [0.1, 0.5, 1.0, 2.0], [1.0, 0.5, 0.0, -1.0], [1.0, 0.1, 0.2, 0.01]])
def test_rope_freqs_by_parts_refuses_frequencies_that_do_not_fall(f):
    with pytest.raises(ValueError):
        rope_freqs(8, inv_freq=f, factor=2.0, trained=1000, device="cpu")
    assert rope_freqs(8, inv_freq=f, factor=2.0, device="cpu").shape == (4,)
    with pytest.raises(ValueError):  # (one pair has no neighbour)
        rope_freqs(2, inv_freq=[1.0], factor=2.0, trained=1000, device="cpu")


@pytest.mark.parametrize("kw", [dict(base=-2.0), dict(base=0.0), dict(base=float("nan")), dict(base=float("inf")),
                                dict(base=1.0, trained=100), dict(base=0.5, trained=100), dict(trained=0), dict(trained=-5),
                                dict(trained=float("nan")), dict(trained=100, slow=0.0), dict(trained=100, slow=-1.0),
                                dict(trained=100, fast=1.0, slow=32.0), dict(trained=100, fast=float("nan")),
                                dict(trained=100, fast=float("inf")), dict(inv_freq=[1e300] * 4, factor=1e-300)])
def test_rope_freqs_refuses_what_no_formula_covers(kw):
    with pytest.raises(ValueError):
        rope_freqs(8, device="cpu", **{"factor": 2.0, **kw})
