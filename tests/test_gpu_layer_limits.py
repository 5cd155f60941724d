"""The layer's operators where calls meet: first calls inside a capture, graphs
replayed side by side, a call right behind another that writes its operands,
offsets past 32 bits, and every depth of the product's ring run often."""

import os
import subprocess
import sys

import pytest
import torch

import mxfp8_moe_decode_gb300 as M

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

FIRST = """
import torch
import mxfp8_moe_decode_gb300 as M
from mxfp8_moe_decode_gb300 import _lib
dev = torch.device("cuda:0")
g = torch.Generator().manual_seed(1)
x = torch.randn(5, 1024, generator=g).bfloat16().to(dev)
w, wc = M.quant_x4(torch.randn(700, 1024, generator=g).to(dev))
nw = torch.ones(1024, dtype=torch.bfloat16, device=dev)
pos = torch.arange(5, dtype=torch.int32, device=dev)
f = M.rope_freqs(128, device=dev)
blocks, codes = M.kv_cache_x8(5, 2, 128, dev)
table, had = torch.arange(5, dtype=torch.int32, device=dev).view(5, 1), torch.zeros(5, dtype=torch.int32, device=dev)
torch.cuda.synchronize()

def step():
    res, x8, c, _ = M.norm_add_norm_x8(x, x, nw, nw)
    a, b = M.linear_x4(x8, w, wc, x_codes=c), M.linear_x4(res, w, wc)
    q = M.rope(x.view(5, 8, 128), pos, f)
    return res, x8, a, b, q, *M.rope_kv_append_x8(blocks, codes, q, q[:, :2], q[:, 2:4], table, had, f)

graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    got = step()
graph.replay()
torch.cuda.synchronize()
kept = [t.clone() for t in got]
want = step()
torch.cuda.synchronize()
assert all(torch.equal(p, q) for p, q in zip(kept, want)), [torch.equal(p, q) for p, q in zip(kept, want)]
print("same")
"""


def test_first_calls_inside_a_capture():
    r = subprocess.run([sys.executable, "-c", FIRST], cwd=ROOT, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "same" in r.stdout, r.stderr[-2000:]


def _case(m, n, k, mx, seed=0):
    g = torch.Generator(device=DEV).manual_seed(seed + m + n + k)
    w = torch.randint(0, 256, (n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
    wc = torch.randint(110, 130, (n, k // 32), generator=g, device=DEV, dtype=torch.uint8)
    x = torch.randn(m, k, generator=g, device=DEV).bfloat16()
    if not mx:
        return x, w, wc, None
    one = torch.ones(k, dtype=torch.bfloat16, device=DEV)
    _, x8, c, _ = M.norm_add_norm_x8(x, x, None, one) if k <= 8192 else (None, x.view(torch.uint8)[:, :k] & 0x77, wc[:1].expand(m, -1).contiguous(), None)
    return x8, w, wc, c


def _check(out, x, w, wc, xc, columns):
    """Some columns of out against fp64 (bounds as tests/test_gpu_layer.py: the sums, and bf16 rows off by 2^-21 of
    their group's largest at most). At the smallest numbers the formats' steps end: half of bf16's last step, 2^-133,
    and of lo's, E4M3's 2^-9 under the code 0 (2^-127), for every value of x."""
    m, k = x.shape
    pick = torch.tensor(columns, device=DEV)
    rows = M.dequant_x4(w[pick], wc[pick]).double()
    v = x.double() if xc is None else (x.view(torch.float8_e4m3fn).double().view(m, -1, 32) *
                                       torch.exp2(xc.double() - 127)[..., None]).view(m, -1)
    slack = (k / 32 * 2.0 ** -23 + 2.0 ** -19) * v.abs() @ rows.abs().t()
    slack += 2.0 ** -134
    if xc is None:
        slack += 2.0 ** -21 * v.abs().view(m, -1, 32).amax(-1).repeat_interleave(32, 1) @ rows.abs().t()
        slack += 2.0 ** -137 * rows.abs().sum(1)
    exact = v @ rows.t()
    assert ((out[:, pick].double() - exact).abs() <= 2.0 ** -8 * exact.abs() + slack).all()


@pytest.mark.parametrize("mx", [True, False])
@pytest.mark.parametrize("m", [1, 24, 40, 56, 72, 90, 110, 130, 150, 170, 192])
@pytest.mark.parametrize("n,k", [(152 * 128 + 5, 640), (300, 128 * 21), (2000, 128 * 33), (152 * 128 * 2 + 1, 128 * 5)])
def test_linear_is_the_same_every_time(m, n, k, mx):
    """Every number of slots, warps and shares of K, tiles with a group of a single K block too: 60 runs back to
    back, bit for bit, and equal to a row-by-row product in fp64 at some rows."""
    x, w, wc, xc = _case(m, n, k, mx)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    want = M.linear_x4(x, w, wc, x_codes=xc, status=status).clone()
    out = torch.empty_like(want)
    wrong = torch.zeros((), dtype=torch.int64, device=DEV)
    for _ in range(60):
        out.fill_(float("nan"))
        M.linear_x4(x, w, wc, x_codes=xc, out=out, status=status)
        wrong += (out.view(torch.int16) != want.view(torch.int16)).sum()
    assert wrong.item() == 0 and status.item() == 0
    _check(want, x, w, wc, xc, sorted({0, n // 2, n - 130, n - 1}))


@pytest.mark.parametrize("m,n,k", [(3, 150, 1024), (16, 600, 4096), (60, 300, 256),        # taken apart in the kernel
                                   (24, 150, 65536), (60, 20000, 1024), (13, 40000, 1024),  # in front of it
                                   (400, 3000, 1024), (150, 5000, 2048)])                   # as two products
def test_linear_rows_taken_apart(m, n, k):
    """bf16 rows on every way to the tensor cores: values over 2^-30 .. 2^30, groups of zeros, of the smallest and of
    the largest numbers, and rows that are not finite, which touch no other."""
    g = torch.Generator(device=DEV).manual_seed(m + n + k)
    w = torch.randint(0, 256, (n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
    wc = torch.randint(115, 122, (n, k // 32), generator=g, device=DEV, dtype=torch.uint8)
    x = torch.randn(m, k, generator=g, device=DEV) * torch.exp2(torch.randint(-30, 31, (m, k), generator=g, device=DEV).float())
    x[:, 32:64] = 0.0
    x[1] = 1e-39 * torch.randn(k, generator=g, device=DEV)                 # (subnormal in fp32 too)
    x[m - 1] = x[m - 1].sign() * 1e38 * (1 + x[m - 1].abs() % 1)
    x = x.bfloat16()
    columns = sorted({0, 1, 100, 127, 128, n // 2, n - 20, n - 1})
    out = M.linear_x4(x, w, wc)
    seen = torch.isfinite(out[m - 1, columns]).all(0).item()               # (sums past fp32's range are infinite)
    last = m if seen else m - 1
    _check(out[:last], x[:last], w, wc, None, columns)
    assert out[1, columns].double().abs().max() < 2.0 ** -90
    bad = sorted({0, m // 2, m - 1})
    x2 = x.clone()
    x2[0, k - 1], x2[m // 2, 5], x2[m - 1, 40] = float("inf"), float("nan"), -float("inf")
    out2 = M.linear_x4(x2, w, wc)
    assert torch.isnan(out2[bad]).all()
    rows = [i for i in range(m) if i not in bad]
    assert torch.equal(out2[rows], out[rows])


def test_linear_graphs_side_by_side():
    """Two graphs, each with its calls' own workspaces, replayed on two streams at once."""
    sides = []
    for i, (m, n, k) in enumerate(((8, 4000, 1024), (60, 5000, 896))):
        x, w, wc, _ = _case(m, n, k, False, seed=i)
        want = M.linear_x4(x, w, wc).clone()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = M.linear_x4(x, w, wc)
        sides.append((graph, got, want, torch.cuda.Stream(), (x, w, wc)))
    torch.cuda.synchronize()
    for _ in range(50):
        for graph, _, _, stream, _ in sides:
            with torch.cuda.stream(stream):
                graph.replay()
    torch.cuda.synchronize()
    assert all(torch.equal(got, want) for _, got, want, _, _ in sides)


@pytest.mark.parametrize("mx", [True, False])
def test_linear_right_behind_what_writes_its_operands(mx):
    """Weights, rows and the rows' buffer written by the call before, on one stream, over and over."""
    m, n, k = 20, 3000, 1280
    sets = [_case(m, n, k, mx, seed=s) for s in range(3)]
    want = [M.linear_x4(x, w, wc, x_codes=xc).clone() for x, w, wc, xc in sets]
    x, w, wc, xc = (None if t is None else t.clone() for t in sets[0])
    need = M.linear_x4_workspace_bytes(m, k, mx)
    ws = torch.empty(max(need, 16), dtype=torch.uint8, device=DEV)
    out = torch.empty_like(want[0])
    got = []
    for i in range(60):
        for t, s in zip((x, w, wc, xc), sets[i % 3]):
            if t is not None:
                t.copy_(s)
        M.linear_x4(x, w, wc, x_codes=xc, out=out, workspace=ws)
        M.linear_x4(x, w, wc, x_codes=xc, out=out, workspace=ws)
        got.append(out.clone())
    torch.cuda.synchronize()
    assert all(torch.equal(t, want[i % 3]) for i, t in enumerate(got))


def test_norm_straight_into_linear():
    """A chain of framework kernels alone: each may start before the one in front has ended, and waits for it."""
    k, m = 2048, 33
    g = torch.Generator(device=DEV).manual_seed(2)
    w, wc = M.quant_x4(torch.randn(k, k, generator=g, device=DEV) * k ** -0.5)
    one = torch.ones(k, dtype=torch.bfloat16, device=DEV)
    x0 = torch.randn(m, k, generator=g, device=DEV).bfloat16()

    def chain(sync):
        x, r = x0, x0
        for _ in range(12):
            r, x8, c, _ = M.norm_add_norm_x8(x, r, one, one)
            if sync:
                torch.cuda.synchronize()
            x = M.linear_x4(x8, w, wc, x_codes=c)
            if sync:
                torch.cuda.synchronize()
            x = M.linear_x4(x, w, wc)
            if sync:
                torch.cuda.synchronize()
        return x

    want = chain(True)
    assert torch.isfinite(want).all()
    for _ in range(20):
        assert torch.equal(chain(False), want)


# ---------------------------------------------------------------- past 32 bits
def test_linear_rows_past_32_bits():
    """out of 4.4 GB, and x of rows far apart."""
    m, n, k = 17000, 130000, 128
    x, w, wc, _ = _case(m, n, k, False)
    _check(M.linear_x4(x, w, wc), x, w, wc, None, [0, 1, 127, 128, n // 2, n - 129, n - 128, n - 1])
    wide = torch.empty(9, 300_000_000, dtype=torch.bfloat16, device=DEV)
    wide[:, :k] = x[:9]
    assert torch.equal(M.linear_x4(wide[:, :k], w, wc), M.linear_x4(x[:9].contiguous(), w, wc))


@pytest.mark.parametrize("mx", [True, False])
@pytest.mark.parametrize("m,n,k", [(1 << 20, 130, 128), (3, 1 << 24, 128)])
def test_linear_at_its_limits(m, n, k, mx):
    x, w, wc, xc = _case(m, n, k, mx)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    out = M.linear_x4(x, w, wc, x_codes=xc, status=status)
    assert status.item() == 0
    _check(out, x, w, wc, xc, sorted({0, 1, 129, n // 2, n - 1}))


def test_norm_and_rope_rows_past_32_bits():
    m, h = 430000, 5120
    g = torch.Generator(device=DEV).manual_seed(3)
    x = torch.randn(m, h, generator=g, device=DEV, dtype=torch.bfloat16)
    one = torch.ones(h, dtype=torch.bfloat16, device=DEV)
    res, x8, c, _ = M.norm_add_norm_x8(x, x, one, one, gate=x)
    for lo in (0, m // 2, m - 5):
        part = x[lo:lo + 5].clone()
        for a, b in zip((res, x8, c), M.norm_add_norm_x8(part, part, one, one, gate=part)):
            assert torch.equal(a[lo:lo + 5], b)
    del res, x8, c
    pos = torch.arange(m, dtype=torch.int32, device=DEV)
    f = M.rope_freqs(128, device=DEV)
    out = M.rope(x.view(m, 40, 128), pos, f)
    for lo in (0, m // 2, m - 5):
        assert torch.equal(out[lo:lo + 5], M.rope(x[lo:lo + 5].view(5, 40, 128), pos[lo:lo + 5], f))


def test_rope_append_into_a_cache_past_32_bits():
    """Pages whose bytes begin past 2^32."""
    blocks, codes = M.kv_cache_x8(40000, 8, 128, DEV)
    small, small_codes = M.kv_cache_x8(4, 8, 128, DEV)
    g = torch.Generator(device=DEV).manual_seed(4)
    qkv = torch.randn(100, 24, 128, generator=g, device=DEV).bfloat16()
    q, k, v = qkv.split(8, dim=1)
    f = M.rope_freqs(128, device=DEV)
    cu, had = (torch.tensor(t, dtype=torch.int32, device=DEV) for t in ([0, 70, 100], [0, 0]))
    near, far = (torch.tensor(t, dtype=torch.int32, device=DEV) for t in ([[3, 0], [2, 1]], [[39999, 36000], [39998, 1]]))
    blocks[[39999, 36000, 39998, 1]] = small[[3, 0, 2, 1]]
    a, *_ = M.rope_kv_append_x8(blocks, codes, q, k, v, far, had, f, cu_q=cu)
    b, *_ = M.rope_kv_append_x8(small, small_codes, q, k, v, near, had, f, cu_q=cu)
    assert torch.equal(a, b) and torch.equal(blocks[[39999, 36000, 39998, 1]], small[[3, 0, 2, 1]])
    assert torch.equal(codes[[39999, 36000, 39998, 1]], small_codes[[3, 0, 2, 1]])
