"""linear_x4 on every way through its kernels: which kernel runs, whether bf16 rows are
taken apart in it or in front of it, whether a cluster shares K and where its exchange
buffer lies, how many issuers, slots and warps. A case says which way it is for, and
linear_x4_shape is asked whether it takes it: where a rule is changed the cases move.
(They take their ways also on GPUs that hold fewer or more clusters of a size.)

Bounds as tests/test_gpu_layer_limits.py.
"""

import random

import pytest
import torch

import mxfp8_moe_decode_gb300 as M
from mxfp8_moe_decode_gb300.linear import linear_x4_shape
from test_gpu_layer_limits import _case, _check

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
FIELDS = ("products", "images", "stacked", "inside", "over", "shared", "issuers", "slots", "weight_warps", "row_warps")

# rows, out, K, MXFP8 or bf16, the way (FIELDS)
WAYS = [
    (246, 14085, 1152, 0, (1, 1, 1, 0, 0, 0, 1, 6, 1, 4)),
    (247, 12972, 1280, 0, (1, 1, 1, 0, 0, 0, 1, 6, 2, 4)),
    (396, 300, 2688, 0, (1, 1, 1, 0, 0, 0, 2, 10, 2, 4)),
    (973, 525, 1152, 0, (1, 1, 1, 0, 0, 0, 2, 6, 1, 4)),
    (689, 798, 1280, 0, (1, 1, 1, 0, 0, 0, 2, 6, 2, 4)),
    (642, 385, 1664, 0, (1, 1, 1, 0, 0, 0, 2, 8, 1, 4)),
    (620, 391, 1408, 0, (1, 1, 1, 0, 0, 0, 2, 8, 2, 4)),
    (63, 19933, 3712, 0, (1, 1, 1, 0, 0, 1, 1, 4, 1, 2)),
    (1, 65, 41472, 0, (1, 1, 1, 0, 0, 1, 2, 10, 2, 2)),
    (486, 395, 4096, 0, (1, 1, 1, 0, 0, 1, 2, 4, 1, 2)),
    (390, 429, 3712, 0, (1, 1, 1, 0, 0, 1, 2, 6, 1, 2)),
    (331, 396, 3968, 0, (1, 1, 1, 0, 0, 1, 2, 6, 2, 2)),
    (13, 64, 20608, 0, (1, 1, 1, 0, 0, 1, 2, 8, 1, 2)),
    (9, 65, 21504, 0, (1, 1, 1, 0, 0, 1, 2, 8, 2, 2)),
    (184, 9808, 128, 0, (1, 1, 1, 1, 0, 0, 1, 6, 1, 4)),
    (171, 9750, 256, 0, (1, 1, 1, 1, 0, 0, 1, 6, 2, 4)),
    (1, 64, 1152, 0, (1, 1, 1, 1, 0, 0, 2, 10, 2, 4)),
    (1013, 513, 640, 0, (1, 1, 1, 1, 0, 0, 2, 6, 1, 4)),
    (828, 643, 256, 0, (1, 1, 1, 1, 0, 0, 2, 6, 2, 4)),
    (609, 386, 1152, 0, (1, 1, 1, 1, 0, 0, 2, 8, 1, 4)),
    (402, 646, 1280, 0, (1, 1, 1, 1, 0, 0, 2, 8, 2, 4)),
    (1, 64, 1664, 0, (1, 1, 1, 1, 0, 1, 2, 10, 2, 4)),
    (198, 348, 3200, 0, (1, 1, 1, 1, 0, 1, 2, 6, 1, 4)),
    (198, 261, 3456, 0, (1, 1, 1, 1, 0, 1, 2, 6, 2, 4)),
    (9, 64, 3712, 0, (1, 1, 1, 1, 0, 1, 2, 8, 1, 4)),
    (9, 64, 1920, 0, (1, 1, 1, 1, 0, 1, 2, 8, 2, 4)),
    (1605, 2699, 1152, 0, (2, 1, 0, 0, 0, 0, 1, 4, 1, 1)),
    (1308, 1058, 1152, 0, (2, 1, 0, 0, 0, 0, 2, 4, 1, 1)),
    (1245, 900, 1152, 0, (2, 1, 0, 0, 0, 0, 2, 6, 1, 1)),
    (1066, 1057, 1280, 0, (2, 1, 0, 0, 0, 0, 2, 6, 2, 1)),
    (447, 898, 3968, 0, (2, 1, 0, 0, 1, 1, 2, 4, 1, 1)),
    (386, 955, 3712, 0, (2, 1, 0, 0, 1, 1, 2, 6, 1, 1)),
    (633, 446, 2944, 0, (2, 1, 0, 0, 1, 1, 2, 6, 2, 1)),
    (1469, 1699, 1152, 0, (2, 2, 0, 0, 0, 0, 1, 3, 1, 1)),
    (2105, 2202, 1152, 0, (2, 2, 0, 0, 0, 0, 1, 4, 1, 1)),
    (1282, 1704, 1152, 0, (2, 2, 0, 0, 0, 0, 2, 4, 1, 1)),
    (1343, 1136, 5632, 0, (2, 2, 0, 0, 1, 1, 1, 3, 1, 1)),
    (1084, 1069, 4992, 0, (2, 2, 0, 0, 1, 1, 2, 4, 1, 1)),
    (1773, 2468, 1152, 1, (1, 1, 0, 0, 0, 0, 1, 6, 1, 4)),
    (2115, 2078, 1280, 1, (1, 1, 0, 0, 0, 0, 1, 6, 2, 4)),
    (1, 64, 1152, 1, (1, 1, 0, 0, 0, 0, 2, 10, 2, 4)),
    (1295, 1100, 1152, 1, (1, 1, 0, 0, 0, 0, 2, 6, 1, 4)),
    (1053, 1299, 1280, 1, (1, 1, 0, 0, 0, 0, 2, 6, 2, 4)),
    (835, 650, 1152, 1, (1, 1, 0, 0, 0, 0, 2, 8, 1, 4)),
    (694, 778, 1280, 1, (1, 1, 0, 0, 0, 0, 2, 8, 2, 4)),
    (1, 64, 1920, 1, (1, 1, 0, 0, 0, 1, 2, 10, 2, 2)),
    (481, 486, 4736, 1, (1, 1, 0, 0, 0, 1, 2, 6, 1, 2)),
    (492, 398, 3968, 1, (1, 1, 0, 0, 0, 1, 2, 6, 2, 2)),
    (197, 261, 3200, 1, (1, 1, 0, 0, 0, 1, 2, 8, 1, 2)),
    (311, 142, 2432, 1, (1, 1, 0, 0, 0, 1, 2, 8, 2, 2)),
    (671, 686, 5248, 1, (1, 1, 0, 0, 1, 1, 2, 6, 1, 2)),
    (651, 734, 4608, 1, (1, 1, 0, 0, 1, 1, 2, 6, 2, 2)),
    (473, 802, 4224, 1, (1, 1, 0, 0, 1, 1, 2, 8, 1, 2)),
    (639, 399, 4096, 1, (1, 1, 0, 0, 1, 1, 2, 8, 2, 2)),
    (1958, 3070, 1152, 1, (1, 2, 0, 0, 0, 0, 1, 4, 1, 2)),
    (2227, 2063, 1152, 1, (1, 2, 0, 0, 0, 0, 1, 6, 1, 4)),
    (2698, 1740, 1280, 1, (1, 2, 0, 0, 0, 0, 1, 6, 2, 4)),
    (1336, 2099, 1152, 1, (1, 2, 0, 0, 0, 0, 2, 4, 1, 2)),
    (1301, 1708, 1152, 1, (1, 2, 0, 0, 0, 0, 2, 6, 1, 4)),
    (1295, 1732, 1280, 1, (1, 2, 0, 0, 0, 0, 2, 6, 2, 4)),
    (503, 1687, 6784, 1, (1, 2, 0, 0, 1, 1, 2, 4, 1, 2)),
    (424, 1691, 5760, 1, (1, 2, 0, 0, 1, 1, 2, 6, 1, 2)),
    (1032, 1071, 5632, 1, (1, 2, 0, 0, 1, 1, 2, 6, 2, 2)),
]


def _way(m, n, k, mx):
    s = linear_x4_shape(m, k, n, bool(mx), DEV)
    s["shared"] = int(s["split"] > 1)
    return tuple(s[f] for f in FIELDS)


def _wide_rows(m, k, seed):
    """bf16 rows of values over 2^-30 .. 2^30 with groups of zeros, K + 64 columns apart with NaN between them."""
    g = torch.Generator(device=DEV).manual_seed(seed)
    x = torch.randn(m, k, generator=g, device=DEV)
    x *= torch.exp2(torch.randint(-30, 31, (m, k), generator=g, device=DEV).float())
    x[:, 32:64] = 0.0
    room = torch.full((m, k + 64), float("nan"), dtype=torch.bfloat16, device=DEV)
    room[:, :k] = x
    return room[:, :k]


class Guarded:
    """A workspace of exactly the bytes that a call needs, filled with a pattern, between guards."""

    def __init__(self, m, k, mx, fill):
        self.need, self.fill = M.linear_x4_workspace_bytes(m, k, bool(mx)), fill
        self.room = torch.full((self.need + 512,), 0x33, dtype=torch.uint8, device=DEV)
        self.ws = self.room[256:256 + self.need]
        self.ws.fill_(fill)

    def arg(self):
        return self.ws if self.need else None

    def whole(self):
        return (self.room[:256] == 0x33).all().item() and (self.room[256 + self.need:] == 0x33).all().item()

    def untouched(self):
        return (self.ws == self.fill).all().item()


@pytest.mark.parametrize("m,n,k,mx,way", WAYS)
def test_linear_ways(m, n, k, mx, way):
    """Strided rows in and out, a workspace of exactly its size, rows that are not finite, the same bits every time."""
    assert dict(zip(FIELDS, _way(m, n, k, mx))) == dict(zip(FIELDS, way))
    x, w, wc, xc = _case(m, n, k, bool(mx), seed=9)
    if not mx:
        x = _wide_rows(m, k, m + n)
    status = torch.zeros(1, dtype=torch.int32, device=DEV)
    room = torch.full((m + 2, n + 3), 7.0, dtype=torch.bfloat16, device=DEV)
    out = room[1:m + 1, 2:n + 2]
    spaces = [Guarded(m, k, mx, fill) for fill in (0x55, 0xAA)]
    want = M.linear_x4(x, w, wc, x_codes=xc, out=out, workspace=spaces[0].arg(), status=status).clone()
    _check(want, x, w, wc, xc, sorted({0, n // 2, max(n - 130, 0), n - 1}))
    wrong = torch.zeros((), dtype=torch.int64, device=DEV)
    for _ in range(20):
        out.fill_(float("nan"))
        M.linear_x4(x, w, wc, x_codes=xc, out=out, workspace=spaces[1].arg(), status=status)
        wrong += (out != want).sum()
    assert wrong.item() == 0 and status.item() == 0
    assert (room[0] == 7).all() and (room[m + 1] == 7).all() and (room[:, :2] == 7).all() and (room[:, n + 2:] == 7).all()
    assert all(s.whole() for s in spaces)
    if spaces[0].need:
        inside = way[FIELDS.index("inside")]
        assert all(s.untouched() == inside for s in spaces)
        assert inside or m * k // 32 % 16 or torch.equal(spaces[0].ws, spaces[1].ws)  # (every byte of it is written)
    bad = sorted({0, m // 2, m - 1})
    x2 = x.clone()
    if mx:
        x2[0, k - 1], x2[m // 2, 5], x2[m - 1, 40] = 0x7F, 0xFF, 0x7F
    else:
        x2[0, k - 1], x2[m // 2, 5], x2[m - 1, 40] = float("inf"), float("nan"), -float("inf")
    out2 = M.linear_x4(x2, w, wc, x_codes=xc)
    assert torch.isnan(out2[bad]).all()
    rows = [i for i in range(m) if i not in bad]
    assert torch.equal(out2[rows], want[rows])


# bf16 rows that a kernel in front takes apart into the workspace
FRONT = [(13, 40000, 1024), (60, 20000, 1024), (48, 5120, 5120), (400, 3000, 1024), (72, 4096, 4096), (170, 38913, 640)]


def _front(m, n, k):
    assert not linear_x4_shape(m, k, n, False, DEV)["inside"]


def test_the_ways_of_rows_in_a_workspace():
    for m, n, k in FRONT:
        _front(m, n, k)
    ways = [dict(zip(FIELDS, _way(m, n, k, 0))) for m, n, k in FRONT]
    assert {w["products"] for w in ways} == {1, 2} and {w["over"] for w in ways} == {0, 1}


@pytest.mark.parametrize("m,n,k", FRONT)
def test_linear_workspace_is_used_again(m, n, k):
    """One workspace for calls right behind one another on other rows: the rows of a call are not taken apart over
    those that the call before still reads, nor read before they are there."""
    _front(m, n, k)
    x0, w, wc, _ = _case(m, n, k, False)
    xs = [x0] + [_case(m, 1, k, False, seed=s)[0] for s in (1, 2)]
    want = [M.linear_x4(x, w, wc).clone() for x in xs]
    torch.cuda.synchronize()
    space = Guarded(m, k, False, 0x55)
    outs = [torch.empty_like(want[0]) for _ in range(3)]
    wrong = torch.zeros((), dtype=torch.int64, device=DEV)
    for i in range(20):
        for x, out in zip(xs, outs):
            M.linear_x4(x, w, wc, out=out, workspace=space.ws)
        for out, v in zip(outs, want):
            wrong += (out != v).sum()
    assert wrong.item() == 0 and space.whole() and not space.untouched()


@pytest.mark.parametrize("m,n,k", FRONT)
def test_linear_right_behind_a_norm_and_in_front_of_one(m, n, k):
    """Rows that a framework kernel writes just before, and out that another reads just behind: no wait on the host."""
    _front(m, n, k)
    x, w, wc, _ = _case(m, n, k, False)
    one = torch.ones(k, dtype=torch.bfloat16, device=DEV)
    wide = n // 64 * 32 if n < 16384 else 8192
    ones = torch.ones(wide, dtype=torch.bfloat16, device=DEV)
    room = torch.zeros(m, (n + 7) // 8 * 8, dtype=torch.bfloat16, device=DEV)
    space = Guarded(m, k, False, 0x55)

    def chain(x, sync):
        r, *_ = M.add_norm_x8(x, x, one)
        if sync:
            torch.cuda.synchronize()
        y = M.linear_x4(r, w, wc, out=room[:, :n], workspace=space.ws)
        if sync:
            torch.cuda.synchronize()
        return M.add_norm_x8(y[:, :wide], y[:, :wide], ones)[0]

    xs = [(x.float() * f).bfloat16() for f in (1.0, 0.75, -2.0)]
    want = [chain(x, True) for x in xs]
    got = [chain(x, False) for _ in range(10) for x in xs]
    torch.cuda.synchronize()
    assert all(torch.equal(g, want[i % 3]) for i, g in enumerate(got)) and space.whole()


def test_linear_workspaces_side_by_side():
    """Every call has its own workspace: eager ones on streams of their own, and captured ones, at once."""
    sides = []
    for i, (m, n, k) in enumerate(FRONT):
        _front(m, n, k)
        x, w, wc, _ = _case(m, n, k, False, seed=i)
        want, space = M.linear_x4(x, w, wc).clone(), Guarded(m, k, False, 0x55)
        out = torch.empty_like(want)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = M.linear_x4(x, w, wc)  # (a workspace of the graph's own)
        sides.append((graph, got, want, out, space, torch.cuda.Stream(), torch.cuda.Stream(), (x, w, wc)))
    torch.cuda.synchronize()
    for _ in range(15):
        for graph, _, _, out, space, s, t, (x, w, wc) in sides:
            with torch.cuda.stream(s):
                graph.replay()
            with torch.cuda.stream(t):
                M.linear_x4(x, w, wc, out=out, workspace=space.ws)
    torch.cuda.synchronize()
    for graph, got, want, out, space, s, t, args in sides:
        assert torch.equal(got, want) and torch.equal(out, want) and space.whole() and not space.untouched()
    graph, got, *_, (x, w, wc) = sides[0]
    for seed in (1, 2):  # a replay takes the rows that are there then
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got, M.linear_x4(x, w, wc))


@pytest.mark.parametrize("seed", range(4))
def test_linear_random_shapes(seed):
    """Shapes over the whole range, three calls at once on three streams, three times each: the same bits, within the
    bounds, no status."""
    rng = random.Random(seed)
    streams = [torch.cuda.Stream() for _ in range(3)]
    for i in range(60):
        jobs = []
        for s in streams:
            k, n, m = 128 * int(2 ** rng.uniform(0, 7.5)), int(2 ** rng.uniform(0, 15)), int(2 ** rng.uniform(0, 10.5))
            mx = rng.random() < 0.5
            k, n = min(k, 8192) if mx else k, max(1, min(n, int(3e8) // k))
            m = max(1, min(m, int(1e11) // (n * k)))
            x, w, wc, xc = _case(m, n, k, mx, seed=i)
            jobs.append((s, (x, w, wc, xc), torch.zeros(1, dtype=torch.int32, device=DEV), [],
                         sorted({0, n // 2, rng.randrange(n), n - 1})))
        torch.cuda.synchronize()
        for _ in range(3):
            for s, (x, w, wc, xc), status, outs, _ in jobs:
                with torch.cuda.stream(s):
                    outs.append(M.linear_x4(x, w, wc, x_codes=xc, status=status))
        torch.cuda.synchronize()
        for _, (x, w, wc, xc), status, outs, columns in jobs:
            assert status.item() == 0 and torch.equal(outs[0], outs[1]) and torch.equal(outs[0], outs[2]), (x.shape, w.shape)
            _check(outs[0], x, w, wc, xc, columns)


@pytest.mark.parametrize("m,n,k", [(6, 150, 384), (64, 20000, 1280), (170, 400, 4096), (1295, 1732, 1280)])
def test_linear_rows_under_a_nan_code(m, n, k):
    """The code 255 of a row's group makes that row NaN, also where the group's bytes are zeros, and no other row."""
    x, w, wc, xc = _case(m, n, k, True)
    want = M.linear_x4(x, w, wc, x_codes=xc)
    x2, xc2 = x.clone(), xc.clone()
    xc2[0, 0], xc2[m // 2, k // 32 - 1], xc2[m - 1, 3] = 255, 255, 255
    x2[m // 2, k - 32:] = 0
    out = M.linear_x4(x2, w, wc, x_codes=xc2)
    bad = [0, m // 2, m - 1]
    rows = [i for i in range(m) if i not in bad]
    assert torch.isnan(out[bad]).all() and torch.equal(out[rows], want[rows])


# ---------------------------------------------------------------- what two parts hold of a bf16 value
PARTS = [(3, 1100, 1024), (16, 1100, 4096), (13, 40000, 1024), (48, 5120, 5120), (400, 3000, 1024), (72, 4096, 4096),
         (170, 38913, 640)]


@pytest.mark.parametrize("m,n,k", PARTS)
def test_linear_bf16_values_beside_a_large_one(m, n, k):
    """Every weight row has a single 1, so a column of out is a column of x as hi and lo hold it: itself from 2^-13 of
    its group's largest value on, below within 2^-21 of that largest. (Down to 2^-14 is not exact: beside 225, which
    leaves no scale unused, 225 * 2^-14 lies at 7.03 of hi's steps and its rest at half of lo's last one.)"""
    g = torch.Generator(device=DEV).manual_seed(m + n + k)
    top = torch.exp2(torch.randint(-90, 90, (m, k // 32, 1), generator=g, device=DEV).float())
    top *= 1 + torch.randint(0, 128, top.shape, generator=g, device=DEV) / 128.0
    top[0] = 225.0
    x = torch.randn(m, k // 32, 32, generator=g, device=DEV).sign()
    x *= top * torch.exp2(-18.0 * torch.rand(x.shape, generator=g, device=DEV))
    x[:, :, 1] = top[:, :, 0] * 2.0 ** -13
    x[:, :, 2] = top[:, :, 0] * 2.0 ** -14
    x[:, :, 3] = -top[:, :, 0] * (2.0 ** -13 * 1.5)
    x[:, :, 17] = top[:, :, 0]
    x = x.bfloat16()
    x = torch.where(x.float().abs() > top, top.bfloat16(), x)  # (rounded past the largest)
    w = torch.zeros(n, k // 2, dtype=torch.uint8, device=DEV)
    column = (torch.arange(n, device=DEV) * 7 + 1) % k
    w[torch.arange(n, device=DEV), column // 2] = torch.where(column % 2 == 0, 0x02, 0x20).to(torch.uint8)  # 1.0
    wc = torch.full((n, k // 32), 127, dtype=torch.uint8, device=DEV)
    out = M.linear_x4(x.view(m, k), w, wc).double()
    want, largest = x.view(m, k).double()[:, column], top.expand(-1, -1, 32).reshape(m, k).double()[:, column]
    exact = want.abs() >= 2.0 ** -13 * largest
    assert exact.any() and (~exact).any() and torch.equal(out[exact], want[exact])
    # (below it lo's step is 2^-13 where the largest is above 224: hi + lo has 7 bits at most, out's rounding changes
    # nothing, and half of that step is below 2^-21 * 224)
    assert ((out - want).abs() <= 2.0 ** -21 * largest).all()


def test_ways_of_the_two_parts():
    ways = [dict(zip(FIELDS, _way(m, n, k, 0))) for m, n, k in PARTS]
    assert {(w["products"], w["images"], w["inside"]) for w in ways} >= {(1, 1, 1), (1, 1, 0), (2, 1, 0), (2, 2, 0)}
