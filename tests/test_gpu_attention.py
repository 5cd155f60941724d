"""The attention side's kernels against the float64 oracle.

Bounds (half a step of bf16, with its 8 significant bits, is 2^-8 of the value, of f16 2^-11):
* add_norm: the sum bit for bit; the norm as tests/test_gpu_attn_seam.py (1e-5
  of the row's largest value) plus bf16's rounding; bytes and codes bit for
  bit those of the attention seam's kernel on the summed rows.
* append: bytes and codes bit for bit (scales are powers of two).
* attention, per value: 2^-8 |out| (the output's rounding) + (2^-11 + 2 slack)
  * sum_j w_j |v_j| (the weights' f16 rounding, and scores off by at most
  `slack`: 2 D fp32 roundings of the product and the part of q below what the
  two E4M3 parts hold) + 2^-20 sum w |v| (fp32 sums of a page, exp2's two units
  and the joins). lse: slack + (n / 8 + 64) 2^-24 + 2^-22 (1 + |lse|).
"""

import numpy as np
import pytest
import torch

import mxfp8_moe_decode_gb300 as M
from mxfp8_moe_decode_gb300 import _lib
from oracle import attention as A
from oracle import moe as O

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
PAGE = 64


def f64(t):
    return t.detach().cpu().double().numpy()


# ---------------------------------------------------------------- add + norm
def _norm_case(m, h, seed=0, pad_x=0, pad_r=0):
    g = torch.Generator().manual_seed(seed + 7 * m + h)
    x = torch.randn(m, h + pad_x, generator=g).bfloat16().to(DEV)[:, :h]
    r = (3 * torch.randn(m, h + pad_r, generator=g)).bfloat16().to(DEV)[:, :h]
    w = (1 + 0.1 * torch.randn(h, generator=g)).bfloat16().to(DEV)
    return x, r, w


def _check_norm(x, r, w, eps=1e-6, **kw):
    normed = torch.empty(x.shape, dtype=torch.bfloat16, device=DEV)
    res, x8, codes, n = M.add_norm_x8(x, r, w, eps, normed=normed, **kw)
    torch.cuda.synchronize()
    assert n is normed
    want = A.add(f64(x), f64(r))
    assert np.array_equal(f64(res), want)
    ys = O.attn_norm(want, f64(w), eps)
    top = np.abs(ys).max(-1, keepdims=True)
    assert (np.abs(f64(normed) - ys) <= 1e-5 * top + 2.0 ** -8 * np.abs(ys)).all()
    for lo in range(0, x.shape[0], 48):
        s8, sc, _ = M.attn_seam_x8(res[lo:lo + 48].contiguous(), w, eps)
        assert torch.equal(x8[lo:lo + 48], s8) and torch.equal(codes[lo:lo + 48], sc)
    return res, x8, codes


@pytest.mark.parametrize("h", [32, 96, 1024, 1056, 5120, 8192])
@pytest.mark.parametrize("m", [1, 3, 48, 131])
def test_add_norm(m, h):
    _check_norm(*_norm_case(m, h))


def test_add_norm_strided_rows_and_in_place():
    x, r, w = _norm_case(19, 1056, pad_x=8, pad_r=64)
    a = _check_norm(x, r, w)
    r2 = r.contiguous().clone()
    res, x8, codes, normed = M.add_norm_x8(x, r2, w, res_out=r2)
    assert res is r2 and normed is None
    assert torch.equal(res, a[0]) and torch.equal(x8, a[1]) and torch.equal(codes, a[2])


def test_add_norm_rows_apart():
    """A row of NaN or infinity leaves the others alone; no rows are fine."""
    x, r, w = _norm_case(9, 512)
    a = M.add_norm_x8(x, r, w)
    x2 = x.clone()
    x2[3, 5], x2[6, 100] = float("nan"), float("inf")
    b = M.add_norm_x8(x2, r, w)
    keep = [0, 1, 2, 4, 5, 7, 8]
    for p, q in zip(a[:3], b[:3]):
        assert torch.equal(p[keep], q[keep])
    e = M.add_norm_x8(x[:0], r[:0], w)
    assert e[0].shape == (0, 512) and e[2].shape == (0, 16)


def test_add_norm_many_rows():
    x, r, w = _norm_case(70000, 32)
    res, x8, codes, _ = M.add_norm_x8(x, r, w)
    part = M.add_norm_x8(x[69000:], r[69000:], w)
    assert torch.equal(res[69000:], part[0]) and torch.equal(x8[69000:], part[1])
    assert torch.equal(codes[69000:], part[2])


# ---------------------------------------------------------------- the cache
class Cache:
    """A pool, page tables in shuffled order, and the same on the host."""

    def __init__(self, lens, kvh, d, seed=0, spare=2, extra_width=0):
        rng = np.random.default_rng(seed)
        self.rng = rng
        need = [-(-n // PAGE) for n in lens]
        self.pages = sum(need) + spare
        order = rng.permutation(self.pages)
        width = max(max(need, default=1), 1) + extra_width
        self.table = rng.integers(-3, self.pages + 3, (len(lens), width)).astype(np.int32)  # junk past the ends
        at = 0
        for b, n in enumerate(need):
            self.table[b, :n] = order[at:at + n]
            at += n
        self.blocks = np.full((self.pages, kvh, 2, PAGE * d), 0x7F, dtype=np.uint8)
        self.codes = rng.integers(0, 256, (self.pages, kvh, 2)).astype(np.uint8)
        self.lens, self.kvh, self.d = list(lens), kvh, d

    def fill(self, amp=1.0):
        """Written tokens of every sequence; the rest of the pool stays NaN."""
        k = (amp * self.rng.standard_normal((sum(self.lens), self.kvh, self.d)) *
             np.exp(self.rng.standard_normal((1, self.kvh, 1))))
        v = self.rng.standard_normal((sum(self.lens), self.kvh, self.d))
        cu = np.concatenate(([0], np.cumsum(self.lens))).tolist()
        self.blocks, self.codes = A.append(self.blocks, self.codes, A.bf16_rne(k), A.bf16_rne(v), self.table,
                                           [0] * len(self.lens), cu)
        return self

    def gpu(self):
        return (torch.from_numpy(self.blocks).to(DEV), torch.from_numpy(self.codes).to(DEV),
                torch.from_numpy(self.table).to(DEV))


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def _append_case(had, new, kvh, d, seed=0, cu=True, amp=None):
    c = Cache([a + b for a, b in zip(had, new)], kvh, d, seed)
    lens, c.lens = c.lens, list(had)
    c.fill()
    c.lens = lens
    cu_q = np.concatenate(([0], np.cumsum(new))).tolist()
    t = cu_q[-1]
    x = c.rng.standard_normal((t, 2, kvh, d))
    if amp is not None:
        x = x * amp[:t, None, None, None]
    x = torch.from_numpy(x).bfloat16().to(DEV)
    blocks, codes, table = c.gpu()
    status = i32([0])
    M.kv_append_x8(blocks, codes, x[:, 0], x[:, 1], table, i32(had), cu_q=i32(cu_q) if cu else None, status=status)
    want = A.append(c.blocks, c.codes, f64(x[:, 0]), f64(x[:, 1]), c.table, had, cu_q)
    torch.cuda.synchronize()
    assert status.item() == 0
    got = blocks.cpu().numpy()
    # bytes of later tokens of a touched page are unspecified: compare what the sequences hold
    held = np.zeros((c.pages, PAGE), dtype=bool)
    for b, n in enumerate(c.lens):
        for j in range(n):
            held[c.table[b, j // PAGE], j % PAGE] = True
    untouched = np.ones(c.pages, dtype=bool)
    for b, n in enumerate(new):
        for p in range(had[b] // PAGE, -(-(had[b] + n) // PAGE) if n else 0):
            untouched[c.table[b, p]] = False
    assert np.array_equal(got[untouched], c.blocks[untouched])
    for kind, image in enumerate(A.image_bytes(d)):
        a, w = got[:, :, kind][..., image], want[0][:, :, kind][..., image]
        h = np.broadcast_to(held[:, None, :, None], a.shape)
        nan = (a & 0x7F == 0x7F) & (w & 0x7F == 0x7F)
        assert ((a == w) | nan | ~h).all()
    assert np.array_equal(codes.cpu().numpy(), want[1])
    return blocks, codes, table, x, cu_q


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("had,new", [
    ([0], [1]), ([63], [1]), ([64], [1]), ([5], [0]), ([0, 17, 64, 100], [1, 1, 1, 1]),
    ([0, 60, 3], [64, 8, 9]), ([1, 63, 0, 30, 127], [200, 2, 130, 0, 65]), ([50], [300]),
])
def test_append(had, new, d):
    _append_case(had, new, 3, d, seed=d + len(had))
    if all(n == 1 for n in new):
        _append_case(had, new, 2, d, seed=d, cu=False)


def test_append_scales_grow_and_stay():
    """Loud new tokens move a page's earlier bytes, quiet ones do not (also by
    more than E4M3's range, where they vanish)."""
    for amp in (2.0 ** 3, 2.0 ** 8, 2.0 ** 30, 2.0 ** 90, 2.0 ** -20, 2.0 ** -110, 0.0):
        _append_case([40, 7], [9, 1], 2, 128, amp=np.full(10, amp))


def test_append_keeps_non_finite_values_apart():
    amp = np.ones(70)
    amp[3], amp[20], amp[69] = np.nan, np.inf, -np.inf
    _append_case([10], [70], 1, 64, amp=amp)


def test_append_many_sequences():
    rng = np.random.default_rng(3)
    had = rng.integers(0, 130, 300).tolist()
    _append_case(had, rng.integers(0, 3, 300).tolist(), 1, 64)


def test_append_again_changes_nothing_and_strides():
    blocks, codes, table, x, cu_q = _append_case([30], [50], 2, 128)
    b0, c0 = blocks.clone(), codes.clone()
    wide = torch.zeros(50, 3, 2, 128, dtype=torch.bfloat16, device=DEV)
    wide[:, 1], wide[:, 2] = x[:, 0], x[:, 1]
    M.kv_append_x8(blocks, codes, wide[:, 1], wide[:, 2], table, i32([30]), cu_q=i32(cu_q))
    assert torch.equal(codes, c0)
    val = M.kv_dequant_x8(blocks, codes)[table[0, :2].long()]
    was = M.kv_dequant_x8(b0, c0)[table[0, :2].long()]
    tok = torch.arange(128, device=DEV).view(2, 1, 1, 64, 1) < 80
    assert torch.equal(torch.where(tok, val, 0), torch.where(tok, was, 0))


def test_append_reports_bad_pages_and_lengths():
    """Page ids out of range, lengths below 0 or past the table: skipped and
    reported, nothing else is written."""
    c = Cache([10, 10, 10, 64], 2, 64).fill()
    k = torch.ones(4, 2, 64, dtype=torch.bfloat16, device=DEV)
    for table, start, bit in [((0, -1), 0, _lib.KV_STATUS_PAGE), ((0, c.pages), 0, _lib.KV_STATUS_PAGE),
                              (None, -5, _lib.KV_STATUS_LENGTH), (None, 64, _lib.KV_STATUS_LENGTH)]:
        t = c.table.copy()
        start0 = [10, 10, 10, 63]
        if table:
            t[0, 0] = table[1]
            t[1:3, 0] = -1
            t[3, 0] = c.pages + 100
        else:
            start0 = [start] * 4
        blocks, codes, _ = c.gpu()
        status = i32([0])
        M.kv_append_x8(blocks, codes, k, k, torch.from_numpy(t).to(DEV), i32(start0), status=status)
        torch.cuda.synchronize()
        assert status.item() == bit
        assert np.array_equal(blocks.cpu().numpy(), c.blocks) and np.array_equal(codes.cpu().numpy(), c.codes)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("cu_q", [[0, 6, 2, 8], [0, 3, 1, 2], [0, 8, 0, 8], [5, 0, 8, 8]])
def test_append_refuses_row_starts_that_do_not_ascend(cu_q, d):
    c = Cache([20, 64, 100], 2, d, seed=2, spare=5, extra_width=1).fill()
    c.table[:] = np.arange(9).reshape(3, 3)  # (no page twice)
    blocks, codes, table = c.gpu()
    x = torch.ones(8, 2, d, dtype=torch.bfloat16, device=DEV)
    status = i32([0])
    M.kv_append_x8(blocks, codes, x, x, table, i32([20, 64, 100]), cu_q=i32(cu_q), status=status)
    torch.cuda.synchronize()
    assert status.item() == _lib.KV_STATUS_LENGTH
    assert np.array_equal(blocks.cpu().numpy(), c.blocks) and np.array_equal(codes.cpu().numpy(), c.codes)
    M.kv_append_x8(blocks, codes, x, x, table, i32([20, 64, 100]), cu_q=i32(cu_q))  # (without a status)
    torch.cuda.synchronize()
    assert np.array_equal(blocks.cpu().numpy(), c.blocks) and np.array_equal(codes.cpu().numpy(), c.codes)


# ---------------------------------------------------------------- the attention
def _check_attn(c, n, heads, window=0, sinks=0, cu=True, q=None, max_q=None, lens=None, scale=None, ws=None, tiny=0.0):
    lens = c.lens if lens is None else lens
    cu_q = np.concatenate(([0], np.cumsum(n))).tolist()
    t = cu_q[-1]
    if q is None:
        q = torch.from_numpy(2 * c.rng.standard_normal((t, heads, c.d))).bfloat16().to(DEV)
    blocks, codes, table = c.gpu()
    lse = torch.full((t, heads), 7.0, device=DEV)
    status = i32([0])
    ws = M.attn_x8_workspace(DEV) if ws is None else ws
    args = dict(cu_q=i32(cu_q) if cu else None, max_q=max(max(n), 1) if max_q is None else max_q, scale=scale,
                window=window, sinks=sinks, workspace=ws, status=status)
    out, got_lse = M.attn_x8(q, blocks, codes, table, i32(lens), lse=lse, **args)
    torch.cuda.synchronize()
    assert status.item() == 0 and got_lse is lse
    s = c.d ** -0.5 if scale is None else scale
    want, wl, spread, slack = A.attention(f64(q), A.cache_values(c.blocks, c.codes), c.table, lens, cu_q, s,
                                          window, sinks)
    got, gl = f64(out), f64(lse)
    bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -20 + 2 * slack[..., None]) * spread + tiny
    assert np.isfinite(got).all()
    assert (np.abs(got - want) <= bound).all(), float((np.abs(got - want) - bound).max())
    empty = np.isinf(wl)
    assert np.array_equal(np.isinf(gl), empty) and (gl[empty] < 0).all() and (got[empty] == 0).all()
    tol = slack + (max(lens) / 8 + 64) * 2.0 ** -24 + 2.0 ** -22 * (1 + np.abs(wl))
    assert (np.abs(gl[~empty] - wl[~empty]) <= tol[~empty]).all()
    again, _ = M.attn_x8(q, blocks, codes, table, i32(lens), **args)  # and the same bits again
    assert torch.equal(again, out)
    return out, lse


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("kvh,group", [(1, 1), (2, 5), (3, 8), (1, 16), (2, 13)])
def test_attention_single_tokens(kvh, group, d):
    c = Cache([1, 64, 65, 7, 200, 128], kvh, d, seed=group).fill()
    _check_attn(c, [1] * 6, kvh * group, cu=False)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n,lens", [
    ([3, 0, 8, 1], [70, 64, 8, 500]),   # a sequence without rows, one that is all query rows
    ([5, 2], [3, 0]),                   # more rows than tokens: rows that see nothing
    ([48], [190]), ([20, 1, 7], [64, 129, 63]),
])
@pytest.mark.parametrize("group", [1, 5, 8])
def test_attention_several_tokens(n, lens, group, d):
    c = Cache(lens, 2, d, seed=d + group).fill()
    _check_attn(c, n, 2 * group)


@pytest.mark.parametrize("window,sinks", [(1, 0), (64, 0), (65, 1), (100, 64), (7, 130), (1000, 5), (130, 0)])
@pytest.mark.parametrize("n", [[1, 1, 1], [6, 3, 9]])
def test_attention_window_and_sinks(window, sinks, n):
    c = Cache([640, 130, 65], 2, 128, seed=window).fill()
    _check_attn(c, n, 10, window, sinks)
    _check_attn(c, n, 2, window, sinks)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 5, 2 ** 30, 192, 191])
@pytest.mark.parametrize("n,lens", [([8], [1]), ([7, 10, 1], [5, 3, 150]), ([40, 30], [33, 2])])
def test_attention_window_beyond_every_length(n, lens, window, d):
    """Windows up to the largest int with rows before the first token: position -
    window stays in range, and the rows that see tokens see all of them."""
    c = Cache(lens, 1, d, seed=len(n), extra_width=3 - max(-(-max(lens) // PAGE), 1)).fill()
    assert c.table.shape[1] == 3  # 192 tokens at most
    for heads in (1, 3):  # (by the rows per key/value head: few, shared pages, many)
        q = torch.from_numpy(c.rng.standard_normal((sum(n), heads, d))).bfloat16().to(DEV)
        plain, _ = _check_attn(c, n, heads, q=q)
        out, _ = _check_attn(c, n, heads, window, 2, q=q)
        assert torch.equal(out, plain)


def test_attention_one_long_sequence_over_all_ctas():
    c = Cache([20000], 1, 64, seed=5).fill()
    ws = M.attn_x8_workspace(DEV)
    for _ in range(2):  # the workspace is ready again after each call
        _check_attn(c, [1], 5, cu=False, ws=ws)
    assert not ws[:4096].any()


def test_attention_many_short_sequences():
    rng = np.random.default_rng(0)
    lens = rng.integers(0, 90, 600).tolist()
    c = Cache(lens, 1, 64).fill()
    _check_attn(c, [1] * 600, 3, cu=False)


def test_attention_variants_agree():
    """max_q only picks the kernel: one row, two tiles, shared pages."""
    c = Cache([700, 90], 2, 128, seed=9).fill()
    q = torch.from_numpy(c.rng.standard_normal((2, 6, 128))).bfloat16().to(DEV)
    for max_q in (1, 4, 20, 40):
        _check_attn(c, [1, 1], 6, q=q, max_q=max_q)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(0, 0), (150, 5)])
def test_attention_kernels_agree(window, sinks, d):
    """The same rows in every kernel: a sequence of 40 rows leaves max_q of 1, 2, 4
    and 40 (6, 12, 24 and 240 rows per key/value head) as they are given. Their
    weights are rounded in other places: within both bounds of one another."""
    c = Cache([700, 90, 300], 2, d, seed=9).fill()
    n = [1, 40, 2]
    q = torch.from_numpy(c.rng.standard_normal((43, 12, d))).bfloat16().to(DEV)
    outs = [_check_attn(c, n, 12, window, sinks, q=q, max_q=max_q) for max_q in (1, 2, 4, 40)]
    want, _, spread, slack = A.attention(f64(q), A.cache_values(c.blocks, c.codes), c.table, c.lens, [0, 1, 41, 43],
                                         d ** -0.5, window, sinks)
    bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -20 + 2 * slack[..., None]) * spread
    seen = [f64(o) for o, _ in outs]
    for i in range(4):
        for j in range(i):
            assert (np.abs(seen[i] - seen[j]) <= 2 * bound).all()
    # (not one kernel four times: some roundings differ)
    assert any(not np.array_equal(seen[i], seen[0]) for i in range(1, 4))


@pytest.mark.parametrize("amp,qamp", [(40.0, 1.0), (1.0, 2.0 ** 60), (2.0 ** -60, 1.0), (1.0, 0.0)])
def test_attention_peaked_flat_and_far_scales(amp, qamp):
    """Scores of hundreds, rows of large, tiny and zero values."""
    c = Cache([300, 64], 2, 128, seed=1).fill(amp)
    q = torch.from_numpy(qamp * c.rng.standard_normal((2, 4, 128))).bfloat16().to(DEV)
    _check_attn(c, [1, 1], 4, q=q, scale=128 ** -0.5 / max(qamp, 1.0))


def test_attention_long_tail_is_kept():
    """One token 2^-17 times heavier than each of 6000 others: the others still
    hold their share (8-bit weights would lose it)."""
    c = Cache([6001], 1, 64, seed=2)
    k = np.zeros((6001, 1, 64))
    k[0, 0, 0] = 448.0
    v = np.ones((6001, 1, 64))
    v[0] = -1.0
    c.blocks, c.codes = A.append(c.blocks, c.codes, k, v, c.table, [0], [0, 6001])
    q = torch.zeros(1, 1, 64, dtype=torch.bfloat16, device=DEV)
    q[0, 0, 0] = 1.0
    _check_attn(c, [1], 1, cu=False, q=q, scale=17 * np.log(2) / 448)


def test_attention_nan_stays_where_it_is_masked():
    """A NaN token is seen by the rows after it only, also on the same page and
    in the same tile of rows; one outside the window by none."""
    c = Cache([200], 1, 128, seed=4).fill()
    blocks, codes, table = c.gpu()
    q = torch.from_numpy(c.rng.standard_normal((6, 3, 128))).bfloat16().to(DEV)
    key, value = A.image_bytes(128)
    clean, _ = M.attn_x8(q, blocks, codes, table, i32([200]), cu_q=i32([0, 6]), max_q=6)
    page = c.table[0, 197 // 64]
    for kind, image in ((0, key), (1, value)):
        b = blocks.clone()
        b[page, 0, kind, torch.from_numpy(image[197 % 64]).to(DEV)] = 0x7F
        out, _ = M.attn_x8(q, b, codes, table, i32([200]), cu_q=i32([0, 6]), max_q=6)
        torch.cuda.synchronize()
        assert torch.equal(out[:3], clean[:3])  # rows 194, 195, 196
        assert torch.isnan(out[3:]).all()
    clean, _ = M.attn_x8(q, blocks, codes, table, i32([200]), cu_q=i32([0, 6]), max_q=6, window=20, sinks=2)
    b = blocks.clone()
    for t in (2, 100, 174):
        for kind, image in ((0, key), (1, value)):
            b[c.table[0, t // 64], 0, kind, torch.from_numpy(image[t % 64]).to(DEV)] = 0x7F
    out, _ = M.attn_x8(q, b, codes, table, i32([200]), cu_q=i32([0, 6]), max_q=6, window=20, sinks=2)
    assert torch.equal(out, clean)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("n,group", [(7, 5), (23, 8)])  # one tile of rows, two
@pytest.mark.parametrize("steps", [[0, 3, 6, 9, 12, 15], [15, 12, 9, 6, 3, 0], [4, 0, 9, 9, 1, 7]])
def test_attention_many_rows_scales_that_differ_by_page(d, n, group, steps):
    """Keys and values 2^0 .. 2^7.5 apart from page to page, in rising, falling and
    mixed order: running maxima far above the first page's, value scales on
    both sides of the ones before. Where every token of weight has a zero, the
    others' e^-130 of a value is below fp32's smallest normal number, 2^-126."""
    c = Cache([6 * PAGE - 3], 2, d, seed=sum(steps) + n)
    grow = np.repeat(2.0 ** (np.array(steps) / 2), PAGE)[:c.lens[0], None, None]
    k = grow * c.rng.standard_normal((c.lens[0], 2, d)) / 4
    v = grow * c.rng.standard_normal((c.lens[0], 2, d))
    c.blocks, c.codes = A.append(c.blocks, c.codes, A.bf16_rne(k), A.bf16_rne(v), c.table, [0], [0, c.lens[0]])
    _check_attn(c, [n], 2 * group, tiny=2.0 ** -126)


def _check_long_runs(c, n, heads, q, window=0, scale=None):
    """c's one sequence as it is (its pages spread over the CTAs), and so many
    times in one call that a CTA walks many pages of an item: each copy against
    the oracle. Returns the copies' rows."""
    s = c.d ** -0.5 if scale is None else scale
    want, _, spread, slack = A.attention(f64(q), A.cache_values(c.blocks, c.codes), c.table, c.lens, [0, n], s, window)
    bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -20 + 2 * slack[..., None]) * spread + 2.0 ** -126
    blocks, codes, table = c.gpu()
    most = -(-300 // c.kvh)
    for times in (1, most):
        out, _ = M.attn_x8(q.to(DEV).repeat(times, 1, 1), blocks, codes, table.repeat(times, 1), i32(c.lens * times),
                           cu_q=i32([n * i for i in range(times + 1)]), max_q=n, window=window, scale=scale)
        out = out.view(times, n, heads, c.d)
        excess = (out.double() - torch.from_numpy(want).to(DEV)).abs() - torch.from_numpy(bound).to(DEV)
        assert (excess <= 0).all(), excess.max().item()
    return out


def _paged_values(c, steps, dims, d, loud_key=None):
    """Fills c's one sequence: values of page i times 2^steps[i], where steps[i] is
    not 0 in the first `dims` dims only (0 elsewhere: what the quiet pages hold
    there is all there is). loud_key: dim 0 of the keys of pages with steps[i] > 0."""
    e = np.array(steps)[np.arange(c.lens[0]) // PAGE]
    k = c.rng.standard_normal((e.size, c.kvh, d)) / 2
    v = c.rng.standard_normal((e.size, c.kvh, d)) * 2.0 ** e[:, None, None]
    v[e != 0, :, dims:] = 0.0
    if loud_key is not None:
        k[e > 0, :, 0] = loud_key
    c.blocks, c.codes = A.append(c.blocks, c.codes, A.bf16_rne(k), A.bf16_rne(v), c.table, [0], [0, c.lens[0]])


LOUD = [[60, 0, 0, 0, 0, 0], [0, 0, 60, 0, 0, 0], [0, 0, 0, 0, 0, 60], [60, 0, 60, 0, 60, 0],
        [0, -60, 0, -60, 60, 0], [0, 20, 40, 60, 40, 0], [0, 12, 0, 9, 0, 25], [8, 0, 4, 0, 8, 1]]


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n,group", [(3, 1), (7, 5), (23, 8)])  # few rows, one tile, two
@pytest.mark.parametrize("steps", LOUD)
def test_attention_loud_pages_keep_the_others(steps, n, group, d):
    """Pages up to 2^60 louder than the others (2^120 between two), with values in
    8 dims: in all other dims the quiet pages' values are the whole answer."""
    c = Cache([6 * PAGE - 3], 2, d, seed=len(steps) + n)
    _paged_values(c, steps, 8, d)
    _check_long_runs(c, n, 2 * group, torch.from_numpy(c.rng.standard_normal((n, 2 * group, d))).bfloat16())


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n,group", [(3, 1), (7, 5), (23, 8)])
@pytest.mark.parametrize("loud", [30, 110])
@pytest.mark.parametrize("at", [0, 2, 5])
def test_attention_loud_pages_without_weight(at, loud, n, group, d):
    """A page 2^30 or 2^110 louder whose scores lie some 290 log2 units below the others':
    its share is nothing, and so is its trace."""
    c = Cache([6 * PAGE - 3], 2, d, seed=at + n)
    steps = [0] * 6
    steps[at] = loud
    _paged_values(c, steps, 8, d, loud_key=-448.0)
    q = torch.from_numpy(c.rng.standard_normal((n, 2 * group, d)) / 2).bfloat16()
    q[..., 0] = 3.0
    _check_long_runs(c, n, 2 * group, q, scale=0.15)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("group", [1, 8])
@pytest.mark.parametrize("loud", [30, 110])
def test_attention_loud_pages_behind_the_mask(loud, group, d):
    """A loud page before the window of some rows and in that of others, and a loud
    page that only the last rows are past: rows that mask it keep their bits."""
    kv, n, window = 6 * PAGE - 10, 120, 160
    c = Cache([kv], 1, d, seed=group)
    steps = [0] * 6
    steps[1] = steps[5] = loud
    _paged_values(c, steps, d, d)
    q = torch.from_numpy(c.rng.standard_normal((n, group, d))).bfloat16()
    out = _check_long_runs(c, n, group, q, window)
    quiet = Cache([kv], 1, d, seed=group)
    _paged_values(quiet, steps, d, d)
    quiet.codes[quiet.table[0, [1, 5]], 0, 1] -= loud
    same = _check_long_runs(quiet, n, group, q, window)
    pos = kv - n + np.arange(n)
    masks = torch.from_numpy((pos - window + 1 >= 2 * PAGE) & (pos < 5 * PAGE))
    assert 0 < masks.sum() < n
    assert torch.equal(out[:, masks], same[:, masks])


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n,group", [(1, 5), (2, 8), (9, 8)])
@pytest.mark.parametrize("kv", [300, 9001])  # one CTA's pages; parts of many
@pytest.mark.parametrize("amp", [2.0 ** 119, 2.0 ** 100, 2.0 ** -100, 2.0 ** -116])
def test_attention_values_near_the_ends_of_the_range(amp, kv, n, group, d):
    """Values up to bf16's largest and down to its smallest normal ones; what is
    below that is rounded to bf16's multiples of 2^-133."""
    c = Cache([kv], 1, d, seed=n)
    k = c.rng.standard_normal((kv, 1, d)) / 2
    v = amp * np.clip(c.rng.standard_normal((kv, 1, d)), -5, 5)
    c.blocks, c.codes = A.append(c.blocks, c.codes, A.bf16_rne(k), A.bf16_rne(v), c.table, [0], [0, kv])
    _check_attn(c, [n], group, tiny=2.0 ** -133)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("n,group", [(3, 16), (17, 8)])
def test_attention_many_rows_of_one_long_sequence(d, n, group):
    c = Cache([9001], 1, d, seed=n).fill()
    ws = M.attn_x8_workspace(DEV)
    _check_attn(c, [n], group, ws=ws)
    _check_attn(c, [n], group, window=5000, sinks=70, ws=ws)


@pytest.mark.parametrize("d", [64, 128, 256])
def test_attention_ragged_batch_of_many_rows(d):
    """Items of one and of two tiles of rows, none and many pages, in the same runs."""
    rng = np.random.default_rng(d)
    n = rng.integers(0, 12, 40)
    n[::9] = rng.integers(20, 40, n[::9].size)
    lens = rng.integers(0, 900, 40)
    lens[5] = 0
    c = Cache(lens.tolist(), 2, d, seed=d).fill()
    _check_attn(c, n.tolist(), 2 * 8)


@pytest.mark.parametrize("d", [64, 128])
@pytest.mark.parametrize("group", [3, 8])
def test_attention_short_items_of_rows_of_other_sizes(group, d):
    """400 items of one to three pages, several in turn on a CTA, the rows of
    neighbours 2^20 apart: an item scaled by another's factors shows."""
    rng = np.random.default_rng(group)
    n = rng.integers(24 // group, 24 // group + 5, 200)
    lens = np.maximum(rng.integers(1, 190, 200), n)
    c = Cache(lens.tolist(), 2, d, seed=d).fill()
    amp = np.repeat(2.0 ** (10 * (np.arange(200) % 3 - 1)), n)[:, None, None]
    q = torch.from_numpy(amp * c.rng.standard_normal((n.sum(), 2 * group, d))).bfloat16().to(DEV)
    _check_attn(c, n.tolist(), 2 * group, q=q, scale=2.0 ** -10 * d ** -0.5)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("window,sinks", [(0, 0), (40, 0), (300, 3)])
def test_attention_many_rows_see_their_nan_only(d, window, sinks):
    """A NaN token every 61 over many pages that causality and the window cut:
    the rows that see one are NaN, the others keep their bits."""
    kv, n = 700, 500
    c = Cache([kv], 1, d, seed=12).fill()
    blocks, codes, table = c.gpu()
    q = torch.from_numpy(c.rng.standard_normal((n, 1, d))).bfloat16().to(DEV)
    args = dict(cu_q=i32([0, n]), max_q=n, window=window, sinks=sinks)
    clean, _ = M.attn_x8(q, blocks, codes, table, i32([kv]), **args)
    key, value = A.image_bytes(d)
    bad = list(range(330, kv, 61))
    hit = [any(t in bad for t in A.visible(kv - n + i, kv, window, sinks)) for i in range(n)]
    assert any(hit) and not all(hit)
    hit = torch.tensor(hit, device=DEV)
    for kind, image in ((0, key), (1, value)):
        b = blocks.clone()
        for t in bad:
            b[c.table[0, t // PAGE], 0, kind, torch.from_numpy(image[t % PAGE]).to(DEV)] = 0x7F
        out, _ = M.attn_x8(q, b, codes, table, i32([kv]), **args)
        torch.cuda.synchronize()
        assert torch.isnan(out[hit]).all() and torch.equal(out[~hit], clean[~hit])


@pytest.mark.parametrize("d", [64, 128, 256])
def test_attention_many_rows_report_bad_pages_and_lengths(d):
    c = Cache([400, 70], 1, d, seed=3).fill()
    q = torch.from_numpy(c.rng.standard_normal((2 * 9, 4, d))).bfloat16().to(DEV)
    blocks, codes, _ = c.gpu()
    ws = M.attn_x8_workspace(DEV)

    def call(table, lens):
        status = i32([0])
        out, _ = M.attn_x8(q, blocks, codes, torch.from_numpy(table).to(DEV), i32(lens), cu_q=i32([0, 9, 18]),
                           max_q=9, workspace=ws, status=status)
        torch.cuda.synchronize()
        return out, status.item()

    good, st = call(c.table, [400, 70])
    assert st == 0
    for bad in (-1, c.pages, 1 << 30):
        t = c.table.copy()
        t[0, 1] = bad
        out, st = call(t, [400, 70])
        assert st == _lib.KV_STATUS_PAGE and torch.equal(out[9:], good[9:]) and torch.isfinite(out).all()
    out, st = call(c.table, [-4, 70])
    assert st == _lib.KV_STATUS_LENGTH and (out[:9] == 0).all() and torch.equal(out[9:], good[9:])


def test_attention_row_of_nan_queries_touches_no_other():
    c = Cache([100, 100], 1, 128, seed=6).fill()
    q = torch.from_numpy(c.rng.standard_normal((2, 4, 128))).bfloat16().to(DEV)
    blocks, codes, table = c.gpu()
    a, _ = M.attn_x8(q, blocks, codes, table, i32([100, 100]))
    q2 = q.clone()
    q2[0, 1, 3], q2[1, 2, 0] = float("nan"), float("inf")
    b, _ = M.attn_x8(q2, blocks, codes, table, i32([100, 100]))
    a, b = a.clone(), b.clone()
    for t in (a, b):
        t[0, 1] = 0
        t[1, 2] = 0
    assert torch.equal(a, b)


def test_attention_strided_queries_and_other_stream():
    c = Cache([150, 33], 2, 64, seed=8).fill()
    wide = torch.from_numpy(c.rng.standard_normal((2, 10, 64))).bfloat16().to(DEV)
    q = wide[:, :6]
    a, _ = _check_attn(c, [1, 1], 6, q=q)
    blocks, codes, table = c.gpu()
    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(s):
        b, _ = M.attn_x8(q, blocks, codes, table, i32([150, 33]), cu_q=i32([0, 1, 2]), max_q=1)
    s.synchronize()
    assert torch.equal(a, b)


def test_attention_reports_bad_pages_and_lengths():
    c = Cache([200, 70], 1, 64, seed=3).fill()
    q = torch.from_numpy(c.rng.standard_normal((2, 2, 64))).bfloat16().to(DEV)
    blocks, codes, _ = c.gpu()
    ws = M.attn_x8_workspace(DEV)

    def call(table, lens):
        status = i32([0])
        out, _ = M.attn_x8(q, blocks, codes, torch.from_numpy(table).to(DEV), i32(lens), workspace=ws, status=status)
        torch.cuda.synchronize()
        return out, status.item()

    good, st = call(c.table, [200, 70])
    assert st == 0
    for bad in (-1, c.pages, 1 << 30):
        t = c.table.copy()
        t[0, 1] = bad
        out, st = call(t, [200, 70])
        assert st == _lib.KV_STATUS_PAGE and torch.equal(out[1], good[1]) and torch.isfinite(out).all()
    width = c.table.shape[1] * 64
    out, st = call(c.table, [-4, 70])
    assert st == _lib.KV_STATUS_LENGTH and (out[0] == 0).all() and torch.equal(out[1], good[1])
    full = Cache([width, 70], 1, 64, seed=3).fill()
    blocks, codes, _ = full.gpu()
    good, st = call(full.table, [width, 70])
    out, st2 = call(full.table, [width + 5, 70])
    assert (st, st2) == (0, _lib.KV_STATUS_LENGTH) and torch.equal(out, good)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("max_q", [1, 8, 40])
def test_attention_refuses_row_starts_that_do_not_ascend(d, max_q):
    c = Cache([100, 100, 100], 1, d, seed=2).fill()
    q = torch.ones(8, 2, d, dtype=torch.bfloat16, device=DEV)
    blocks, codes, table = c.gpu()
    ws = M.attn_x8_workspace(DEV)
    out = torch.full_like(q, 5.0)
    status = i32([0])
    M.attn_x8(q, blocks, codes, table, i32(c.lens), cu_q=i32([0, 6, 2, 8]), max_q=max_q, out=out, workspace=ws,
              status=status)
    torch.cuda.synchronize()
    assert status.item() == _lib.KV_STATUS_LENGTH and (out == 5).all()
    status.zero_()
    M.attn_x8(q, blocks, codes, table, i32(c.lens), cu_q=i32([0, 6, 6, 8]), max_q=max_q, out=out, workspace=ws,
              status=status)
    torch.cuda.synchronize()
    assert status.item() == 0 and torch.isfinite(out).all() and not (out == 5).all()


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("max_q", [1, 2, 8, 40])  # 2, 4, 16 and 80 rows: each kernel
@pytest.mark.parametrize("cu_q", [[0, 30, 10, 40], [0, 20, 19, 21], [0, 40, 0, 40], [5, 0, 40, 40]])
def test_attention_refuses_any_fall_of_the_row_starts(cu_q, max_q, d):
    """Also where the sequences' rows together are no more than the call's, and in
    every kernel (by max_q of 40 rows)."""
    c = Cache([100, 100, 100], 1, d, seed=2).fill()
    q = torch.ones(40, 2, d, dtype=torch.bfloat16, device=DEV)
    blocks, codes, table = c.gpu()
    ws = M.attn_x8_workspace(DEV)
    out = torch.full_like(q, 5.0)
    status = i32([0])
    args = dict(max_q=max_q, out=out, workspace=ws, status=status)
    M.attn_x8(q, blocks, codes, table, i32(c.lens), cu_q=i32(cu_q), **args)
    torch.cuda.synchronize()
    assert status.item() == _lib.KV_STATUS_LENGTH and (out == 5).all()
    status.zero_()
    M.attn_x8(q, blocks, codes, table, i32(c.lens), cu_q=i32([0, 30, 30, 40]), **args)
    torch.cuda.synchronize()
    assert status.item() == 0 and torch.isfinite(out).all() and not (out == 5).all()
    assert not ws[:4096].any()


def test_bindings_refuse_wrong_tensors():
    """Wrong types, shapes, devices and strides, one argument at a time."""
    d = 64
    x = torch.zeros(3, 96, dtype=torch.bfloat16, device=DEV)
    norm = dict(x=x, residual=x.clone(), norm_w=x[0].clone(), res_out=x.clone(),
                x8=torch.zeros(3, 96, dtype=torch.uint8, device=DEV),
                codes=torch.zeros(3, 3, dtype=torch.uint8, device=DEV), normed=x.clone())
    blocks, codes = M.kv_cache_x8(2, 2, d, DEV)
    k = torch.zeros(2, 2, d, dtype=torch.bfloat16, device=DEV)
    seqs = dict(page_table=i32([[0], [1]]), cu_q=i32([0, 1, 2]), status=i32([0]))
    append = dict(blocks=blocks, codes=codes, k=k, v=k.clone(), start=i32([0, 0]), **seqs)
    attn = dict(q=torch.zeros(2, 4, d, dtype=torch.bfloat16, device=DEV), blocks=blocks, codes=codes, kv_len=i32([1, 1]),
                out=torch.zeros(2, 4, d, dtype=torch.bfloat16, device=DEV),
                lse=torch.zeros(2, 4, device=DEV), workspace=M.attn_x8_workspace(DEV), **seqs)
    for fn, args in ((M.add_norm_x8, norm), (M.kv_append_x8, append), (M.attn_x8, attn)):
        fn(**args)
        for name, t in args.items():
            bad = [t.cpu(), t.unsqueeze(0), 5]
            if name != "workspace":  # (any type, any shape)
                bad += [t.double(), t.flatten()[:-1]]
            if t.dim() > 1:
                bad.append(t.transpose(-1, -2).contiguous().transpose(-1, -2))
            for b in bad[:-2] if name == "workspace" else bad:
                if isinstance(b, torch.Tensor) and b.shape == t.shape and b.stride() == t.stride() \
                        and b.dtype == t.dtype and b.device == t.device:
                    continue  # (one column: still contiguous)
                with pytest.raises(ValueError):
                    fn(**{**args, name: b})
    for name, b in (("max_q", 2 ** 40), ("window", 2 ** 31), ("sinks", -2 ** 40)):
        with pytest.raises(ValueError):
            M.attn_x8(**{**attn, name: b})
    with pytest.raises(_lib.MoeError):
        M.attn_x8(**{**attn, "window": -1})
    with pytest.raises(_lib.MoeError):
        M.attn_x8(**{**attn, "workspace": attn["workspace"][:4096]})
    with pytest.raises(TypeError):
        M.attn_x8(**{**attn, "scale": "1"})
    with pytest.raises(ValueError):
        M.kv_append_x8(**{**append, "cu_q": None, "page_table": i32([[0]]), "start": i32([0])})
    torch.cuda.synchronize()


def test_append_then_attention_in_a_graph():
    """A decode step captured once and replayed as the sequences grow."""
    d, kvh, heads = 128, 2, 10
    c = Cache([130, 64], kvh, d, seed=11, extra_width=1).fill()
    c.table[1, 1] = [p for p in range(c.pages) if p not in set(c.table[0, :3]) | {c.table[1, 0]}][0]
    blocks, codes, table = c.gpu()
    start, lens = i32([130, 64]), i32([131, 65])
    x = torch.zeros(2, 2, kvh, d, dtype=torch.bfloat16, device=DEV)
    q = torch.zeros(2, heads, d, dtype=torch.bfloat16, device=DEV)
    out = torch.empty_like(q)
    ws = M.attn_x8_workspace(DEV)

    def step():
        M.kv_append_x8(blocks, codes, x[:, 0], x[:, 1], table, start)
        M.attn_x8(q, blocks, codes, table, lens, out=out, workspace=ws)
        start.add_(1)
        lens.add_(1)

    s = torch.cuda.Stream()
    s.wait_stream(torch.cuda.current_stream())
    keep = [t.clone() for t in (blocks, codes, start, lens)]
    with torch.cuda.stream(s):
        step()
    torch.cuda.current_stream().wait_stream(s)
    for t, k in zip((blocks, codes, start, lens), keep):
        t.copy_(k)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    hb, hc = c.blocks, c.codes
    for i in range(3):
        xn = torch.from_numpy(c.rng.standard_normal(tuple(x.shape)) * 4 ** i).bfloat16()
        qn = torch.from_numpy(c.rng.standard_normal(tuple(q.shape))).bfloat16()
        x.copy_(xn)
        q.copy_(qn)
        graph.replay()
        torch.cuda.synchronize()
        at = [130 + i, 64 + i]
        hb, hc = A.append(hb, hc, f64(xn)[:, 0], f64(xn)[:, 1], c.table, at, [0, 1, 2])
        want, _, spread, slack = A.attention(f64(qn), A.cache_values(hb, hc), c.table, [a + 1 for a in at],
                                             [0, 1, 2], d ** -0.5)
        bound = 2.0 ** -8 * np.abs(want) + (2.0 ** -11 + 2.0 ** -20 + 2 * slack[..., None]) * spread
        assert (np.abs(f64(out) - want) <= bound).all()
