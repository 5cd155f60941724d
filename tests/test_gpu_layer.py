"""The layer's operators (norms around a block, rotary positions alone and with
the cache's append, products with 4-bit weights) against the float64 oracle.

Bounds (half a step of bf16, with its 8 significant bits, is 2^-8 of the value):
* norm_add_norm: the new residual rows within 2^-8 of their value (the one
  rounding) plus 2^-17 of the block's part and of the residual's (fp32: a sum
  of at most 8192 squares in chains of 64 and a tree, some 80 roundings, halved
  by the root, rsqrtf's two units, five products: below 2^-18); the norm of
  what came out as tests/test_gpu_attention.py, its bytes and codes bit for bit.
* rope: 2^-8 of the value plus 2^-21 scale (|u| + |v|): the angle to 2^-33
  turns (7e-10 radians), the series' left-out terms (2.5e-8), and the fp32
  roundings of sine, cosine and of the two products (some 2^-23 in all).
* rope_kv_append: bit for bit rope and append one after the other.
* linear: 2^-8 of the value plus (K / 32 2^-23 + 2^-19) sum |x| |w|: products are
  exact, K / 32 times 32 of them are added to an fp32 sum, each time within a
  unit of it, and within a product's 33 terms 2^-24 of the largest each; bf16
  rows also 2^-21 of their group's largest value for every column (what lo's
  subnormals leave).
"""

import numpy as np
import pytest
import torch

import mxfp8_moe_decode_gb300 as M
from mxfp8_moe_decode_gb300 import _lib
from oracle import layer as L
from oracle import moe as O
from oracle.numerics import e4m3_decode

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


def f64(t):
    return t.detach().cpu().double().numpy()


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------- norms around a block
def _norm_case(m, h, gate, post=True, seed=0, pad=0):
    g = torch.Generator().manual_seed(seed + 7 * m + h)

    def draw(*shape, amp=1.0):
        return (amp * torch.randn(*shape, generator=g)).bfloat16().to(DEV)

    x, r = draw(m, h + pad)[:, :h], draw(m, h + 2 * pad, amp=3.0)[:, :h]
    post_w = (1 + 0.1 * torch.randn(h, generator=g)).bfloat16().to(DEV) if post else None
    w = (1 + 0.1 * torch.randn(h, generator=g)).bfloat16().to(DEV)
    gt = {"none": None, "channel": draw(h), "row": draw(m, h + pad)[:, :h], "one": draw(1, h).expand(m, h)}[gate]
    return x, r, post_w, w, gt


def _check_norm(x, r, post_w, w, gate, rs=0.75, bs=1.5, eps=1e-6, **kw):
    normed = torch.empty(x.shape, dtype=torch.bfloat16, device=DEV)
    res, x8, codes, n = M.norm_add_norm_x8(x, r, post_w, w, gate=gate, res_scale=rs, block_scale=bs, eps=eps, normed=normed, **kw)
    torch.cuda.synchronize()
    assert n is normed
    r64 = f64(r) if "res_out" not in kw or kw["res_out"] is not r else kw["was"]
    want, block = L.block_residual(f64(x), r64, None if post_w is None else f64(post_w),
                                   None if gate is None else f64(gate), rs, bs, eps)
    assert (np.abs(f64(res) - want) <= 2.0 ** -8 * np.abs(want) + 2.0 ** -17 * (np.abs(block) + np.abs(rs * r64))).all()
    ys = O.attn_norm(f64(res), f64(w), eps)
    top = np.abs(ys).max(-1, keepdims=True)
    assert (np.abs(f64(normed) - ys) <= 1e-5 * top + 2.0 ** -8 * np.abs(ys)).all()
    for lo in range(0, x.shape[0], 48):
        s8, sc, _ = M.attn_seam_x8(res[lo:lo + 48].contiguous(), w, eps)
        assert torch.equal(x8[lo:lo + 48], s8) and torch.equal(codes[lo:lo + 48], sc)
    return res, x8, codes


@pytest.mark.parametrize("gate", ["none", "channel", "row", "one"])
@pytest.mark.parametrize("m,h", [(1, 32), (3, 96), (48, 1024), (5, 1056), (2, 5120), (131, 2080), (1, 8192)])
def test_norm_add_norm(m, h, gate):
    _check_norm(*_norm_case(m, h, gate))


@pytest.mark.parametrize("gate", ["none", "row"])
def test_norm_add_norm_without_post_norm(gate):
    _check_norm(*_norm_case(9, 640, gate, post=False))
    # with nothing in front it is add_norm_x8, bit for bit
    x, r, _, w, _ = _norm_case(9, 640, "none", post=False)
    a, b = M.norm_add_norm_x8(x, r, None, w), M.add_norm_x8(x, r, w)
    assert all(torch.equal(p, q) for p, q in zip(a[:3], b[:3]))


def test_norm_add_norm_strided_rows_and_in_place():
    x, r, pw, w, g = _norm_case(19, 1056, "row", pad=8)
    a = _check_norm(x, r, pw, w, g)
    r2, x2 = r.contiguous().clone(), x.contiguous().clone()
    kw = dict(gate=g, res_scale=0.75, block_scale=1.5)
    b = M.norm_add_norm_x8(x, r2, pw, w, res_out=r2, **kw)
    assert b[0] is r2 and b[3] is None and all(torch.equal(p, q) for p, q in zip(a, b[:3]))
    b = M.norm_add_norm_x8(x2, r, pw, w, res_out=x2, **kw)
    assert all(torch.equal(p, q) for p, q in zip(a, b[:3]))


def test_norm_add_norm_rows_apart():
    """A row of NaN or infinity leaves the others alone; rows of zeros and no rows are fine."""
    x, r, pw, w, g = _norm_case(9, 512, "row")
    a = M.norm_add_norm_x8(x, r, pw, w, gate=g)
    x2 = x.clone()
    x2[3, 5], x2[6, 100] = float("nan"), float("inf")
    b = M.norm_add_norm_x8(x2, r, pw, w, gate=g)
    keep = [0, 1, 2, 4, 5, 7, 8]
    for p, q in zip(a[:3], b[:3]):
        assert torch.equal(p[keep], q[keep])
    zero = torch.zeros_like(x)
    z = M.norm_add_norm_x8(zero, zero, pw, w)
    assert not z[0].any() and not z[1].any() and not z[2].any()
    e = M.norm_add_norm_x8(x[:0], r[:0], pw, w)
    assert e[0].shape == (0, 512) and e[2].shape == (0, 16)


def test_norm_add_norm_scales():
    x, r, pw, w, g = _norm_case(4, 256, "channel")
    _check_norm(x, r, pw, w, g, rs=0.0, bs=1.0)
    _check_norm(x, r, pw, w, g, rs=-1.0, bs=0.0)
    _check_norm(x, r, pw, w, g, rs=1.0, bs=1.0, eps=0.0)


# ---------------------------------------------------------------- rotary positions
def _freqs(rot, base=10000.0):
    return M.rope_freqs(rot, base, device=DEV)


def _check_rope(x, positions, freqs, first, interleaved, scale, out):
    whole = [int(v) % (1 << 64) for v in freqs.tolist()]
    want = L.rope(f64(x), positions.tolist(), whole, first, interleaved, scale)
    rot = 2 * len(whole)
    got = f64(out)
    still = np.ones(x.shape[2], bool)
    still[first:first + rot] = False
    assert np.array_equal(got[..., still], f64(x)[..., still])
    p = np.abs(f64(x)[..., first:first + rot])
    size = p + (p.reshape(*p.shape[:2], -1, 2)[..., ::-1].reshape(p.shape) if interleaved else np.roll(p, rot // 2, -1))
    a, b = got[..., first:first + rot], want[..., first:first + rot]
    assert (np.abs(a - b) <= 2.0 ** -8 * np.abs(b) + 2.0 ** -21 * abs(scale) * size + 2.0 ** -133).all()


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("tokens,heads,dim,rot,first", [
    (1, 1, 16, 16, 0), (1, 40, 128, 128, 0), (3, 5, 64, 32, 8), (7, 2, 256, 64, 192), (2, 3, 96, 48, 16),
    (5, 1, 1024, 1024, 0), (130, 9, 80, 16, 64), (4, 64, 192, 96, 0)])
def test_rope(tokens, heads, dim, rot, first, interleaved):
    g = torch.Generator().manual_seed(tokens + dim)
    x = torch.randn(tokens, heads, dim, generator=g).bfloat16().to(DEV)
    pos = torch.randint(-100, 200000, (tokens,), generator=g).int().to(DEV)
    f = _freqs(rot)
    _check_rope(x, pos, f, first, interleaved, 1.25, M.rope(x, pos, f, first, interleaved, 1.25))


def test_rope_far_positions_and_small_angles():
    """Any 32-bit position; the slowest pairs at the first ones (angles of 1e-4 to 1e-12)."""
    x = torch.randn(8, 2, 128, generator=torch.Generator().manual_seed(2)).bfloat16().to(DEV)
    x[:, :, :64] = 0  # (u = 0: the results are v times the sine alone)
    pos = i32([0, 1, -1, 3, 2 ** 31 - 1, -2 ** 31, 1000003, 16777217])
    f = _freqs(128, 1e6)
    _check_rope(x, pos, f, 0, False, 1.0, M.rope(x, pos, f))
    out = M.rope(x, pos, f)
    assert torch.equal(out[0], x[0])  # position 0: nothing moves


def test_rope_quarter_turns_are_exact():
    x = torch.randn(5, 3, 32, generator=torch.Generator().manual_seed(4)).bfloat16().to(DEV)
    f = torch.full((16,), 1 << 62, dtype=torch.int64, device=DEV)
    out = M.rope(x, i32([0, 1, 2, 3, 4]), f)
    u, v = x[..., :16], x[..., 16:]
    assert torch.equal(out[0], x[0]) and torch.equal(out[4], x[4]) and torch.equal(out[2], -x[2])
    assert torch.equal(out[1, :, :16], -v[1]) and torch.equal(out[1, :, 16:], u[1])
    assert torch.equal(out[3, :, :16], v[3]) and torch.equal(out[3, :, 16:], -u[3])


def test_rope_strided_rows_in_place_and_back():
    g = torch.Generator().manual_seed(9)
    qkv = torch.randn(33, 14, 64, generator=g).bfloat16().to(DEV)
    x, f = qkv[:, 2:12], _freqs(64)
    pos = torch.arange(33, dtype=torch.int32, device=DEV) * 777
    want = M.rope(x, pos, f)
    assert want.is_contiguous()
    room = torch.full((33, 20, 64), 7.0, dtype=torch.bfloat16, device=DEV)
    out = M.rope(x, pos, f, out=room[:, 4:14])
    assert torch.equal(out, want) and (room[:, :4] == 7).all() and (room[:, 14:] == 7).all()
    before = qkv.clone()
    same = M.rope(x, pos, f, out=x)
    assert same is x and torch.equal(x, want)
    assert torch.equal(qkv[:, :2], before[:, :2]) and torch.equal(qkv[:, 12:], before[:, 12:])
    with pytest.raises(_lib.MoeError):  # rows off 16 bytes
        M.rope(x, pos, f, out=room.as_strided(x.shape, (20 * 64 - 4, 64, 1)))


def test_rope_many_tokens_and_none():
    x = torch.randn(40000, 3, 32, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    pos = torch.arange(40000, dtype=torch.int32, device=DEV)
    f = _freqs(32)
    out = M.rope(x, pos, f)
    assert torch.equal(out[39990:], M.rope(x[39990:], pos[39990:], f))
    _check_rope(x[20000:20020], pos[20000:20020], f, 0, False, 1.0, out[20000:20020])
    assert M.rope(x[:0], pos[:0], f).shape == (0, 3, 32)


def test_rope_keeps_non_finite_values_apart():
    x = torch.ones(1, 2, 32, dtype=torch.bfloat16, device=DEV)
    x[0, 0, 3], x[0, 1, 20] = float("nan"), float("inf")
    out = f64(M.rope(x, i32([5]), _freqs(32)))
    bad = ~np.isfinite(out)
    assert bad[0, 0, [3, 19]].all() and bad[0, 1, [4, 20]].any() and bad.sum() <= 4


# ---------------------------------------------------------------- with the cache's append
def _append_case(had, new, heads, kvh, d, rot, first, interleaved, far, cu=True, seed=0, in_place=False):
    g = torch.Generator().manual_seed(seed + d + sum(new))
    need = [-(-(a + b) // 64) for a, b in zip(had, new)]
    pages = sum(need) + 2
    order = torch.randperm(pages, generator=g).int()
    table = torch.zeros(len(had), max(need + [1]), dtype=torch.int32)
    at = 0
    for b, n in enumerate(need):
        table[b, :n] = order[at:at + n]
        at += n
    t = sum(new)
    qkv = torch.randn(t, heads + 2 * kvh, d, generator=g).bfloat16().to(DEV)
    q, k, v = qkv.split((heads, kvh, kvh), dim=1)
    blocks = torch.randint(0, 256, (pages, kvh, 2, 64 * d), generator=g).to(torch.uint8)
    blocks[(blocks & 0x7F) == 0x7F] = 0  # (finite bytes)
    codes = torch.randint(100, 130, (pages, kvh, 2), generator=g).to(torch.uint8)
    starts = np.concatenate(([0], np.cumsum(new))).tolist()
    place = [had[b] + i for b in range(len(had)) for i in range(new[b])]
    f = _freqs(rot)
    pos = (torch.randint(0, 3000000, (t,), generator=g).int() if far else torch.tensor(place, dtype=torch.int32)).to(DEV)
    args = (table.to(DEV), i32(had))
    b1, c1, b2, c2 = blocks.to(DEV), codes.to(DEV), blocks.to(DEV), codes.to(DEV)
    cu_q = i32(starts) if cu else None
    want_q = M.rope(q, pos, f, first, interleaved, 0.9)
    M.kv_append_x8(b1, c1, M.rope(k, pos, f, first, interleaved, 0.9), v, *args, cu_q=cu_q)
    status = i32([0])
    kept = qkv.clone()
    out, b, c = M.rope_kv_append_x8(b2, c2, q, k, v, *args, f, cu_q=cu_q, positions=pos if far else None, first=first,
                                    interleaved=interleaved, scale=0.9, q_out=q if in_place else None, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0 and b is b2 and c is c2 and (out is q) == in_place
    assert torch.equal(out, want_q) and torch.equal(b1, b2) and torch.equal(c1, c2)
    assert torch.equal(qkv[:, heads:], kept[:, heads:])
    return b1, blocks


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("d,rot,first", [(64, 64, 0), (64, 16, 48), (128, 128, 0), (128, 48, 8), (256, 256, 0),
                                         (256, 64, 192)])
@pytest.mark.parametrize("had,new,far", [([0], [1], False), ([63, 5], [1, 1], True), ([5], [0], False),
                                         ([0, 60, 3, 0], [64, 8, 0, 1], False), ([1, 63, 0, 30], [200, 2, 130, 65], True)])
def test_rope_append(had, new, far, d, rot, first, interleaved):
    got, was = _append_case(had, new, 6, 2, d, rot, first, interleaved, far)
    assert sum(new) == 0 or not torch.equal(got.cpu(), was)
    if all(n == 1 for n in new):
        _append_case(had, new, 3, 3, d, rot, first, interleaved, far, cu=False, in_place=True)


def test_rope_append_many_sequences():
    rng = np.random.default_rng(3)
    had = rng.integers(0, 130, 300).tolist()
    _append_case(had, rng.integers(0, 3, 300).tolist(), 4, 1, 64, 64, 0, False, False)
    _append_case([4000 + 3 * i for i in range(48)], [1] * 48, 40, 8, 128, 128, 0, False, False, cu=False)


def test_rope_append_many_query_heads():
    """So much work that a thread takes several heads of a token."""
    _append_case([10, 100], [2500, 1500], 40, 2, 128, 128, 0, False, False)


def test_rope_append_leaves_rows_of_no_sequence():
    """Rows before the first sequence, behind the last and of a refused one stay as they were; row starts that fall
    write nothing at all."""
    d, f = 64, _freqs(64)
    table = i32([[0], [1], [2]])
    q = torch.randn(9, 2, d, generator=torch.Generator().manual_seed(1)).bfloat16().to(DEV)
    k = q[:, :1].contiguous()

    def run(cu, start):
        blocks, codes = torch.zeros(3, 1, 2, 64 * d, dtype=torch.uint8, device=DEV), torch.zeros(3, 1, 2, dtype=torch.uint8, device=DEV)
        out, status = torch.full_like(q, 7.0), i32([0])
        M.rope_kv_append_x8(blocks, codes, q, k, k, table, i32(start), f, cu_q=i32(cu), q_out=out, status=status)
        torch.cuda.synchronize()
        return out, blocks, status.item()

    out, blocks, status = run([1, 3, 3, 7], [0, 0, 5])
    assert status == 0 and (out[0] == 7).all() and (out[7:] == 7).all()
    assert torch.equal(out[1:3], M.rope(q[1:3], i32([0, 1]), f))
    assert torch.equal(out[3:7], M.rope(q[3:7], i32([5, 6, 7, 8]), f))
    out, _, status = run([0, 3, 6, 9], [0, -1, 2])
    assert status == _lib.KV_STATUS_LENGTH and (out[3:6] == 7).all()
    assert torch.equal(out[6:], M.rope(q[6:], i32([2, 3, 4]), f))
    out, blocks, status = run([0, 6, 3, 9], [0, 0, 0])
    assert status == _lib.KV_STATUS_LENGTH and (out == 7).all() and not blocks.any()


def test_rope_append_bad_pages_and_table_ends():
    """A page out of range, or a token beyond the table, leaves keys and values out; the queries turn all the same."""
    d, f = 128, _freqs(128)
    q = torch.randn(4, 3, d, generator=torch.Generator().manual_seed(5)).bfloat16().to(DEV)
    k = q[:, :1].contiguous()
    for table, start, bit in (([[9]], [3], _lib.KV_STATUS_PAGE), ([[-1]], [0], _lib.KV_STATUS_PAGE),
                              ([[0]], [64], _lib.KV_STATUS_LENGTH)):
        blocks, codes = torch.zeros(2, 1, 2, 64 * d, dtype=torch.uint8, device=DEV), torch.zeros(2, 1, 2, dtype=torch.uint8, device=DEV)
        status = i32([0])
        out, _, _ = M.rope_kv_append_x8(blocks, codes, q, k, k, i32(table), i32(start), f, cu_q=i32([0, 4]), status=status)
        torch.cuda.synchronize()
        assert status.item() == bit and not blocks.any()
        assert torch.equal(out, M.rope(q, i32([start[0] + i for i in range(4)]), f))


# ---------------------------------------------------------------- products with 4-bit weights
def _weights(n, k, g, low=105, high=135):
    w = torch.randint(0, 256, (n, k // 2), generator=g).to(torch.uint8)
    return w.to(DEV), torch.randint(low, high, (n, k // 32), generator=g).to(torch.uint8).to(DEV)


def _rows(m, k, form, g, pad=0):
    """x, its codes, the values, and the largest of each value's group (bf16 rows)."""
    amp = torch.exp2(torch.randint(-12, 13, (m, k // 32), generator=g).float()).repeat_interleave(32, 1)
    x = torch.randn(m, k, generator=g) * amp * torch.exp2(torch.randint(-8, 1, (m, k), generator=g).float())
    x[torch.rand(m, k, generator=g) < 0.05] = 0.0
    if form == "bf16":
        x = torch.cat((x, torch.full((m, pad), float("nan"))), 1).bfloat16().to(DEV)[:, :k]
        v = f64(x)
        top = np.abs(v).reshape(m, -1, 32).max(-1).repeat(32, 1)
        return x, None, v, top
    b = torch.randint(0, 256, (m, k + pad), generator=g).to(torch.uint8)
    b[(b & 0x7F) == 0x7F] = 0x38
    c = torch.randint(100, 150, (m, k // 32), generator=g).to(torch.uint8)
    return b.to(DEV)[:, :k], c.to(DEV), L.mxfp8_rows(b[:, :k].numpy(), c.numpy()), None


def _check_linear(got, v, top, w, wc):
    want, size = L.linear(v, w.cpu().numpy(), wc.cpu().numpy())
    k = v.shape[1]
    slack = (k / 32 * 2.0 ** -23 + 2.0 ** -19) * size
    if top is not None:
        slack = slack + 2.0 ** -21 * L.linear(top, w.cpu().numpy(), wc.cpu().numpy())[1]
    assert (np.abs(f64(got) - want) <= 2.0 ** -8 * np.abs(want) + slack + 2.0 ** -133).all()


SIZES = [(1, 1, 128), (1, 128, 256), (2, 130, 384), (7, 1000, 640), (8, 127, 128), (9, 129, 512), (16, 500, 1152),
         (17, 64, 2048), (31, 300, 384), (33, 257, 256), (48, 640, 1024), (49, 129, 640), (64, 200, 896), (65, 200, 384),
         (80, 300, 256), (96, 129, 1280), (97, 300, 512), (128, 140, 640), (129, 130, 384), (176, 300, 256),
         (192, 129, 768), (193, 257, 384), (400, 300, 256), (1000, 130, 128)]


@pytest.mark.parametrize("form", ["mxfp8", "bf16"])
@pytest.mark.parametrize("m,n,k", SIZES)
def test_linear(m, n, k, form):
    g = torch.Generator().manual_seed(m + 3 * n + k)
    w, wc = _weights(n, k, g)
    x, xc, v, top = _rows(m, k, form, g)
    status = i32([0])
    out = M.linear_x4(x, w, wc, x_codes=xc, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0 and out.shape == (m, n) and out.dtype == torch.bfloat16
    _check_linear(out, v, top, w, wc)
    assert torch.equal(out, M.linear_x4(x, w, wc, x_codes=xc))  # the same from run to run


@pytest.mark.parametrize("form", ["mxfp8", "bf16"])
@pytest.mark.parametrize("m,n,k", [(3, 40000, 256), (40, 27000, 384), (5, 20500, 1408), (100, 21000, 128), (300, 20000, 256),
                                   (20, 25000, 128)])
def test_linear_many_tiles(m, n, k, form):
    """More tiles than the GPU takes at once, K whole and shared within a cluster: single rows and columns checked."""
    g = torch.Generator().manual_seed(m + n)
    w, wc = _weights(n, k, g)
    x, xc, v, top = _rows(m, k, form, g)
    status = i32([0])
    out = M.linear_x4(x, w, wc, x_codes=xc, status=status)
    torch.cuda.synchronize()
    assert status.item() == 0
    pick = torch.cat((torch.arange(0, n, 97), torch.arange(n - 150, n)))
    _check_linear(out[:, pick.to(DEV)], v, top, w[pick.to(DEV)], wc[pick.to(DEV)])


@pytest.mark.parametrize("m", [1, 20, 70, 200])
def test_linear_long_rows(m):
    """The longest rows; sums of 65536 products."""
    g = torch.Generator().manual_seed(m)
    w, wc = _weights(140, 65536, g)
    x, xc, v, top = _rows(m, 65536, "mxfp8", g)
    _check_linear(M.linear_x4(x, w, wc, x_codes=xc), v, None, w, wc)


@pytest.mark.parametrize("m", [5, 40, 130])
def test_linear_single_values(m):
    """Rows with one value: every weight comes out as it is, wherever it lies."""
    n, k = 300, 640
    g = torch.Generator().manual_seed(m)
    w, wc = _weights(n, k, g, 120, 134)
    for at in range(0, k, m):
        x = torch.zeros(m, k, dtype=torch.bfloat16, device=DEV)
        rows = torch.arange(min(m, k - at), device=DEV)
        x[rows, at + rows] = 1.0
        out = f64(M.linear_x4(x, w, wc))
        d = L.linear(np.eye(k)[at:at + len(rows)], w.cpu().numpy(), wc.cpu().numpy())[0]
        assert np.array_equal(out[:len(rows)], d) and not out[len(rows):].any()


@pytest.mark.parametrize("form", ["mxfp8", "bf16"])
def test_linear_strided_rows_and_workspace(form):
    g = torch.Generator().manual_seed(12)
    m, n, k = 21, 333, 384
    w, wc = _weights(n, k, g)
    x, xc, v, top = _rows(m, k, form, g, pad=64)
    want = M.linear_x4(x.contiguous(), w, wc, x_codes=xc)
    _check_linear(want, v, top, w, wc)
    need = M.linear_x4_workspace_bytes(m, k, form == "mxfp8")
    ws = torch.full((need + 32,), 0x55, dtype=torch.uint8, device=DEV)
    room = torch.full((m + 2, n + 5), 7.0, dtype=torch.bfloat16, device=DEV)
    out = M.linear_x4(x, w, wc, x_codes=xc, out=room[1:m + 1, 3:n + 3], workspace=ws[:need] if need else None)
    assert torch.equal(out, want)
    assert (room[0] == 7).all() and (room[m + 1] == 7).all() and (room[:, :3] == 7).all() and (room[:, n + 3:] == 7).all()
    assert (ws[need:] == 0x55).all()


def test_linear_codes_off_16_bytes():
    """Codes that only lie on 4 bytes (the 8 and 16-byte loads are not for them)."""
    g = torch.Generator().manual_seed(13)
    m, n, k = 19, 200, 512
    w, wc = _weights(n, k, g)
    x, xc, v, _ = _rows(m, k, "mxfp8", g)
    a, b = (torch.zeros(t.numel() + 8, dtype=torch.uint8, device=DEV)[4:4 + t.numel()].view(t.shape) for t in (wc, xc))
    a.copy_(wc), b.copy_(xc)
    assert a.data_ptr() % 8 == 4 and torch.equal(M.linear_x4(x, w, a, x_codes=b), M.linear_x4(x, w, wc, x_codes=xc))


@pytest.mark.parametrize("m", [6, 60, 150])
@pytest.mark.parametrize("form", ["mxfp8", "bf16"])
def test_linear_rows_and_columns_apart(m, form):
    """A row that is not finite, or a NaN code, makes its row (a weight's code its column) NaN and touches no other."""
    g = torch.Generator().manual_seed(m)
    n, k = 150, 384
    w, wc = _weights(n, k, g)
    w[:, 50:60] = 0x22  # (columns 100 .. 119: no zeros, a NaN or infinity there reaches every sum)
    x, xc, _, _ = _rows(m, k, form, g)
    want = M.linear_x4(x, w, wc, x_codes=xc)
    x2, wc2 = x.clone(), wc.clone()
    if form == "bf16":
        x2[1, 100], x2[3, 110], x2[4, 119] = float("nan"), float("inf"), -float("inf")
        bad = [1, 3, 4]
    else:
        x2[1, 100], x2[3, 110] = 0x7F, 0xFF
        bad = [1, 3]
    wc2[77, 3] = 255
    out = M.linear_x4(x2, w, wc2, x_codes=xc)
    rows = [i for i in range(m) if i not in bad]
    cols = [i for i in range(n) if i != 77]
    assert torch.isnan(out[bad]).all() and torch.isnan(out[:, 77]).all()
    assert torch.equal(out[rows][:, cols], want[rows][:, cols])


def test_linear_extreme_scales():
    """Scales whose product is in range although each is far out; sums that overflow are infinite; zeros are zero."""
    m, n, k = 4, 5, 128
    w = torch.full((n, k // 2), 0x22, dtype=torch.uint8, device=DEV)  # 1.0
    wc = torch.full((n, k // 32), 1, dtype=torch.uint8, device=DEV)
    x8 = torch.full((m, k), 0x38, dtype=torch.uint8, device=DEV)      # 1.0
    xc = torch.full((m, k // 32), 253, dtype=torch.uint8, device=DEV)
    assert (M.linear_x4(x8, w, wc, x_codes=xc) == k).all()            # 2^-126 * 2^126
    wc[:] = 254
    assert torch.isinf(M.linear_x4(x8, w, wc, x_codes=xc)).all()
    assert not M.linear_x4(torch.zeros_like(x8), w, wc, x_codes=xc).any()
    big = torch.full((m, k), 3e38, dtype=torch.bfloat16, device=DEV)
    wc[:] = 100                                                       # 2^-27
    out = f64(M.linear_x4(big, w, wc))
    assert np.allclose(out, float(big[0, 0]) * k * 2.0 ** -27, rtol=2.0 ** -8)
    small = torch.full((m, k), 2.0 ** -126, dtype=torch.bfloat16, device=DEV)
    wc[:] = 247                                                       # 2^120
    assert (M.linear_x4(small, w, wc) == k * 2.0 ** -6).all()


def test_linear_of_no_rows_or_columns():
    g = torch.Generator().manual_seed(1)
    w, wc = _weights(10, 128, g)
    x = torch.randn(3, 128).bfloat16().to(DEV)
    assert M.linear_x4(x[:0], w, wc).shape == (0, 10)
    assert M.linear_x4(x, w[:0], wc[:0]).shape == (3, 0)


def test_linear_of_a_norms_rows():
    """The rows that add_norm_x8 writes go in as they are."""
    g = torch.Generator().manual_seed(6)
    x, r = (torch.randn(19, 512, generator=g).bfloat16().to(DEV) for _ in range(2))
    nw = torch.ones(512, dtype=torch.bfloat16, device=DEV)
    w, wc = _weights(200, 512, g)
    _, x8, codes, _ = M.add_norm_x8(x, r, nw)
    _check_linear(M.linear_x4(x8, w, wc, x_codes=codes), L.mxfp8_rows(x8.cpu().numpy(), codes.cpu().numpy()), None, w, wc)


def test_linear_captured_and_on_two_streams():
    """Captured calls replay on new rows; calls on two streams with workspaces of their own do not touch each other."""
    g = torch.Generator().manual_seed(8)
    cases = []
    for m, n, k in ((6, 700, 512), (90, 500, 384)):
        w, wc = _weights(n, k, g)
        x, _, v, top = _rows(m, k, "bf16", g)
        ws = torch.empty(M.linear_x4_workspace_bytes(m, k, False), dtype=torch.uint8, device=DEV)
        cases.append((x, w, wc, ws, torch.empty(m, n, dtype=torch.bfloat16, device=DEV)))
    want = [M.linear_x4(x, w, wc).clone() for x, w, wc, _, _ in cases]
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    for _ in range(20):
        for s, (x, w, wc, ws, out) in zip(streams, cases):
            with torch.cuda.stream(s):
                M.linear_x4(x, w, wc, out=out, workspace=ws)
    torch.cuda.synchronize()
    assert all(torch.equal(c[4], v) for c, v in zip(cases, want))
    x, w, wc, ws, out = cases[0]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        M.linear_x4(x, w, wc, out=out)
    for seed in (1, 2):
        x.copy_(torch.randn(x.shape, generator=torch.Generator().manual_seed(seed)))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, M.linear_x4(x, w, wc))


# ---------------------------------------------------------------- bindings on a GPU
def test_bindings_refuse_wrong_tensors():
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device=DEV)
    w, h = x[0].clone(), torch.zeros(4, 256, dtype=torch.float16, device=DEV)
    for args, kw in (((h, x, w, w), {}), ((x, x[:3], w, w), {}), ((x, x, w[:128], w), {}), ((x, x, w, w.float()), {}),
                     ((x, x, w, w), dict(gate=x[:2])), ((x, x, w, w), dict(gate=w[:100])), ((x, x, w, w), dict(gate=x.t())),
                     ((x, x, w.cpu(), w), {}), ((x, x, w, w), dict(normed=x[:2]))):
        with pytest.raises(ValueError):
            M.norm_add_norm_x8(*args, **kw)
    q, pos, f = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device=DEV), i32([0, 1, 2, 3]), _freqs(64)
    for args in ((h, pos, f), (q, pos[:3], f), (q, pos.long(), f), (q, pos, f.float()), (q, pos, f.cpu()), (q.cpu(), pos, f),
                 (q.transpose(0, 1), pos, f)):
        with pytest.raises(ValueError):
            M.rope(*args)
    with pytest.raises(_lib.MoeError):
        M.rope(q, pos, f, first=8)
    w4, wc = torch.zeros(10, 128, dtype=torch.uint8, device=DEV), torch.zeros(10, 8, dtype=torch.uint8, device=DEV)
    x8, xc = torch.zeros(4, 256, dtype=torch.uint8, device=DEV), torch.zeros(4, 8, dtype=torch.uint8, device=DEV)
    for args, kw in (((h, w4, wc), {}), ((x, w4[:, :64], wc), {}), ((x, w4, wc[:9]), {}), ((x, w4.cpu(), wc), {}),
                     ((x8, w4, wc), {}), ((x, w4, wc), dict(x_codes=xc)), ((x8, w4, wc), dict(x_codes=xc[:3])),
                     ((x8.t(), w4, wc), dict(x_codes=xc)), ((x, w4, wc), dict(out=x)),
                     ((x, w4, wc), dict(workspace=x.cpu())), ((x, w4, wc), dict(status=pos))):
        with pytest.raises(ValueError):
            M.linear_x4(*args, **kw)
    with pytest.raises(_lib.MoeError):
        M.linear_x4(x, w4, wc, workspace=x8[0, :16])
    with pytest.raises(_lib.MoeError):  # rows of 96 columns
        M.linear_x4(x[:, :96], w4[:, :48].contiguous(), wc[:, :3].contiguous())
