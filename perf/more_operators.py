"""The parts of a decoder layer between its attention and its experts, measured:
the norms behind and before a block with its gate and residual scale, rotary
positions (alone, and in front of the 8-bit paged cache's append), and the
products with 4-bit weights (MXFP4: E2M1 with one E8M0 code per 32 columns of a
row) of a projection.

Each operator is written here in its plain form (elementary torch operations in
32 bits, the angles of positions in 64, rounded once at the end); with ``own``
set, ``run`` calls the framework's kernels instead. Every case is real work of a
layer over hidden size 5120 (40 heads of 128 over 8 key/value heads) or of a
generic one.

Formulas.
  norm    b = x * (mean(x^2) + eps)^(-1/2) * post_w
          res = bf16(res_scale * residual + block_scale * gate * b)
          y = res * (mean(res^2) + eps)^(-1/2) * norm_w, as E4M3 bytes with one
          E8M0 code per 32 columns, and in bf16
  rope    pair i of a head's rotated dims turns by the angle of pos * freqs[i]
          turns, freqs in units of 2^-64 turns; cos and sin times `scale`; pairs
          are (i, i + rot / 2) or (2 i, 2 i + 1) of the dims first .. first + rot
  append  keys turned so and rounded to bf16, then written with the values into
          the cache (a page of 64 tokens: ``blocks`` uint8 [pages, kv_heads, 2,
          64 * D], ``codes`` uint8 [pages, kv_heads, 2]; a byte b under code c
          stands for e4m3(b) * 2^(c - 127)); queries turned into rows of their own.
          In the images 16-byte chunks are permuted within rows:
            keys:   token r, dim d:  r * D + 16 * ((d / 16) ^ s(r)) + d % 16, with
                    s(r) = r % 8 (D = 128, 256) or (r / 2) % 4 (D = 64)
            values: token t, dim d:  d * 64 + 16 * ((t / 16) ^ ((d / 2) % 4)) + w(t % 16),
                    with w(j) = 4 * ((j % 8) / 2) + 2 * (j / 8) + j % 2
  linear  out = x w^T, w uint8 [N, K / 2] (column 2 j in the low nibble of byte j)
          with w_codes uint8 [N, K / 32]; x bf16, or E4M3 bytes with codes like w's
"""

import math

import numpy as np
import torch

own = False

PAGE = 64
FLT_MIN = 1.1754943508222875e-38
GOLDEN = 0.6180339887498949
E2M1 = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0]


# ------------------------------------------------------------------ the cases
def listed():
    return [
        # a decode step's rows behind a block, each channel with its own gate
        {"name": "norm 48x5120", "op": "norm", "rows": 48, "hidden": 5120, "gate": "channel", "normed": True},
        # a long prompt's rows, gated row by row (a conditioned block), 8-bit output only
        {"name": "norm 12000x5120", "op": "norm", "rows": 12000, "hidden": 5120, "gate": "row", "normed": False},
        # the query heads of one token: latency alone
        {"name": "rope 1x40x128", "op": "rope", "tokens": 1, "heads": 40, "dim": 128, "rot": 128, "first": 0,
         "interleaved": False, "far": 100000},
        # a long prompt's query heads, the last dims of each turned, neighbours paired
        {"name": "rope 8000x40x128 part", "op": "rope", "tokens": 8000, "heads": 40, "dim": 128, "rot": 64,
         "first": 64, "interleaved": True, "far": 1000000},
        # a decode step of 48 sequences: one new token each
        {"name": "append 48x1", "op": "append", "seqs": 48, "new_min": 1, "new_max": 1, "had_min": 0,
         "had_max": 4000, "heads": 40, "kv_heads": 8, "dim": 128, "rot": 128, "first": 0, "interleaved": False,
         "far": 0},
        # drafted tokens at positions of their own, far into a document whose start left the cache
        {"name": "append 6x8 far", "op": "append", "seqs": 6, "new_min": 5, "new_max": 8, "had_min": 100,
         "had_max": 4000, "heads": 40, "kv_heads": 8, "dim": 128, "rot": 128, "first": 0, "interleaved": False,
         "far": 500000},
        # prompts written in one call, starting inside pages
        {"name": "append 2x4100", "op": "append", "seqs": 2, "new_min": 3900, "new_max": 4300, "had_min": 30,
         "had_max": 90, "heads": 40, "kv_heads": 8, "dim": 128, "rot": 128, "first": 0, "interleaved": False,
         "far": 0},
        # one token's q, k and v: latency and the weights' stream
        {"name": "linear 1 5120->7168", "op": "linear", "rows": 1, "cols": 5120, "out": 7168, "form": "mxfp8"},
        # the widest decode step behind the attention, rows in bf16
        {"name": "linear 48 5120->5120 bf16", "op": "linear", "rows": 48, "cols": 5120, "out": 5120, "form": "bf16"},
        # a few sequences' rows onto a vocabulary of an odd size
        {"name": "linear 7 5120->129281", "op": "linear", "rows": 7, "cols": 5120, "out": 129281, "form": "bf16"},
        # a short prompt through a block of 2048 columns, nothing a multiple of a tile
        {"name": "linear 333 2048->5011 bf16", "op": "linear", "rows": 333, "cols": 2048, "out": 5011,
         "form": "bf16"},
        # a long prompt's q, k and v
        {"name": "linear 4000 5120->7168", "op": "linear", "rows": 4000, "cols": 5120, "out": 7168, "form": "mxfp8"},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "rope", "append", "linear", "linear"])
    if op == "norm":
        return {"op": op, "rows": _log(rng, 1, 9000), "hidden": 32 * _log(rng, 8, 200),
                "gate": rng.choice(["none", "channel", "row"]), "normed": rng.random() < 0.5}
    if op == "linear":
        cols = 128 * _log(rng, 2, 64)
        out = _log(rng, 60, min(150000, (600 << 20) // cols))
        rows = _log(rng, 1, max(1, min(5000, int(1.4e11) // (cols * out))))
        return {"op": op, "rows": rows, "cols": cols, "out": out, "form": rng.choice(["mxfp8", "bf16"])}
    dim = rng.choice([64, 128, 128, 256])
    rot = rng.choice([dim, dim, dim // 2, dim // 4])
    case = {"op": op, "dim": dim, "rot": rot, "first": rng.choice([0, dim - rot]),
            "interleaved": rng.random() < 0.5, "far": rng.choice([0, 1]) * _log(rng, 10000, 4000000)}
    if op == "rope":
        heads = rng.choice([1, 5, 8, 32, 40, 64])
        return {**case, "tokens": _log(rng, 1, max(2, (32 << 20) // (heads * dim))), "heads": heads}
    kvh = rng.choice([1, 2, 4, 8, 8])
    seqs = _log(rng, 1, 48)
    new = _log(rng, 1, max(2, 8000 // seqs))
    had = _log(rng, 1, 3000)
    return {**case, "seqs": seqs, "new_min": rng.randint(0, new), "new_max": new, "had_min": rng.randint(0, had),
            "had_max": had, "heads": kvh * rng.choice([1, 2, 4, 5]), "kv_heads": kvh}


def _spread(lo, hi, n, at):
    """n whole numbers over [lo, hi], spread by the golden ratio's multiples."""
    return [lo + int((hi - lo + 1) * ((at + i * GOLDEN) % 1.0)) for i in range(n)]


def work(case):
    if case["op"] == "norm":
        r, h = case["rows"], case["hidden"]
        out = 2 + 1 + 1 / 32 + (2 if case["normed"] else 0)
        gate = {"none": 0, "channel": 2 * h, "row": 2 * r * h}[case["gate"]]
        return {"bytes": int(r * h * (4 + out) + 4 * h + gate), "flops": r * h * 14}
    if case["op"] == "rope":
        n, rot = case["tokens"] * case["heads"], case["rot"]
        return {"bytes": n * case["dim"] * 4 + 4 * case["tokens"], "flops": n * rot * 3 + case["tokens"] * rot * 20}
    if case["op"] == "append":
        t = sum(_spread(case["new_min"], case["new_max"], case["seqs"], 0.5))
        d = case["dim"]
        turned = t * (case["heads"] + case["kv_heads"]) * case["rot"]
        return {"bytes": t * d * (case["heads"] * 4 + case["kv_heads"] * 2 * 3),
                "flops": turned * 3 + t * case["kv_heads"] * d * 6 + t * case["rot"] * 20}
    m, k, n = case["rows"], case["cols"], case["out"]
    x = m * k * 2 if case["form"] == "bf16" else m * k + m * k // 32
    return {"bytes": n * k // 2 + n * k // 32 + x + 2 * m * n, "flops": 2 * m * n * k}


# ------------------------------------------------------------------ the cache's layout, codes and bytes
def _key_index(d, device):
    """Byte of (token, dim) in a page's key image, flat over [64, d]."""
    r = torch.arange(PAGE, device=device)[:, None]
    c = torch.arange(d, device=device)[None, :]
    s = r % 8 if d >= 128 else (r // 2) % 4
    return (r * d + 16 * ((c // 16) ^ s) + c % 16).reshape(-1)


def _value_index(d, device):
    """Byte of (token, dim) in a page's value image, flat over [64, d]."""
    t = torch.arange(PAGE, device=device)[:, None]
    c = torch.arange(d, device=device)[None, :]
    j = t % 16
    w = 4 * ((j % 8) // 2) + 2 * (j // 8) + j % 2
    return (c * PAGE + 16 * ((t // 16) ^ ((c // 2) % 4)) + w).reshape(-1)


def _code_of(amax):
    """clamp(ceil(log2(amax / 448)) + 127, 0, 254), amax floored at the smallest normal."""
    m, e = torch.frexp(amax.clamp(min=FLT_MIN) / 448.0)
    return (torch.where(m == 0.5, e - 1, e) + 127).clamp(0, 254)


def _pow2(e):
    """2^e in fp32 for whole e in [-126, 127], exact; smaller ones by two factors."""
    a = e.clamp(-126, 127)
    f = ((a + 127).to(torch.int32) << 23).view(torch.float32)
    return f * (((e - a).clamp(min=-126) + 127).to(torch.int32) << 23).view(torch.float32)


def _e4m3(v):
    """fp32 -> E4M3 bytes, clamped to +-448 and rounded to nearest even."""
    return v.clamp(-448.0, 448.0).to(torch.float8_e4m3fn).view(torch.uint8)


def _mxfp8(y):
    """Rows' E4M3 bytes and their codes, one per 32 columns."""
    groups = y.view(y.shape[0], -1, 32)
    code = _code_of(groups.abs().amax(-1))
    return _e4m3(groups * _pow2(127 - code)[..., None]).view(y.shape), code.to(torch.uint8)


# ------------------------------------------------------------------ inputs
def prepare(case, seed):
    g = torch.Generator(device="cuda").manual_seed(1000 * seed + 29)

    def randn(*shape):
        return torch.randn(*shape, generator=g, device="cuda")

    if case["op"] == "norm":
        r, h = case["rows"], case["hidden"]
        # a residual stream grows over the layers and has a few strong columns
        strong = 1.0 + 8.0 * (torch.rand(h, generator=g, device="cuda") < 0.01)
        gate = {"none": None, "channel": (0.3 + 0.1 * randn(h)).bfloat16(),
                "row": (0.5 * randn(r, h)).bfloat16() if case["gate"] == "row" else None}[case["gate"]]
        return {"case": case, "x": randn(r, h).bfloat16(), "residual": (3.0 * randn(r, h) * strong).bfloat16(),
                "post_w": (1.0 + 0.1 * randn(h)).bfloat16(), "norm_w": (1.0 + 0.1 * randn(h)).bfloat16(),
                "gate": gate, "res_scale": 0.875, "block_scale": 1.25, "eps": 1e-6}
    if case["op"] == "linear":
        return _prepare_linear(case, g, randn)

    d, rot = case["dim"], case["rot"]
    # pos * base^(-2 i / rot) radians, in units of 2^-64 turns
    turns = [10000.0 ** (-2.0 * i / rot) / (2.0 * math.pi) for i in range(rot // 2)]
    freqs = torch.tensor([int(math.ldexp(t, 64)) for t in turns], dtype=torch.int64, device="cuda")
    state = {"case": case, "freqs": freqs, "scale": 1.0 if case["far"] == 0 else 1.15}
    if case["op"] == "rope":
        t = case["tokens"]
        # rows of one projection's output, keys and values behind the query heads
        rows = randn(t, case["heads"] + 2, d).bfloat16()
        state.update(x=rows[:, :case["heads"]],
                     positions=(case["far"] + torch.arange(t, device="cuda")).to(torch.int32))
        return state

    seqs, heads, kvh = case["seqs"], case["heads"], case["kv_heads"]
    new = _spread(case["new_min"], case["new_max"], seqs, 0.5)
    had = _spread(case["had_min"], case["had_max"], seqs, 0.35)
    need = [-(-(a + b) // PAGE) for a, b in zip(had, new)]
    pages = sum(need) + 3
    order = torch.randperm(pages, generator=g, device="cuda").to(torch.int32).cpu()
    table = torch.zeros(seqs, max(max(need), 1), dtype=torch.int32)
    have = torch.zeros(pages, dtype=torch.int64)
    at = 0
    for b, n in enumerate(need):  # a sequence's pages lie anywhere in the pool
        table[b, :n] = order[at:at + n]
        have[table[b, :n].long()] = (had[b] - PAGE * torch.arange(n)).clamp(0, PAGE)
        at += n
    have = have.cuda()
    # keys and values of different strength from head to head; every byte of
    # the pool starts as NaN, so what was never written is never a number
    blocks = torch.full((pages, kvh, 2, PAGE * d), 0x7F, dtype=torch.uint8, device="cuda")
    codes = torch.zeros(pages, kvh, 2, dtype=torch.uint8, device="cuda")
    loud = torch.exp(0.7 * randn(1, kvh, 1, 1))
    token = torch.arange(PAGE, device="cuda")
    for kv, index in ((0, _key_index(d, "cuda")), (1, _value_index(d, "cuda"))):
        t = randn(pages, kvh, PAGE, d) * loud
        written = (token < have[:, None])[:, None, :, None]
        code = _code_of(torch.where(written, t, 0.0).abs().amax((2, 3)))
        b8 = _e4m3(t * _pow2(127 - code)[:, :, None, None])
        b8 = torch.where(written, b8, torch.full_like(b8, 0x7F)).reshape(pages, kvh, -1)
        blocks[:, :, kv].index_copy_(2, index, b8)
        codes[:, :, kv] = code.to(torch.uint8)
    rows = sum(new)
    qkv = randn(rows, heads + 2 * kvh, d)
    qkv[:, heads:] *= torch.cat((loud, loud), 1).view(1, 2 * kvh, 1)
    qkv = qkv.bfloat16()
    starts = torch.tensor([0] + new).cumsum(0).to(torch.int32)
    positions = None
    if case["far"]:
        positions = torch.cat([case["far"] + 1000 * b + torch.arange(n) for b, n in enumerate(new)]).to(torch.int32).cuda()
    state.update(blocks=blocks, codes=codes, table=table.cuda(), q=qkv[:, :heads], k=qkv[:, heads:heads + kvh],
                 v=qkv[:, heads + kvh:], start=torch.tensor(had, dtype=torch.int32).cuda(),
                 cu_q=None if all(n == 1 for n in new) else starts.cuda(), positions=positions)
    return state


def _prepare_linear(case, g, randn):
    m, k, n = case["rows"], case["cols"], case["out"]
    w = torch.empty(n, k // 2, dtype=torch.uint8, device="cuda")
    codes = torch.empty(n, k // 32, dtype=torch.uint8, device="cuda")
    border = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    step = max(1, (64 << 20) // k)
    for lo in range(0, n, step):
        # a layer's weights, rows of different strength
        t = randn(min(step, n - lo), k) * torch.exp(0.3 * randn(min(step, n - lo), 1)) * k ** -0.5
        groups = t.view(t.shape[0], -1, 32)
        _, e = torch.frexp(groups.abs().amax(-1) / 6.0)
        groups = groups * _pow2(-e)[..., None]
        nibble = torch.bucketize(groups.abs(), border).to(torch.uint8) | ((groups < 0).to(torch.uint8) << 3)
        nibble = nibble.view(t.shape[0], k // 2, 2)
        w[lo:lo + t.shape[0]] = nibble[..., 0] | (nibble[..., 1] << 4)
        codes[lo:lo + t.shape[0]] = (e + 127).to(torch.uint8)
    # rows behind a norm: a few strong columns
    strong = 1.0 + 6.0 * (torch.rand(k, generator=g, device="cuda") < 0.01)
    x = randn(m, k) * strong
    state = {"case": case, "w": w, "w_codes": codes, "x": x.bfloat16(), "x_codes": None}
    if case["form"] == "mxfp8":
        state["x"], state["x_codes"] = _mxfp8(x)
    return state


# ------------------------------------------------------------------ one pass
def run(state):
    case = state["case"]
    if own:
        import mxfp8_moe_decode_gb300 as M

        if case["op"] == "norm":
            normed = torch.empty_like(state["x"]) if case["normed"] else None
            res, x8, codes, normed = M.norm_add_norm_x8(
                state["x"], state["residual"], state["post_w"], state["norm_w"], gate=state["gate"],
                res_scale=state["res_scale"], block_scale=state["block_scale"], eps=state["eps"], normed=normed)
            return _norm_out(res, x8, codes, normed)
        if case["op"] == "rope":
            return M.rope(state["x"], state["positions"], state["freqs"], first=case["first"],
                          interleaved=case["interleaved"], scale=state["scale"])
        if case["op"] == "append":
            q, blocks, codes = M.rope_kv_append_x8(
                state["blocks"], state["codes"], state["q"], state["k"], state["v"], state["table"], state["start"],
                state["freqs"], cu_q=state["cu_q"], positions=state["positions"], first=case["first"],
                interleaved=case["interleaved"], scale=state["scale"])
            return _append_out(q, blocks, codes)
        return M.linear_x4(state["x"], state["w"], state["w_codes"], x_codes=state["x_codes"])
    if case["op"] == "norm":
        return _norm_plain(state)
    if case["op"] == "rope":
        return _turn(state["x"], state["positions"], state)
    if case["op"] == "append":
        return _append_plain(state)
    return _linear_plain(state)


def _norm_out(res, x8, codes, normed):
    out = {"res": res, "x8": x8.view(torch.float8_e4m3fn), "codes": codes.view(torch.float8_e8m0fnu)}
    return out if normed is None else {**out, "normed": normed}


def _norm_plain(s):
    x = s["x"].float()
    b = x * torch.rsqrt((x * x).mean(-1, keepdim=True) + s["eps"]) * s["post_w"].float()
    if s["gate"] is not None:
        b = b * s["gate"].float()
    res = (s["res_scale"] * s["residual"].float() + s["block_scale"] * b).bfloat16()
    f = res.float()
    y = f * torch.rsqrt((f * f).mean(-1, keepdim=True) + s["eps"]) * s["norm_w"].float()
    x8, code = _mxfp8(y)
    return _norm_out(res, x8, code, y.bfloat16() if s["case"]["normed"] else None)


def _turn(x, positions, s):
    """x [tokens, heads, d] turned by its positions, in bf16."""
    case = s["case"]
    first, rot = case["first"], case["rot"]
    turns = (positions.long()[:, None] * s["freqs"]).double() * 2.0 ** -64  # (whole turns fall away)
    angle = (turns * (2.0 * math.pi))[:, None, :]
    cos, sin = (torch.cos(angle) * s["scale"]).float(), (torch.sin(angle) * s["scale"]).float()
    part = x[..., first:first + rot].float()
    if case["interleaved"]:
        a, b = part[..., 0::2], part[..., 1::2]
        part = torch.stack((a * cos - b * sin, b * cos + a * sin), -1).flatten(-2)
    else:
        a, b = part[..., :rot // 2], part[..., rot // 2:]
        part = torch.cat((a * cos - b * sin, b * cos + a * sin), -1)
    return torch.cat((x[..., :first], part.bfloat16(), x[..., first + rot:]), -1)


def _append_out(q, blocks, codes):
    return {"q": q, "blocks": blocks.view(torch.float8_e4m3fn), "codes": codes.view(torch.float8_e8m0fnu)}


def _rows_of(s, rows):
    """Each row's sequence and its place among the sequence's new rows."""
    t = torch.arange(rows, device="cuda")
    if s["cu_q"] is None:
        return t, torch.zeros_like(t)
    b = torch.searchsorted(s["cu_q"].long(), t, right=True) - 1
    return b, t - s["cu_q"].long()[b]


def _append_plain(s):
    blocks, codes, table = s["blocks"], s["codes"], s["table"]
    rows, kvh, d = s["k"].shape
    b, i = _rows_of(s, rows)
    at = s["start"].long()[b] + i
    positions = at if s["positions"] is None else s["positions"]
    q, k = _turn(s["q"], positions, s), _turn(s["k"], positions, s)
    page, slot = table[b, at // PAGE].long(), at % PAGE
    pages = blocks.shape[0]
    first = torch.full((pages,), PAGE, device="cuda").scatter_reduce(0, page, slot, "amin")
    touched = (first < PAGE).nonzero()[:, 0]
    place = torch.full((pages,), -1, device="cuda")
    place[touched] = torch.arange(touched.shape[0], device="cuda")
    old = (torch.arange(PAGE, device="cuda") < first[touched, None])[:, None, :]  # tokens that stay
    _write(blocks, codes, 0, k, _key_index(d, "cuda"), page, slot, touched, place, first, old)
    _write(blocks, codes, 1, s["v"], _value_index(d, "cuda"), page, slot, touched, place, first, old)
    return _append_out(q, blocks, codes)


def _write(blocks, codes, kv, x, index, page, slot, touched, place, first, old):
    """The new rows x into the keys (kv = 0) or values (1) of the touched pages."""
    rows, kvh, d = x.shape
    x = x.float()
    amax = torch.zeros(blocks.shape[0], kvh, device="cuda")
    amax.scatter_reduce_(0, page[:, None].expand(rows, kvh), x.abs().amax(-1), "amax")
    had = torch.where(first[touched, None] > 0, codes[touched, :, kv].long(), 0)
    code = torch.maximum(_code_of(amax[touched]), had)
    # the tokens that stay, under the new code
    image = blocks[touched, :, kv][:, :, index].view(-1, kvh, PAGE, d)
    again = _e4m3(image.view(torch.float8_e4m3fn).float() * _pow2(had - code)[:, :, None, None])
    image = torch.where(old[..., None] & (code > had)[:, :, None, None], again, image)
    # the new ones
    image[place[page], :, slot] = _e4m3(x * _pow2(127 - code[place[page]])[..., None])
    whole = torch.empty_like(image).view(-1, kvh, PAGE * d)
    whole[:, :, index] = image.view(-1, kvh, PAGE * d)
    blocks[touched, :, kv] = whole
    codes[touched, :, kv] = code.to(torch.uint8)


def _linear_plain(s):
    w, codes, x = s["w"], s["w_codes"], s["x"]
    n, k = w.shape[0], 2 * w.shape[1]
    table = torch.tensor(E2M1, device="cuda")
    byte = torch.arange(256, device="cuda")
    pairs = torch.stack((table[byte & 15], table[byte >> 4]), -1)
    weight = pairs[w.int()].view(n, -1, 32) * _pow2(codes.int() - 127)[..., None]
    x = x.float() if s["x_codes"] is None else (
        x.view(torch.float8_e4m3fn).float().view(x.shape[0], -1, 32) * _pow2(s["x_codes"].int() - 127)[..., None]).view(-1, k)
    return (x @ weight.view(n, k).T).bfloat16()


# ------------------------------------------------------------------ the definitions in 64 bits
def _two(e):
    """2^e in 64 bits, exactly, for whole e."""
    return ((e.to(torch.int64) + 1023) << 52).view(torch.float64)


def _round_bits(a, bits, least):
    """The nearest values of that many significant bits (down to `least`'s step), ties to the even one."""
    step = _two(torch.frexp(a.abs().clamp(min=least))[1] - bits)
    return torch.round(a / step) * step


def _round_e4m3(v):
    return _round_bits(v, 4, 2.0 ** -6).clamp(-448.0, 448.0)


def _exact_exponent(amax):
    """The whole e with 448 * 2^(e - 1) < amax <= 448 * 2^e, from -127 up."""
    e = torch.ceil(torch.log2(amax.clamp(min=1e-300) / 448.0))
    e = torch.where(448.0 * _two(e) < amax, e + 1, torch.where(448.0 * _two(e - 1) >= amax, e - 1, e))
    return e.clamp(min=-127.0)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "norm":
        return _exact_norm(s, case)
    if case["op"] == "rope":
        return _exact_rope(s["x"], s["positions"].tolist(), s, case)
    return _exact_append(s, case) if case["op"] == "append" else _exact_linear(s, case)


def _exact_norm(s, case):
    parts = []
    for lo in range(0, case["rows"], 1024):
        hi = lo + 1024
        x = s["x"][lo:hi].double()
        block = x * s["post_w"].double() / torch.sqrt(torch.sum(x ** 2, 1, keepdim=True) / case["hidden"] + s["eps"])
        if case["gate"] == "channel":
            block = block * s["gate"].double()[None, :]
        elif case["gate"] == "row":
            block = block * s["gate"][lo:hi].double()
        res = _round_bits(s["res_scale"] * s["residual"][lo:hi].double() + s["block_scale"] * block, 8, 2.0 ** -126)
        y = res * s["norm_w"].double() / torch.sqrt(torch.sum(res ** 2, 1, keepdim=True) / case["hidden"] + s["eps"])
        groups = y.reshape(-1, 32)
        e = _exact_exponent(groups.abs().amax(1, keepdim=True))
        parts.append((res, _round_e4m3(groups * _two(-e)).view(y.shape), _two(e).view(y.shape[0], -1), y))
    res, x8, codes, y = (torch.cat(p) for p in zip(*parts))
    out = {"res": res, "x8": x8, "codes": codes}
    return {**out, "normed": y} if case["normed"] else out


def _exact_rope(x, positions, s, case):
    """The turned rows in 64 bits, unrounded: the angles from whole numbers (modulo 2^64)."""
    rot, first = case["rot"], case["first"]
    whole = np.array(positions, dtype=np.uint64)[:, None] * s["freqs"].cpu().numpy().astype(np.uint64)
    a = torch.from_numpy(whole.astype(np.float64) / 2.0 ** 64 * (2.0 * np.pi)).cuda()
    pair = torch.polar(torch.full_like(a, s["scale"]), a)[:, None, :]
    out = x.double().clone()
    i = torch.arange(rot // 2, device="cuda")
    one, two = (first + 2 * i, first + 2 * i + 1) if case["interleaved"] else (first + i, first + rot // 2 + i)
    z = torch.complex(out[:, :, one], out[:, :, two]) * pair
    out[:, :, one], out[:, :, two] = z.real, z.imag
    return out


def _exact_append(s, case):
    value_of = [(-1.0 if v & 128 else 1.0) * ((v & 7) * 2.0 ** -9 if (v >> 3) & 15 == 0 else (8 + (v & 7)) * 2.0 ** (((v >> 3) & 15) - 10))
                if v & 127 != 127 else math.nan for v in range(256)]
    value = torch.tensor(value_of, dtype=torch.float64, device="cuda")[s["blocks"].long()]
    scale = _two(s["codes"].long() - 127)
    kvh, d = s["k"].shape[1:]
    had, pages = s["start"].tolist(), s["table"].tolist()
    cu = list(range(s["k"].shape[0] + 1)) if s["cu_q"] is None else s["cu_q"].tolist()
    at = [had[b] + r - cu[b] for b in range(len(had)) for r in range(cu[b], cu[b + 1])]
    positions = at if s["positions"] is None else s["positions"].tolist()
    q = _exact_rope(s["q"], positions, s, case)
    k = _exact_rope(s["k"], positions, s, case)
    k[:, :, case["first"]:case["first"] + case["rot"]] = _round_bits(
        k[:, :, case["first"]:case["first"] + case["rot"]], 8, 2.0 ** -126)
    # where a token's d bytes lie, found by walking the layout's words
    r = np.arange(PAGE)[:, None]
    c = np.arange(d)[None, :]
    turn = r % 8 if d >= 128 else r // 2 % 4
    in_word = np.array([0, 1, 4, 5, 8, 9, 12, 13, 2, 3, 6, 7, 10, 11, 14, 15])
    where = (r * d + (c // 16 ^ turn) * 16 + c % 16, c * PAGE + (r // 16 ^ c // 2 % 4) * 16 + in_word[r % 16])
    where = [torch.from_numpy(w).cuda() for w in where]
    for b in range(len(had)):
        for lo in range(had[b] // PAGE * PAGE, had[b] + cu[b + 1] - cu[b], PAGE):
            t0, t1 = max(lo, had[b]), min(lo + PAGE, had[b] + cu[b + 1] - cu[b])
            if t1 <= t0:
                continue
            page = pages[b][lo // PAGE]
            for kv, x in ((0, k), (1, s["v"])):
                x = x[cu[b] + t0 - had[b]:cu[b] + t1 - had[b]].double().transpose(0, 1)
                e = _exact_exponent(x.abs().amax((1, 2)))
                if t0 > lo:
                    before = (torch.frexp(scale[page, :, kv])[1] - 1).double()
                    e = torch.maximum(e, before)
                    stay = where[kv][:t0 - lo].reshape(-1)
                    old = value[page, :, kv][:, stay]
                    moved = _round_e4m3(old * _two(before - e)[:, None])
                    value[page, :, kv][:, stay] = torch.where((e > before)[:, None], moved, old)
                scale[page, :, kv] = _two(e)
                new = where[kv][t0 - lo:t1 - lo].reshape(-1)
                value[page, :, kv][:, new] = _round_e4m3(x * _two(-e)[:, None, None]).reshape(kvh, -1)
    return {"q": q, "blocks": value, "codes": scale}


def _exact_linear(s, case):
    k, n = case["cols"], case["out"]
    x = s["x"].double()
    if case["form"] == "mxfp8":
        x = s["x"].view(torch.float8_e4m3fn).double() * _two(s["x_codes"].long() - 127).repeat_interleave(32, 1)
    parts = []
    step = max(1, (64 << 20) // k)
    for lo in range(0, n, step):
        b, e = s["w"][lo:lo + step].long(), s["w_codes"][lo:lo + step].long() - 127
        v = torch.empty(b.shape[0], k, dtype=torch.float64, device="cuda")
        for at, nibble in ((0, b % 16), (1, b // 16)):
            p, m = nibble % 8 // 2, nibble % 2  # exponent and mantissa bits
            size = torch.where(p == 0, 0.5 * m.double(), (1.0 + 0.5 * m.double()) * _two(p - 1))
            v[:, at::2] = torch.where(nibble >= 8, -size, size)
        v *= _two(e).repeat_interleave(32, 1)
        parts.append(x @ v.T)
    return torch.cat(parts, 1)
