"""Cases of the microscaled 4-bit linear and of attention over an 8-bit cache.

Four operators of a decoder that is served in low precision:

``fp4_quantize``   4-bit floating-point (e2m1) codes of a bf16 matrix with a
                   scale for each block of input channels ("mx": 32 channels
                   and a power of two, "nv": 16 channels, an e4m3 scale and a
                   power of two for each row), and the values they stand for.
``fp4_linear``     y = x . w^T of a bf16 activation, quantized in the call,
                   against a weight held in such codes.
``kv8_append``     new keys and values into a paged cache of 8-bit codes
                   (int8 or e4m3) with one scale for each page and head.
``kv8_attention``  causal attention of each sequence's newest tokens over
                   that cache, from one token a sequence to whole prompts.

``run`` computes them from elementary torch operations, or, where ``own`` is
true, through this repository's package.
"""
import math

import torch

own = False

DEV = "cuda"

# Quotients whose rounding decides a code divide by a tensor: a division by a
# Python number may be computed as a product with its rounded reciprocal.
FP4_BLOCK = {"mx": 32, "nv": 16}
KV_QMAX = {"int8": 127.0, "e4m3": 448.0}


# ------------------------------------------------------------------ cases ----

def listed():
    return [
        # one token's hidden state entering an MLP: latency only
        dict(name="quantize-nv-1x2048", op="quantize", fmt="nv", rows=1, k=2048),
        # a 27B-scale up projection, quantized when the weights are loaded
        dict(name="quantize-mx-17408x5120", op="quantize", fmt="mx", rows=17408, k=5120),
        # the q projection of a 1.7B model for one token
        dict(name="linear-mx-m1-2048x2048", op="linear", fmt="mx", m=1, n=2048, k=2048),
        # a 27B-scale up projection for a small odd batch of decoding users
        dict(name="linear-nv-m13-17408x5120", op="linear", fmt="nv", m=13, n=17408, k=5120),
        # a 7B model's up projection over a prompt whose length fits no tile
        dict(name="linear-mx-m1999-11008x4096", op="linear", fmt="mx", m=1999, n=11008, k=4096),
        # a 27B-scale down projection over a large prefill batch
        dict(name="linear-nv-m8192-5120x17408", op="linear", fmt="nv", m=8192, n=5120, k=17408),
        # one new token for each of 64 users
        dict(name="append-e4m3-64x1", op="append", fmt="e4m3", batch=64, new=1, longest=4096,
             q_heads=16, kv_heads=8, d=128, page=64, ragged=False),
        # the prompts of four users, of unequal length, behind a cached prefix
        dict(name="append-e4m3-4x4000", op="append", fmt="e4m3", batch=4, new=4000, longest=6000,
             q_heads=16, kv_heads=8, d=128, page=16, ragged=True),
        # short conversations of a small model: latency only
        dict(name="attention-int8-5x1-300", op="attention", fmt="int8", batch=5, new=1, longest=300,
             q_heads=4, kv_heads=2, d=64, page=16, ragged=False),
        # one user with a long document
        dict(name="attention-int8-1x1-32768", op="attention", fmt="int8", batch=1, new=1,
             longest=32768, q_heads=16, kv_heads=8, d=128, page=64, ragged=False),
        # a full serving batch, lengths spread from an eighth to the longest
        dict(name="attention-e4m3-128x1-4096", op="attention", fmt="e4m3", batch=128, new=1,
             longest=4096, q_heads=32, kv_heads=4, d=128, page=32, ragged=False),
        # two prompts' next chunks over what is cached of them
        dict(name="attention-int8-2x2048-8192", op="attention", fmt="int8", batch=2, new=2048,
             longest=8192, q_heads=16, kv_heads=8, d=128, page=64, ragged=True),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


_HEADS = ((16, 8, 128), (32, 32, 128), (32, 4, 128), (4, 2, 64))


def draw(rng):
    op = rng.choice(("quantize", "linear", "append", "attention", "linear", "attention"))
    if op in ("quantize", "linear"):
        fmt = rng.choice(("mx", "nv"))
        k = 128 * _log(rng, 1, 136)
        if op == "quantize":
            return dict(op=op, fmt=fmt, rows=_log(rng, 1, min(17408, 89_000_000 // k)), k=k)
        n = _log(rng, 64, 17408)
        m = _log(rng, 1, max(1, min(8192, 730_000_000_000 // (n * k))))
        return dict(op=op, fmt=fmt, m=m, n=n, k=k)
    q_heads, kv_heads, d = rng.choice(_HEADS)
    page = rng.choice((16, 32, 64, 128))
    fmt = "e4m3" if op == "append" else rng.choice(("int8", "e4m3"))
    if op == "append" or rng.random() < 0.6:
        # one token each, or appending: the cache's size is the cost
        longest = _log(rng, 1, 32768)
        most = 120_000_000 // (longest * kv_heads * d)
        batch = _log(rng, 1, max(1, min(128, most)))
        new = 1 if op == "attention" else _log(rng, 1, max(1, min(longest, 16000 // batch)))
    else:
        new = _log(rng, 2, 4096)
        longest = new + _log(rng, 1, 8192)
        if new * longest * q_heads * d // 128 > 540_000_000:
            new, longest = new // 4 + 1, longest // 2 + 1
        most = min(16_000 // new, 540_000_000 // (new * longest * q_heads * d // 128),
                   120_000_000 // (longest * kv_heads * d))
        batch = _log(rng, 1, max(1, min(128, most)))
    return dict(op=op, fmt=fmt, batch=batch, new=min(new, longest), longest=longest,
                q_heads=q_heads, kv_heads=kv_heads, d=d, page=page, ragged=rng.random() < 0.5)


def _counts(case):
    """New tokens and lengths after them of each sequence."""
    news, lens = [], []
    for b in range(case["batch"]):
        f = (b * 0.6180339887) % 1.0
        n = case["new"] if not case["ragged"] or b == 0 else max(1, int(case["new"] * (1 - 0.7 * f)))
        ln = case["longest"] if b == 0 else max(1, int(case["longest"] * (1 - 0.875 * f)))
        news.append(n)
        lens.append(max(n, ln))
    return news, lens


def work(case):
    if case["op"] == "quantize":
        r, k, blk = case["rows"], case["k"], FP4_BLOCK[case["fmt"]]
        held = r * k // 2 + r * k // blk + (4 * r if case["fmt"] == "nv" else 0)
        return {"bytes": 2 * r * k + held + 2 * r * k, "flops": 2 * r * k}
    if case["op"] == "linear":
        m, n, k, blk = case["m"], case["n"], case["k"], FP4_BLOCK[case["fmt"]]
        w = n * k // 2 + n * k // blk + (4 * n if case["fmt"] == "nv" else 0)
        return {"bytes": 2 * m * k + w + 2 * m * n, "flops": 2 * m * n * k}
    news, lens = _counts(case)
    row = case["kv_heads"] * case["d"]
    if case["op"] == "append":
        pages = sum((ln + case["page"] - 1) // case["page"] - (ln - n) // case["page"]
                    for n, ln in zip(news, lens))
        return {"bytes": sum(news) * row * 2 * 3 + 8 * pages * case["kv_heads"],
                "flops": 4 * sum(news) * row}
    pages = sum((ln + case["page"] - 1) // case["page"] for ln in lens)
    q = case["q_heads"] * case["d"]
    pairs = sum(n * ln - n * (n - 1) // 2 for n, ln in zip(news, lens))
    return {"bytes": 2 * sum(lens) * row + 8 * pages * case["kv_heads"] + 4 * sum(news) * q,
            "flops": 4 * pairs * q}


# ----------------------------------------------------------------- inputs ----

def _e2m1(a):
    """Magnitudes rounded to {0, .5, 1, 1.5, 2, 3, 4, 6}, ties to the even code, at most 6."""
    a = a.clamp(max=6.0)
    step = torch.where(a < 2.0, 0.5, torch.where(a < 4.0, 1.0, 2.0)).to(a.dtype)
    return torch.round(a / step) * step


def _fp4_parts(x, fmt):
    """(signed e2m1 values [R, K/b, b], block scales [R, K/b] as float32, row scales [R, 1] or None)."""
    r, k = x.shape
    blk = FP4_BLOCK[fmt]
    v = x.float().view(r, k // blk, blk)
    amax = v.abs().amax(2)
    if fmt == "mx":
        # a block's scale: the power of two two binades under its largest value
        e = torch.frexp(amax).exponent - 3
        e = torch.where(amax > 0, e, -127).clamp(-127, 127)
        s = torch.ldexp(torch.ones_like(amax), e)
        u = torch.ldexp(v.abs(), -e.unsqueeze(2))
        return torch.copysign(_e2m1(u), v), s, None
    # a row's scale: the least power of two that leaves its largest value at most 6 * 448
    m, e = torch.frexp(amax.amax(1, keepdim=True))
    e = torch.where(m <= 0.65625, e - 12, e - 11)
    e = torch.where(m > 0, e, 0).clamp(min=-126)
    s = (torch.ldexp(amax, -e) / torch.full_like(amax, 6.0)).to(torch.float8_e4m3fn).float()
    u = torch.ldexp(v.abs(), -e.unsqueeze(2)) / s.unsqueeze(2)
    q = torch.copysign(_e2m1(u.nan_to_num(0.0, posinf=0.0)), v)
    q = torch.where(s.unsqueeze(2) > 0, q, 0.0)
    return q, s, torch.ldexp(torch.ones_like(m), e)


def _fp4_pack(x, fmt):
    """A weight as it is held: codes uint8 [N, K/2], scale bytes in tiles of 128 rows x 4 blocks, row scales."""
    q, s, row = _fp4_parts(x, fmt)
    n, k = x.shape
    a = q.abs().view(n, k)
    code = torch.where(a < 2.0, a * 2, torch.where(a < 4.0, a + 2, a / 2 + 4)).to(torch.uint8)
    code = code | (torch.signbit(q.view(n, k)).to(torch.uint8) << 3)
    codes = (code[:, 0::2] | (code[:, 1::2] << 4)).contiguous()
    if fmt == "mx":
        sb = (torch.frexp(s).exponent + 126).to(torch.uint8)
    else:
        sb = s.to(torch.float8_e4m3fn).view(torch.uint8)
    tiles = (n + 127) // 128
    full = torch.zeros(tiles * 128, sb.shape[1], dtype=torch.uint8, device=x.device)
    full[:n] = sb
    # byte (row % 32) * 16 + (row % 128) / 32 * 4 + block % 4 of tile [row / 128][block / 4]
    t = full.view(tiles, 4, 32, sb.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).contiguous()
    return codes, t.view(tiles, sb.shape[1] // 4, 512), None if row is None else row.view(n).contiguous()


def _scales_of(tiles, n, fmt):
    """Block scales [N, K/b] of the tiled bytes, as float32."""
    t, c, _ = tiles.shape
    b = tiles.view(t, c, 32, 4, 4).permute(0, 3, 2, 1, 4).reshape(t * 128, c * 4)[:n]
    if fmt == "mx":
        return torch.ldexp(torch.ones(b.shape, device=b.device), b.int() - 127)
    return b.contiguous().view(torch.float8_e4m3fn).float()


def _gen(seed):
    return torch.Generator(device=DEV).manual_seed(int(seed))


def prepare(case, seed):
    g = _gen(seed)
    if case["op"] == "quantize":
        r, k = case["rows"], case["k"]
        if r >= 1024:  # a weight: a hundredth of its input channels are outliers
            x = torch.randn(r, k, generator=g, device=DEV) * 0.02
            x[:, torch.randperm(k, generator=g, device=DEV)[: max(1, k // 100)]] *= 10
        else:  # activations, heavy-tailed over channels
            c = torch.randn(k, generator=g, device=DEV).abs() + 0.1
            x = torch.randn(r, k, generator=g, device=DEV) * c
        return dict(case=case, x=x.to(torch.bfloat16))
    if case["op"] == "linear":
        m, n, k = case["m"], case["n"], case["k"]
        w = (torch.randn(n, k, generator=g, device=DEV) * 0.02).to(torch.bfloat16)
        x = torch.randn(m, k, generator=g, device=DEV).to(torch.bfloat16)
        codes, scales, row = _fp4_pack(w, case["fmt"])
        return dict(case=case, x=x, codes=codes, scales=scales, row=row)
    news, lens = _counts(case)
    hq, h, d, page = case["q_heads"], case["kv_heads"], case["d"], case["page"]
    used = [(ln + page - 1) // page for ln in lens]
    width = max(used)
    total = sum(used)
    order = torch.randperm(total, generator=g, device=DEV).to(torch.int32)
    first = torch.tensor([sum(used[:b]) for b in range(len(used))], device=DEV)
    col = torch.arange(width, device=DEV)
    has = col[None, :] < torch.tensor(used, device=DEV)[:, None]
    table = torch.where(has, order[(first[:, None] + col[None, :]).clamp(max=total - 1)], 0).int()
    t = sum(news)
    # one fused projection's output: q, k and v are slices of its rows
    qkv = torch.randn(t, (hq + 2 * h) * d, generator=g, device=DEV).to(torch.bfloat16)
    starts = [sum(news[:b]) for b in range(len(news) + 1)]
    state = dict(case=case, q=qkv[:, : hq * d].view(t, hq, d),
                 k=qkv[:, hq * d: (hq + h) * d].view(t, h, d),
                 v=qkv[:, (hq + h) * d:].view(t, h, d), table=table.contiguous(),
                 lens=torch.tensor(lens, dtype=torch.int32, device=DEV),
                 starts=torch.tensor(starts, dtype=torch.int32, device=DEV),
                 news=news, longest=max(lens))
    # what the cache holds: a spread of scales, exact in bf16 as appending leaves them
    qmax = KV_QMAX[case["fmt"]]
    for name, shape in (("kc", (total, h, page, d)), ("vc", (total, h, d, page))):
        c = torch.randn(shape, generator=g, device=DEV).mul_(qmax / 4).clamp_(-qmax, qmax)
        state[name] = c.round_().to(torch.int8) if case["fmt"] == "int8" else c.to(torch.float8_e4m3fn)
        s = (3.0 + torch.rand(total, h, generator=g, device=DEV) * 2.0) / qmax
        state[name[0] + "s"] = s.to(torch.bfloat16).float()
    return state


# ------------------------------------------------------------ plain forms ----

def _plain_quantize(s):
    q, sc, row = _fp4_parts(s["x"], s["case"]["fmt"])
    v = q * sc.unsqueeze(2)
    if row is not None:
        v = v * row.unsqueeze(2)
    return v.view(s["x"].shape).to(torch.bfloat16)


def _plain_linear(s):
    fmt = s["case"]["fmt"]
    n, k = s["codes"].shape[0], s["codes"].shape[1] * 2
    q, sc, row = _fp4_parts(s["x"], fmt)
    x = (q * sc.unsqueeze(2)).view(-1, k)
    table = torch.tensor([0, .5, 1, 1.5, 2, 3, 4, 6], device=DEV)
    table = torch.cat((table, -table))
    codes = torch.stack((s["codes"] & 15, s["codes"] >> 4), 2).view(n, -1, FP4_BLOCK[fmt])
    w = (table[codes.int()] * _scales_of(s["scales"], n, fmt).unsqueeze(2)).view(n, k)
    y = x @ w.t()
    if row is not None:
        y = y * row * s["row"]
    return y.to(torch.bfloat16)


def _pages(s):
    """Padded to the longest: positions' pages of every sequence [B, P] and the length of that axis."""
    page = s["case"]["page"]
    p = (s["longest"] + page - 1) // page
    return s["table"][:, :p].long(), p * page


def _round_up_bf16(t):
    """float32 values rounded up to the next that bf16 holds."""
    return ((t.contiguous().view(torch.int32) + 0xFFFF) & -0x10000).view(torch.float32)


def _plain_append(s):
    c = s["case"]
    page, qmax, n = c["page"], KV_QMAX[c["fmt"]], c["new"]
    lens, starts = s["lens"].long(), s["starts"].long()
    count = starts[1:] - starts[:-1]
    old = lens - count
    pages, _ = _pages(s)
    # every page that some new token may fall into, padded: [B, W]
    w = (n + page - 2) // page + 1
    at = (old // page)[:, None] + torch.arange(w, device=DEV)[None, :]
    touched = (at * page < lens[:, None]) & ((at + 1) * page > old[:, None])
    ids = pages.gather(1, at.clamp(max=pages.shape[1] - 1))
    pos = at.unsqueeze(2) * page + torch.arange(page, device=DEV)  # [B, W, page]
    new = (pos >= old[:, None, None]) & (pos < lens[:, None, None])
    was = pos < old[:, None, None]
    row = (starts[:-1, None, None] + pos - old[:, None, None]).clamp(0, s["k"].shape[0] - 1)
    ids = ids[touched]
    new, was, row = new[touched][:, None, :, None], was[touched][:, None, :, None], row[touched]
    _plain_pages(s["kc"], s["ks"], s["k"], False, ids, new, was, row, qmax)
    _plain_pages(s["vc"], s["vs"], s["v"], True, ids, new, was, row, qmax)
    return s["kc"], s["ks"], s["vc"], s["vs"]


def _plain_pages(codes, scales, x, turned, ids, new, was, row, qmax):
    """One side's pages `ids` with the rows `row` of x where `new`, old codes rescaled where `was`."""
    x = torch.where(new, x[row].float().transpose(1, 2), 0.0)  # [touched, H, page, d]
    before = codes.view(torch.uint8)[ids].view(codes.dtype).float()
    before = before.transpose(2, 3) if turned else before
    s0 = torch.where(was.any(2).view(-1, 1), scales[ids], 0.0)
    top = x.abs().amax((2, 3))
    s1 = torch.maximum(s0, _round_up_bf16(top / torch.full_like(top, qmax)))
    b1, b0 = s1[:, :, None, None], s0[:, :, None, None]
    fresh = torch.where(b1 > 0, x / b1, 0.0)
    again = torch.where(b1 > b0, before * b0 / b1, before)
    if codes.dtype == torch.int8:
        fresh, again = fresh.round(), again.round()
    fresh, again = fresh.to(codes.dtype).float(), again.to(codes.dtype).float()
    after = torch.where(new, fresh, torch.where(was, again, before)).to(codes.dtype)
    after = after.transpose(2, 3) if turned else after
    codes.view(torch.uint8)[ids] = after.contiguous().view(torch.uint8)
    scales[ids] = s1


def _plain_attention(s):
    c = s["case"]
    hq, h, d = c["q_heads"], c["kv_heads"], c["d"]
    b, n, grp = c["batch"], c["new"], hq // h
    pages, length = _pages(s)
    lens, starts = s["lens"].long(), s["starts"].long()
    count = starts[1:] - starts[:-1]
    # each sequence's new tokens, padded to the most any has: [B, n]
    i = torch.arange(n, device=DEV)[None, :]
    live = i < count[:, None]
    row = (starts[:-1, None] + i).clamp(max=s["q"].shape[0] - 1)
    q = s["q"][row].float().view(b, n, h, grp, d).permute(0, 2, 3, 1, 4).reshape(b, h, grp * n, d)
    k = s["kc"].view(torch.uint8)[pages].view(s["kc"].dtype).float() * s["ks"][pages][..., None, None]
    k = k.permute(0, 2, 1, 3, 4).reshape(b, h, length, d)
    pos = torch.arange(length, device=DEV)
    limit = (lens - count)[:, None] + i  # the last key that each new token sees
    seen = pos[None, None, :] <= limit[:, :, None]
    score = (q @ k.transpose(2, 3)).mul_(1 / math.sqrt(d)).view(b, h, grp, n, length)
    score.masked_fill_(~seen[:, None, None], float("-inf"))
    del k
    score -= score.amax(4, keepdim=True)
    score.exp_()
    score /= score.sum(4, keepdim=True)
    v = s["vc"].view(torch.uint8)[pages].view(s["vc"].dtype).float() * s["vs"][pages][..., None, None]
    v = v.permute(0, 2, 1, 4, 3).reshape(b, h, length, d)
    v = torch.where((pos[None, :] < lens[:, None])[:, None, :, None], v, 0.0)
    o = score.view(b, h, grp * n, length) @ v
    o = o.view(b, h, grp, n, d).permute(0, 3, 1, 2, 4).reshape(b, n, hq, d)
    return o[live].to(torch.bfloat16)


def run(s):
    c = s["case"]
    if not own:
        return {"quantize": _plain_quantize, "linear": _plain_linear, "append": _plain_append,
                "attention": _plain_attention}[c["op"]](s)
    import weight_only_int4_quantize_b200 as w4
    if c["op"] == "quantize":
        return w4.fp4_quantize(s["x"], c["fmt"], values=True)[3]
    if c["op"] == "linear":
        codes, scales, row = w4.fp4_quantize(s["x"], c["fmt"])
        return w4.fp4_linear(codes, scales, row, s["codes"], s["scales"], s["row"], c["fmt"])
    cache = w4.KV8Cache(s["kc"], s["vc"], s["ks"], s["vs"])
    if c["op"] == "append":
        w4.kv8_append(cache, s["k"], s["v"], s["table"], s["lens"], s["starts"], c["new"])
        return s["kc"], s["ks"], s["vc"], s["vs"]
    return w4.kv8_attention(s["q"], cache, s["table"], s["lens"], s["starts"], c["new"])


# ------------------------------------------------------------ definitions ----

def _nearest(v, grid):
    """The value of `grid` (ascending magnitudes, even codes at even places) next to each |v|, sign kept."""
    a = v.abs().clamp(max=float(grid[-1]))
    hi = torch.searchsorted(grid, a.contiguous()).clamp(max=len(grid) - 1)
    lo = (hi - 1).clamp(min=0)
    up, down = grid[hi] - a, a - grid[lo]
    take = torch.where(up < down, hi, torch.where(down < up, lo, torch.where(hi % 2 == 0, hi, lo)))
    return torch.copysign(grid[take], v)


def _grid(codes, mantissa, bias):
    """The magnitudes of a small floating-point type's codes, in 64 bits."""
    one = 1 << mantissa
    return torch.tensor([(c % one) / one * 2.0 ** (1 - bias) if c < one else
                         (1 + (c % one) / one) * 2.0 ** (c // one - bias) for c in range(codes)],
                        dtype=torch.float64, device=DEV)


def _exact_fp4(x, fmt):
    """The 64-bit values that a matrix's 4-bit form stands for."""
    r, k = x.shape
    blk = FP4_BLOCK[fmt]
    v = x.double().view(r, k // blk, blk)
    top = v.abs().amax(2, keepdim=True)
    if fmt == "mx":
        scale = torch.exp2(torch.floor(torch.log2(top.clamp(min=2.0 ** -140))).sub(2).clamp(-127, 127))
        held = scale
    else:
        most = top.amax(1, keepdim=True)
        row = torch.where(most > 0, torch.exp2(torch.ceil(torch.log2(most / torch.full_like(most, 2688.0))).clamp(min=-126)), 1.0)
        held = _nearest(top / row / torch.full_like(top, 6.0), _grid(127, 3, 7)) * row
    q = _nearest(v / torch.where(held > 0, held, 1.0), _grid(8, 1, 1))
    return torch.where(held > 0, q * held, 0.0).view(r, k)


def _exact_append(c, s):
    page, qmax = c["page"], KV_QMAX[c["fmt"]]
    grid = None if c["fmt"] == "int8" else _grid(127, 3, 7)
    table = s["table"].tolist()
    at, sides = 0, []
    for codes, scales, turned in ((s["kc"], s["ks"], False), (s["vc"], s["vs"], True)):
        codes = codes.double()
        sides.append((codes.transpose(2, 3).contiguous() if turned else codes, scales.double()))
    for b, (n, ln) in enumerate(zip(s["news"], s["lens"].tolist())):
        for j in range((ln - n) // page, (ln - 1) // page + 1):
            lo, hi = max(ln - n, j * page), min(ln, (j + 1) * page)
            rows = slice(at + lo - (ln - n), at + hi - (ln - n))
            p = table[b][j]
            for (codes, scales), x in zip(sides, (s["k"], s["v"])):
                x = x[rows].double().transpose(0, 1)
                t = x.abs().amax((1, 2))
                t = t / torch.full_like(t, qmax)
                m, e = torch.frexp(t)
                t = torch.ldexp(torch.ceil(m * 256) / 256, e)
                had = scales[p].clone() if lo > j * page else torch.zeros_like(t)
                now = torch.maximum(had, t)
                safe = torch.where(now > 0, now, 1.0)[:, None, None]
                fresh, again = x / safe, codes[p, :, : lo - j * page] * had[:, None, None] / safe
                if grid is None:
                    fresh, again = fresh.round(), again.round()
                else:
                    fresh, again = _nearest(fresh, grid), _nearest(again, grid)
                codes[p, :, lo - j * page: hi - j * page] = fresh
                codes[p, :, : lo - j * page] = again
                scales[p] = now
        at += n
    return sides[0][0], sides[0][1], sides[1][0].transpose(2, 3).contiguous(), sides[1][1]


def _exact_attention(c, s):
    hq, h, d, page = c["q_heads"], c["kv_heads"], c["d"], c["page"]
    outs, at = [], 0
    for b, (n, ln) in enumerate(zip(s["news"], s["lens"].tolist())):
        ids = s["table"][b, : (ln + page - 1) // page].long()
        k = (s["kc"].view(torch.uint8)[ids].view(s["kc"].dtype).double() * s["ks"][ids].double()[..., None, None])
        v = (s["vc"].view(torch.uint8)[ids].view(s["vc"].dtype).double() * s["vs"][ids].double()[..., None, None])
        k = k.transpose(0, 1).reshape(h, -1, d)[:, :ln]
        v = v.permute(1, 0, 3, 2).reshape(h, -1, d)[:, :ln]
        o = torch.empty(n, hq, d, dtype=torch.float64, device=DEV)
        hidden = torch.arange(ln, device=DEV)[None, :] > (ln - n + torch.arange(n, device=DEV))[:, None]
        for j in range(hq):
            a = s["q"][at: at + n, j].double() @ k[j * h // hq].t() / math.sqrt(d)
            a = torch.softmax(a.masked_fill_(hidden, float("-inf")), 1)
            o[:, j] = a @ v[j * h // hq]
        outs.append(o)
        at += n
    return torch.cat(outs)


def exact(case, seed):
    s = prepare(case, seed)
    if case["op"] == "quantize":
        return _exact_fp4(s["x"], case["fmt"])
    if case["op"] == "linear":
        n, k = case["n"], case["k"]
        grid = torch.cat((_grid(8, 1, 1), -_grid(8, 1, 1)))
        codes = torch.stack((s["codes"] % 16, s["codes"] // 16), 2).view(n, k).int()
        blk = FP4_BLOCK[case["fmt"]]
        j = torch.arange(k // blk, device=DEV)[None, :]
        i = torch.arange(n, device=DEV)[:, None]
        b = s["scales"][i // 128, j // 4, i % 32 * 16 + i % 128 // 32 * 4 + j % 4].long()
        sc = torch.exp2(b.double() - 127) if case["fmt"] == "mx" else _grid(127, 3, 7)[b]
        w = (grid[codes].view(n, k // blk, blk) * sc[:, :, None]).view(n, k)
        if s["row"] is not None:
            w = w * s["row"].double()[:, None]
        return _exact_fp4(s["x"], case["fmt"]) @ w.t()
    return (_exact_append if case["op"] == "append" else _exact_attention)(case, s)
