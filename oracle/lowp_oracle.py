"""Oracle of the microscaled 4-bit linear and of the 8-bit paged KV cache.

Plain numpy in binary64, from the definitions in include/w4.h.  A quotient
that decides a rounding is either exactly on a border or, with scales of 8
significant bits, at least 2^-17 (relative) away from it, with any binary32
scales at least 2^-33, so binary64 decides them exactly.  Shares no code with
the CUDA side.
"""
from __future__ import annotations

import numpy as np

E2M1 = np.array([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0])
E4M3 = np.array([(c & 7) / 8 * 2.0 ** -6 if c < 8 else (1 + (c & 7) / 8) * 2.0 ** ((c >> 3) - 7)
                 for c in range(127)])
BLOCK = {"mx": 32, "nv": 16}
QMAX = {"int8": 127.0, "e4m3": 448.0}


def bf16(bits):
    """float64 values of uint16 bf16 patterns."""
    return (np.asarray(bits, np.uint32) << 16).view(np.float32).astype(np.float64)


def nearest_code(a, grid):
    """Index of the value of `grid` next to a >= 0 (ties to the even index,
    saturating)."""
    a = np.minimum(a, grid[-1])
    hi = np.searchsorted(grid, a)
    lo = np.maximum(hi - 1, 0)
    up, down = grid[hi] - a, a - grid[lo]
    return np.where(up < down, hi, np.where(down < up, lo, np.where(hi % 2 == 0, hi, lo)))


# ------------------------------------------------------------------- fp4 ----

def fp4_quantize(x_bits, fmt):
    """codes uint8 [R, K] (4-bit, sign in bit 3), scale bytes [R, K/block],
    row scales float64 [R] (ones for mx), values float64 [R, K]."""
    x = bf16(x_bits)
    r, k = x.shape
    b = BLOCK[fmt]
    v = x.reshape(r, k // b, b)
    amax = np.abs(v).max(2)
    row = np.ones(r)
    if fmt == "mx":
        with np.errstate(divide="ignore"):
            e = np.floor(np.log2(amax)) - 2
        e = np.clip(e, -127, 127)
        byte = (e + 127).astype(np.uint8)
        scale = 2.0 ** e
    else:
        top = amax.max(1)
        for i in range(r):
            if top[i] > 0:
                e = -126
                while top[i] > 2688.0 * 2.0 ** e:
                    e += 1
                row[i] = 2.0 ** e
        byte = nearest_code(amax / row[:, None] / 6.0, E4M3).astype(np.uint8)
        scale = E4M3[byte]
    held = scale * row[:, None]
    code = nearest_code(np.abs(v) / np.where(held > 0, held, 1.0)[:, :, None], E2M1)
    code = np.where(held[:, :, None] > 0, code, 0)
    value = np.where(np.signbit(v), -1.0, 1.0) * E2M1[code] * held[:, :, None]
    code = code | (np.signbit(v).astype(np.int64) << 3)
    return code.reshape(r, k).astype(np.uint8), byte, row, value.reshape(r, k)


def fp4_pack(codes):
    """[R, K] 4-bit codes -> [R, K/2] bytes, the even channel low."""
    return (codes[:, 0::2] | (codes[:, 1::2] << 4)).astype(np.uint8)


def fp4_scale_byte(tiles, row, block):
    """The byte of (row, block) in tiled scales [row tiles, column tiles, 512]."""
    return tiles[row // 128, block // 4, (row % 32) * 16 + (row % 128) // 32 * 4 + block % 4]


def fp4_values(codes, scale_bytes, row, fmt):
    """float64 values of 4-bit codes [R, K]."""
    s = 2.0 ** (scale_bytes.astype(np.float64) - 127) if fmt == "mx" else E4M3[scale_bytes]
    v = np.where(codes & 8, -1.0, 1.0) * E2M1[codes & 7]
    return v * np.repeat(s, BLOCK[fmt], axis=1) * np.asarray(row, np.float64)[:, None]


# ------------------------------------------------------------------- kv8 ----

def round_up_bf16(t):
    """float64 -> the next value of 8 significant bits, at least 2^-126 (0 for 0)."""
    m, e = np.frexp(t)
    return np.where(t > 0, np.maximum(np.ldexp(np.ceil(m * 256) / 256, e), 2.0 ** -126), 0.0)


def kv_decode(codes, fmt):
    """float64 values (in units of the scale) of cache bytes (uint8)."""
    if fmt == "int8":
        return codes.view(np.int8).astype(np.float64)
    return np.where(codes & 128, -1.0, 1.0) * E4M3[np.minimum(codes & 127, 126)]


def kv_encode(v, fmt):
    """Cache bytes of values in units of the scale."""
    if fmt == "int8":
        return np.clip(np.rint(v), -127, 127).astype(np.int8).view(np.uint8)
    return (nearest_code(np.abs(v), E4M3) | (np.signbit(v).astype(np.int64) << 7)).astype(np.uint8)


def kv_append(kc, vc, ks, vs, k, v, table, lens, starts, page, fmt):
    """Updates copies of the cache (bytes [P, H, page, d] / [P, H, d, page],
    scales float64 [P, H]) and returns them; k, v float64 [T, H, d]."""
    kc, vc, ks, vs = kc.copy(), vc.copy(), ks.copy(), vs.copy()
    for b in range(len(lens)):
        n, ln = starts[b + 1] - starts[b], lens[b]
        done = set()
        for i in range(n):
            p = ln - n + i
            if p < 0 or p // page in done:
                continue
            done.add(p // page)
            lo, hi = p, min(ln, (p // page + 1) * page)
            at, rows = table[b, p // page], slice(starts[b] + i, starts[b] + i + hi - lo)
            for h in range(k.shape[1]):
                for codes, scales, x, turned in ((kc, ks, k, False), (vc, vs, v, True)):
                    cell = codes[at, h].T if turned else codes[at, h]  # [page, d] view
                    new = x[rows, h]
                    had = scales[at, h] if lo % page else 0.0
                    s = max(had, float(round_up_bf16(np.abs(new).max() / QMAX[fmt])))
                    if lo % page and s > had:
                        old = kv_decode(np.ascontiguousarray(cell[: lo % page]), fmt)
                        cell[: lo % page] = kv_encode(old * had / s, fmt)
                    first = lo % page
                    cell[first: first + hi - lo] = kv_encode(new / s, fmt) if s > 0 else 0
                    scales[at, h] = s
    return kc, vc, ks, vs


def kv_attention(q, kc, vc, ks, vs, table, lens, starts, page, fmt, scale):
    """(out, sum p |v|, largest sum |q||k| * scale) float64 of q [T, Hq, d];
    rows of no sequence are NaN."""
    t, hq, d = q.shape
    h = kc.shape[1]
    out = np.full((t, hq, d), np.nan)
    weight = np.zeros((t, hq, d))
    reach = np.zeros((t, hq, 1))
    for b in range(len(lens)):
        n, ln = starts[b + 1] - starts[b], lens[b]
        ids = table[b, : (ln + page - 1) // page]
        for head in range(hq):
            kh = head * h // hq
            kk = (kv_decode(kc[ids, kh], fmt) * ks[ids, kh][:, None, None]).reshape(-1, d)[:ln]
            vv = kv_decode(vc[ids, kh], fmt) * vs[ids, kh][:, None, None]
            vv = vv.transpose(0, 2, 1).reshape(-1, d)[:ln]
            for i in range(n):
                r, seen = starts[b] + i, ln - n + i + 1
                if seen <= 0:
                    out[r, head] = 0.0
                    continue
                s = kk[:seen] @ q[r, head] * scale
                p = np.exp(s - s.max())
                p /= p.sum()
                out[r, head] = p @ vv[:seen]
                weight[r, head] = p @ np.abs(vv[:seen])
                reach[r, head] = (np.abs(kk[:seen]) @ np.abs(q[r, head])).max() * abs(scale)
    return out, weight, reach
