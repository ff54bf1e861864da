"""GPU parity of the microscaled 4-bit floating-point quantization and linear,
and of appending to and attention over the 8-bit paged KV cache, against the
binary64 oracle on identical inputs.

Bars:
  * quantization and appending: every code, scale and value bit-exact;
  * linear: |y - ref| <= 2^-8 |ref| + (K/64 + 64) 2^-23 S + tiny, with
    S = sum_k |x||w|: one rounding to bf16 (at most half a step, 2^-8 of the
    value); K/64 binary32 accumulations that may each lose a unit of 2^-23 of
    a partial sum (<= S), and within one of them 64 products aligned to the
    largest, each losing at most such a unit;
  * attention: |o - ref| <= 2^-8 |ref| + (2^-11 + 2^-18 + 2 delta) W + A with
    W = sum_j p_j |v_j| and delta = (d/16 + 24) 2^-23 max_j scale sum |q||k_j|:
    the rounding to bf16, the probabilities' rounding to fp16 (2^-11), binary32
    sums and exponentials (2^-18), and the scores' binary32 error, which moves
    a probability and the normalizer by at most delta each.
    A = keys 2^-34 V, V the largest magnitude that any page's value scale can
    hold: a weighted probability is kept times 2^14 (rows kernel) or 2^9
    (tcgen05 kernel) in units of the largest value scale, and fp16's spacing
    under 2^-14 is 2^-24, so each of the smallest is off by at most 2^-25 2^-9
    of that (the normalizer is at least the largest probability, 1 in these
    units).
"""
import os
import subprocess
import sys

import numpy as np
import pytest
import torch

import weight_only_int4_quantize_b200 as w4
from oracle import lowp_oracle as L
from weight_only_int4_quantize_b200 import synth

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]

DEV = "cuda:0"
FMTS = ["mx", "nv"]
KV = {"int8": torch.int8, "e4m3": torch.float8_e4m3fn}


@pytest.fixture(autouse=True)
def no_device_error():
    yield
    torch.cuda.synchronize()
    assert w4.device_error(clear=True) == 0


# -------------------------------------------------------------- quantize ----

def check_quantize(x, fmt, x_dev=None):
    codes, scales, row, values = w4.fp4_quantize(x.to(DEV) if x_dev is None else x_dev, fmt,
                                                 values=True)
    plain = w4.fp4_quantize(x.to(DEV) if x_dev is None else x_dev, fmt)
    torch.cuda.synchronize()
    oc, ob, orow, ov = L.fp4_quantize(synth.bits(x), fmt)
    assert np.array_equal(codes.cpu().numpy(), L.fp4_pack(oc)), "codes differ"
    r, blocks = ob.shape
    i, j = np.arange(r)[:, None], np.arange(blocks)[None, :]
    assert np.array_equal(L.fp4_scale_byte(scales.cpu().numpy(), i, j), ob), "scales differ"
    if fmt == "nv":
        assert np.array_equal(row.cpu().numpy().astype(np.float64), orow)
    else:
        assert row is None
    # A value has at most 6 significant bits, so bf16 holds it unless it lies
    # under 2^-126, where bf16's spacing is 2^-133 and values go down to 2^-136.
    held = torch.from_numpy(ov).float().to(torch.bfloat16).double().numpy()
    assert np.array_equal(held[np.abs(ov) >= 2.0 ** -126], ov[np.abs(ov) >= 2.0 ** -126])
    assert np.array_equal(values.cpu().double().numpy(), held), "values differ"
    assert torch.equal(plain[0], codes)  # without values: the same codes
    return codes, scales, row


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("r,k", [(1, 128), (1, 2048), (3, 384), (33, 1024), (129, 1152),
                                 (200, 256), (7, 5120), (5, 17408), (300, 4096), (2, 33920)])
def test_quantize_bit_exact(fmt, r, k):
    check_quantize(synth.normal_weight(r, k, 0.02, seed=r + k, n_outliers=max(1, k // 100),
                                       outlier_scale=20.0), fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_ties_and_extremes(fmt):
    """Values on and next to every rounding border, at scales from the
    smallest subnormals to the largest bf16, zero rows and blocks, -0."""
    g = torch.Generator().manual_seed(5)
    ints = torch.randint(-255, 256, (64, 512), generator=g).float()
    rows = [ints * 2.0 ** e for e in (-135, -133, -126, -60, -8, 0, 40, 118)]
    grid = torch.tensor([0.25, 0.5, 0.75, 1, 1.25, 1.5, 1.75, 2, 2.5, 3, 3.5, 4, 5, 6, 7, -0.0])
    on = grid.repeat(32)[None, :] * 2.0 ** torch.arange(-20, 20).float()[:, None]
    near = on * (1 + torch.randint(-1, 2, on.shape, generator=g) * 2.0 ** -7)
    scaled = torch.randint(128, 256, (64, 32, 1), generator=g).float() / 128
    mixed = (torch.randint(0, 29, (64, 32, 16), generator=g) / 4 * scaled).reshape(64, 512)
    wide = torch.randn(64, 512, generator=g) * 2.0 ** torch.randint(-40, 1, (64, 512), generator=g)
    zero = torch.zeros(3, 512)
    zero[1, 300] = 1.0
    x = torch.cat(rows + [on, near, mixed, wide, zero, -zero]).to(torch.bfloat16)
    x[-1, 5] = 3.3e38
    check_quantize(x, fmt)


@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_strided_rows(fmt):
    wide = synth.normal_activations(37, 3 * 640, seed=9).to(DEV)
    part = wide[:, 640:1280]
    check_quantize(part.cpu().contiguous(), fmt, x_dev=part)


# ---------------------------------------------------------------- linear ----

def fp4_weight(n, k, fmt, seed):
    w = synth.normal_weight(n, k, 0.02, seed=seed, n_outliers=max(1, k // 128), outlier_scale=10.0)
    oc, ob, orow, ov = L.fp4_quantize(synth.bits(w), fmt)
    return w4.fp4_quantize(w.to(DEV), fmt), ov


def linear_bound(ref, xv, wv):
    k = xv.shape[1]
    s = np.abs(xv) @ np.abs(wv).T
    return 2.0 ** -8 * np.abs(ref) + (k / 64 + 64) * 2.0 ** -23 * s + 1e-38


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m,n,k", [
    (1, 1, 128), (1, 128, 256), (1, 2048, 2048), (2, 129, 384), (7, 1000, 1152), (16, 127, 640),
    (17, 300, 2176), (32, 256, 128), (33, 64, 896), (64, 333, 1024), (65, 130, 256),
    (128, 260, 512), (129, 128, 384), (200, 515, 1152), (256, 1001, 256), (257, 96, 128),
    (300, 384, 4096), (513, 2049, 640), (1, 5120, 17408), (13, 640, 17408), (1999, 200, 512),
    (400, 130, 384), (769, 300, 640), (385, 1, 128), (1152, 512, 2048),
    # several tiles for each pair of SMs: 256 and 384 token columns
    (1999, 2951, 384), (2300, 4300, 1536)])
def test_linear(fmt, m, n, k):
    (wc, ws, wr), wv = fp4_weight(n, k, fmt, seed=n + k)
    x = synth.normal_activations(m, k, seed=m + 3)
    _, _, _, xv = L.fp4_quantize(synth.bits(x), fmt)
    xc, xs, xr = w4.fp4_quantize(x.to(DEV), fmt)
    y = w4.fp4_linear(xc, xs, xr, wc, ws, wr, fmt)
    torch.cuda.synchronize()
    ref = xv @ wv.T
    err = np.abs(y.cpu().double().numpy() - ref)
    assert np.all(err <= linear_bound(ref, xv, wv))
    again = w4.fp4_linear(xc, xs, xr, wc, ws, wr, fmt, flags=w4.LINEAR_STATIC_WEIGHTS)
    assert torch.equal(y, again)  # and the same bits on every run


def test_linear_any_row_scales_and_padding_bytes():
    """Row scales that no quantizer of ours writes, and NaN scale bytes in the
    unused rows of the last tiles: neither disturbs a stored output."""
    m, n, k = 5, 70, 512
    (wc, ws, wr), wv = fp4_weight(n, k, "nv", seed=1)
    x = synth.normal_activations(m, k, seed=2)
    xc, xs, xr = w4.fp4_quantize(x.to(DEV), "nv")
    _, _, orow, xv = L.fp4_quantize(synth.bits(x), "nv")
    i = torch.arange(128, device=DEV)
    for tiles, rows in ((xs, m), (ws, n)):
        for j in range(4):
            at = (i[rows:] % 32) * 16 + i[rows:] // 32 * 4 + j
            tiles[0][:, at] = 0x7F
    f = torch.rand(n, generator=torch.Generator().manual_seed(3)) + 0.5
    y = w4.fp4_linear(xc, xs, xr * 0.37, wc, ws, (wr.cpu() * f).to(DEV), "nv")
    torch.cuda.synchronize()
    fx = np.float64(np.float32(0.37))
    ref = (xv * fx) @ (wv * f.double().numpy()[:, None]).T
    # two more binary32 products per side
    bound = linear_bound(ref, xv * fx, wv * f.double().numpy()[:, None]) + 4 * 2.0 ** -24 * np.abs(ref)
    assert np.all(np.abs(y.cpu().double().numpy() - ref) <= bound)


# ----------------------------------------------------------------- cache ----

class Problem:
    """A paged cache of arbitrary bytes, filled through the oracle's appends."""

    def __init__(self, fmt, heads, d, page, lens, news, q_heads, seed, spare_pages=3, pad_rows=0,
                 ragged_scale=1.0):
        g = torch.Generator().manual_seed(seed)
        self.fmt, self.heads, self.d, self.page, self.q_heads = fmt, heads, d, page, q_heads
        self.lens, self.news = np.array(lens), np.array(news)
        used = [-(-int(x) // page) for x in lens]
        total = sum(used) + spare_pages
        order = torch.randperm(total, generator=g).tolist()
        width = max(max(used), 1) + 1
        self.table = np.full((len(lens), width), -7, np.int32)  # never read behind a sequence
        for b, u in enumerate(used):
            for j in range(u):
                self.table[b, j] = order.pop()
        self.starts = np.concatenate([[0], np.cumsum(news)]).astype(np.int64)
        t = int(self.starts[-1]) + pad_rows
        # queries, keys and values are slices of one projection's rows
        width = (q_heads + 2 * heads) * d
        self.qkv = torch.randn(t, width, generator=g)
        self.qkv[:, q_heads * d:] *= ragged_scale ** torch.randint(-2, 3, (t, 1), generator=g)
        self.qkv = self.qkv.to(torch.bfloat16)
        raw = torch.randint(0, 256, (2, total, heads, page, d), generator=g, dtype=torch.uint8)
        if fmt == "int8":
            raw[raw == 128] = 0
        self.kc = raw[0].numpy().copy()
        self.vc = raw[1].numpy().copy().reshape(total, heads, d, page)
        sc = (torch.rand(2, total, heads, generator=g) * 0.05 + 0.002).to(torch.bfloat16)
        if fmt == "e4m3":
            sc = (sc.float() / 4).to(torch.bfloat16)
        self.ks, self.vs = sc.double().numpy()
        if fmt == "e4m3":  # what a sequence holds is a number; anything may lie behind it
            self._no_nan(self.kc, False)
            self._no_nan(self.vc, True)

    def _no_nan(self, codes, turned):
        nan = (codes & 0x7F) == 0x7F
        keep = np.zeros_like(nan)
        for b, ln in enumerate(self.lens):
            for j in range(-(-int(ln) // self.page)):
                cell = keep[self.table[b, j]]
                cell = cell.swapaxes(1, 2) if turned else cell
                cell[:, : min(self.page, int(ln) - j * self.page)] = True
        codes[nan & keep] = 0x38

    def part(self, lo, hi):
        d = self.d
        x = self.qkv.to(DEV)
        return x[:, lo * d: hi * d].view(x.shape[0], hi - lo, d)

    def host(self, lo, hi):
        d = self.d
        return self.qkv[:, lo * d: hi * d].double().numpy().reshape(-1, hi - lo, d)

    def cache(self):
        return w4.KV8Cache(torch.from_numpy(self.kc).to(DEV).view(KV[self.fmt]),
                           torch.from_numpy(self.vc).to(DEV).view(KV[self.fmt]),
                           torch.from_numpy(self.ks).float().to(DEV),
                           torch.from_numpy(self.vs).float().to(DEV))

    def batch(self, with_starts=True):
        table = torch.from_numpy(self.table).to(DEV)
        lens = torch.from_numpy(self.lens.astype(np.int32)).to(DEV)
        if not with_starts:
            return table, lens
        return table, lens, torch.from_numpy(self.starts.astype(np.int32)).to(DEV), \
            max(1, int(self.news.max()))

    def check_append(self, cache=None):
        hq, h = self.q_heads, self.heads
        cache = self.cache() if cache is None else cache
        want = L.kv_append(self.kc, self.vc, self.ks, self.vs, self.host(hq, hq + h),
                           self.host(hq + h, hq + 2 * h), self.table, self.lens, self.starts,
                           self.page, self.fmt)
        for _ in range(2):  # the second time changes nothing
            w4.kv8_append(cache, self.part(hq, hq + h), self.part(hq + h, hq + 2 * h), *self.batch())
            torch.cuda.synchronize()
            got = [x.view(torch.uint8).cpu().numpy() for x in cache[:2]] + \
                  [x.cpu().double().numpy() for x in cache[2:]]
            for name, a, b in zip(("k codes", "v codes", "k scales", "v scales"), got, want):
                assert np.array_equal(a, b), name
        self.kc, self.vc, self.ks, self.vs = want
        return cache

    def check_attention(self, cache=None, scale=None, with_starts=True):
        cache = self.cache() if cache is None else cache
        out = torch.full((self.qkv.shape[0], self.q_heads, self.d), 7.0, dtype=torch.bfloat16,
                         device=DEV)
        got = w4.kv8_attention(self.part(0, self.q_heads), cache, *self.batch(with_starts),
                               scale=scale, out=out)
        torch.cuda.synchronize()
        assert got is out
        sc = float(np.float32(self.d ** -0.5 if scale is None else scale))
        ref, weight, reach = L.kv_attention(self.host(0, self.q_heads), self.kc, self.vc, self.ks,
                                            self.vs, self.table, self.lens, self.starts, self.page,
                                            self.fmt, sc)
        got = got.cpu().double().numpy()
        rows = int(self.starts[-1])
        assert np.all(got[rows:] == 7.0)  # rows of no sequence are left as they were
        delta = (self.d / 16 + 24) * 2.0 ** -23 * reach[:rows]
        bound = 2.0 ** -8 * np.abs(ref[:rows]) + (2.0 ** -11 + 2.0 ** -18 + 2 * delta) * weight[:rows]
        bound = bound + max(self.lens) * 2.0 ** -34 * self.vs.max() * L.QMAX[self.fmt]
        err = np.abs(got[:rows] - ref[:rows])
        assert np.all(err <= bound + 1e-30), float(np.max(err / (bound + 1e-30)))
        again = w4.kv8_attention(self.part(0, self.q_heads), cache, *self.batch(with_starts),
                                 scale=scale, out=torch.empty_like(out))
        assert torch.equal(again[:rows], out[:rows])
        return out


APPENDS = [  # heads, d, page, lens, news
    (1, 64, 16, [1], [1]), (2, 128, 16, [16, 17, 33], [1, 1, 1]), (2, 128, 64, [70], [70]),
    (3, 64, 32, [5, 64, 100], [5, 3, 40]), (2, 128, 128, [128, 129, 300], [128, 2, 172]),
    (1, 128, 32, [40, 0, 7], [9, 0, 7]), (2, 64, 64, [200, 63], [137, 0]),
    (2, 64, 16, [3], [9]),  # longer than what is held: the first six are not
]


@pytest.mark.parametrize("fmt", list(KV))
@pytest.mark.parametrize("heads,d,page,lens,news", APPENDS)
def test_append_bit_exact(fmt, heads, d, page, lens, news):
    Problem(fmt, heads, d, page, lens, news, q_heads=heads, seed=sum(lens) + page,
            pad_rows=3).check_append()


@pytest.mark.parametrize("fmt", list(KV))
@pytest.mark.parametrize("exponent", [-133, -126, -112, 119])
def test_append_extreme_magnitudes(fmt, exponent):
    """bf16 values down to the smallest subnormals and up to the largest
    binades, and rounding borders: integers over 127 (or 448) land on them."""
    p = Problem(fmt, 2, 64, 32, [45], [45], q_heads=1, seed=12)
    g = torch.Generator().manual_seed(7)
    p.qkv = (torch.randint(-255, 256, p.qkv.shape, generator=g) * 2.0 ** exponent).to(torch.bfloat16)
    p.ks[:], p.vs[:] = 0, 0
    cache = p.check_append()
    p.lens, p.news = np.array([48]), np.array([3])
    p.starts = np.array([0, 3])
    p.qkv = (p.qkv.double() * 1.5).to(torch.bfloat16)
    p.check_append(cache)


@pytest.mark.parametrize("fmt", list(KV))
def test_append_growing_scales_and_zeros(fmt):
    """Token by token with magnitudes over 2^+-8, so that pages are rescaled
    again and again, and pages that hold only zeros."""
    p = Problem(fmt, 2, 64, 16, [16, 41], [1, 1], q_heads=2, seed=4)
    for step in range(12):
        p.lens = np.array([5 + step, 30 + step])
        g = torch.Generator().manual_seed(100 + step)
        p.qkv = (torch.randn(p.qkv.shape, generator=g) * 2.0 ** (step % 5 * 2 - 4)).to(torch.bfloat16)
        if step == 3:
            p.qkv.zero_()
        p.check_append()
    z = Problem(fmt, 1, 64, 16, [20], [20], q_heads=1, seed=5)
    z.qkv.zero_()
    z.check_append()
    z.check_attention()


ATTENTION = [  # heads, q_heads, d, page, lens, news
    (1, 1, 64, 16, [1], [1]), (2, 4, 64, 16, [300, 17, 16, 64, 65], [1] * 5),
    (2, 16, 128, 64, [1, 63, 64, 129, 1000], [1] * 5), (8, 16, 128, 64, [2000], [1]),
    (1, 32, 128, 32, [500, 31], [1, 1]), (3, 3, 128, 128, [127, 128, 700], [1] * 3),
    (2, 10, 64, 32, [40, 5], [1, 1]), (2, 4, 128, 16, [100, 20, 0, 9], [7, 20, 0, 1]),
    (1, 7, 64, 64, [200, 90], [33, 90]), (2, 2, 128, 32, [300], [150]),
    (2, 4, 64, 16, [3, 10], [9, 2]),  # tokens in front of position 0 see nothing
    (1, 2, 128, 128, [513, 255], [200, 255]),
]


@pytest.mark.parametrize("fmt", list(KV))
@pytest.mark.parametrize("heads,q_heads,d,page,lens,news", ATTENTION)
def test_attention(fmt, heads, q_heads, d, page, lens, news):
    p = Problem(fmt, heads, d, page, lens, news, q_heads, seed=sum(lens) + d, pad_rows=2)
    p.check_attention()


def test_attention_single_tokens_without_starts():
    p = Problem("int8", 2, 128, 64, [70, 3, 500], [1, 1, 1], 8, seed=3)
    a = p.check_attention(with_starts=False)
    assert torch.equal(a, p.check_attention())


LONG = [  # heads, q_heads, d, page, lens, news: the tcgen05 kernel's problems
    (16, 32, 64, 16, [300, 41], [260, 41]), (24, 48, 128, 64, [513, 255], [200, 255]),
    (12, 36, 64, 128, [385, 128, 0, 77], [200, 128, 0, 77]), (20, 20, 128, 32, [700], [600]),
    (12, 24, 128, 16, [100, 3, 260], [260, 3, 130]),  # some tokens in front of position 0
]


@pytest.mark.parametrize("fmt", list(KV))
@pytest.mark.parametrize("heads,q_heads,d,page,lens,news", LONG)
def test_attention_long_runs(fmt, heads, q_heads, d, page, lens, news):
    """Row tiles of which some warps have no live rows, key tiles that only
    the second row tile has, maxima and value scales that move late (large
    key scales, pages of very different scales)."""
    p = Problem(fmt, heads, d, page, lens, news, q_heads, seed=sum(lens) + d, pad_rows=2)
    for turn in range(2):
        p.check_attention()
        p.ks = p.ks * 4
        p.vs = p.vs * 2.0 ** np.random.RandomState(turn).randint(-4, 5, p.vs.shape)


def test_attention_negative_scale_and_strong_queries():
    p = Problem("int8", 24, 64, 32, [400], [300], 48, seed=6)
    p.check_attention(scale=-0.2)
    p.check_attention(scale=0.0)


@pytest.mark.parametrize("fmt", list(KV))
def test_attention_scales_spread(fmt):
    """Pages whose value scales differ by 2^10 and key scales that make the
    softmax all but one-hot; queries of very different magnitude."""
    p = Problem(fmt, 2, 128, 16, [333, 90], [1, 40], 8, seed=8)
    e = np.random.RandomState(1).randint(-5, 6, p.vs.shape)
    p.vs = p.vs * 2.0 ** e
    p.ks = p.ks * 8
    mult = 2.0 ** torch.randint(-30, 4, (p.qkv.shape[0], 1), generator=torch.Generator().manual_seed(2))
    p.qkv = (p.qkv.float() * mult).to(torch.bfloat16)
    p.check_attention()


def test_decode_steps_together():
    """A prompt and then single tokens through quantize, linear, append and
    attention, as a decoder layer's attention block runs them, on a stream of
    its own and replayed from a graph, against the same steps in binary64."""
    hid, hq, h, d, page, fmt = 512, 8, 4, 64, 16, "nv"
    n_qkv = (hq + 2 * h) * d
    (wc, ws, wr), wv = fp4_weight(n_qkv, hid, fmt, seed=31)
    (oc, os_, or_), ov = fp4_weight(hid, hq * d, fmt, seed=32)
    prompt = [21, 40]
    steps = 3
    cache = w4.kv8_cache(16, h, page, d, device=DEV)
    table = torch.arange(10, dtype=torch.int32).view(2, 5).to(DEV)
    kc, vc = (c.view(torch.uint8).cpu().numpy() for c in cache[:2])
    ks, vs = (c.cpu().double().numpy() for c in cache[2:])
    stream = torch.cuda.Stream(DEV)
    lens = np.zeros(2, np.int64)
    x_buf = lens_buf = graph = y = None
    for step in range(steps + 1):
        news = np.array(prompt if step == 0 else [1, 1])
        starts = np.concatenate([[0], np.cumsum(news)])
        lens = lens + news
        x = synth.normal_activations(int(starts[-1]), hid, seed=40 + step)

        def layer(x, lens_t, starts_t, most):
            qkv = w4.fp4_linear(*w4.fp4_quantize(x, fmt), wc, ws, wr, fmt)
            q = qkv[:, : hq * d].view(-1, hq, d)
            k = qkv[:, hq * d: (hq + h) * d].view(-1, h, d)
            v = qkv[:, (hq + h) * d:].view(-1, h, d)
            w4.kv8_append(cache, k, v, table, lens_t, starts_t, most)
            o = w4.kv8_attention(q, cache, table, lens_t, starts_t, most)
            return qkv, o, w4.fp4_linear(*w4.fp4_quantize(o.view(-1, hq * d), fmt), oc, os_, or_, fmt)

        lens_t = torch.tensor(lens, dtype=torch.int32, device=DEV)
        if step < 2:
            starts_t = torch.tensor(starts, dtype=torch.int32, device=DEV)
            stream.wait_stream(torch.cuda.current_stream())
            xd = x.to(DEV)
            stream.wait_stream(torch.cuda.current_stream())
            with torch.cuda.stream(stream):
                qkv, o, y = layer(xd, lens_t, starts_t, int(news.max()))
            stream.synchronize()
        else:
            if graph is None:
                x_buf, lens_buf = x.to(DEV), lens_t.clone()
                graph = torch.cuda.CUDAGraph()
                torch.cuda.synchronize()
                with torch.cuda.graph(graph):
                    qkv, o, y = layer(x_buf, lens_buf, None, None)
            x_buf.copy_(x.to(DEV))
            lens_buf.copy_(lens_t)
            graph.replay()
            torch.cuda.synchronize()
        xv = L.fp4_quantize(synth.bits(x), fmt)[3]
        ref = xv @ wv.T
        got = qkv.cpu()
        assert np.all(np.abs(got.double().numpy() - ref) <= linear_bound(ref, xv, wv))
        # each further step from the bits that the one before it wrote
        part = got.double().numpy().reshape(-1, hq + 2 * h, d)
        kc, vc, ks, vs = L.kv_append(kc, vc, ks, vs, part[:, hq: hq + h], part[:, hq + h:],
                                     table.cpu().numpy(), lens, starts, page, "int8")
        assert np.array_equal(cache.k_codes.view(torch.uint8).cpu().numpy(), kc)
        assert np.array_equal(cache.v_codes.view(torch.uint8).cpu().numpy(), vc)
        ro, weight, reach = L.kv_attention(part[:, :hq], kc, vc, ks, vs, table.cpu().numpy(), lens,
                                           starts, page, "int8", d ** -0.5)
        delta = (d / 16 + 24) * 2.0 ** -23 * reach
        bound = 2.0 ** -8 * np.abs(ro) + (2.0 ** -11 + 2.0 ** -18 + 2 * delta) * weight
        assert np.all(np.abs(o.cpu().double().numpy() - ro) <= bound + 1e-30)
        oq = L.fp4_quantize(synth.bits(o.cpu().view(-1, hq * d)), fmt)[3]
        ry = oq @ ov.T
        assert np.all(np.abs(y.cpu().double().numpy() - ry) <= linear_bound(ry, oq, ov))


# ------------------------------------------------------- bounds and hazards ----

GUARD = 4096


class Guarded:
    """A tensor inside a byte buffer whose guard regions must stay untouched."""

    def __init__(self, shape, dtype, fill=0x5A):
        n = int(np.prod(shape)) * torch.empty((), dtype=dtype).element_size()
        self.raw = torch.full((GUARD + n + GUARD,), 0x5A, dtype=torch.uint8, device=DEV)
        self.n = n
        self.raw[GUARD: GUARD + n] = fill
        self.t = self.raw[GUARD: GUARD + n].view(dtype).view(shape)

    def check(self, what):
        torch.cuda.synchronize()
        assert bool((self.raw[:GUARD] == 0x5A).all()), f"{what}: write before the buffer"
        assert bool((self.raw[GUARD + self.n:] == 0x5A).all()), f"{what}: write after the buffer"


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("r,k", [(1, 128), (37, 1152), (130, 5120)])
def test_quantize_outputs_guarded(fmt, r, k):
    x = synth.normal_activations(r, k, seed=r).to(DEV)
    codes, scales = Guarded((r, k // 2), torch.uint8), Guarded(w4.fp4_scale_shape(r, k, fmt), torch.uint8)
    row = Guarded((r,), torch.float32) if fmt == "nv" else None
    values = Guarded((r, k), torch.bfloat16)
    assert w4.lib().w4_fp4_quantize(x.data_ptr(), r, k, k, w4.FP4_FORMATS[fmt][0],
                                    codes.t.data_ptr(), scales.t.data_ptr(),
                                    row.t.data_ptr() if row else None, values.t.data_ptr(),
                                    torch.cuda.current_stream().cuda_stream) == 0
    for g, name in ((codes, "codes"), (scales, "scales"), (row, "row scales"), (values, "values")):
        if g is not None:
            g.check(name)
    # bytes of rows behind the last are left as they were
    last, used = scales.t[-1], r - (r - 1) // 128 * 128
    i = torch.arange(used, 128, device=DEV)
    for j in range(4):
        assert bool((last[:, (i % 32) * 16 + i // 32 * 4 + j] == 0x5A).all())


@pytest.mark.parametrize("fmt", FMTS)
@pytest.mark.parametrize("m,n,k", [(1, 77, 2048), (9, 129, 8192), (40, 130, 640), (100, 333, 2048),
                                   (200, 140, 8192), (300, 520, 1152), (1000, 1025, 256)])
def test_linear_output_guarded(fmt, m, n, k):
    (wc, ws, wr), _ = fp4_weight(n, k, fmt, seed=2)
    xc, xs, xr = w4.fp4_quantize(synth.normal_activations(m, k, seed=3).to(DEV), fmt)
    y = Guarded((m, n), torch.bfloat16)
    y.t.fill_(float("nan"))
    w4.fp4_linear(xc, xs, xr, wc, ws, wr, fmt, out=y.t)
    y.check(f"m={m} n={n} k={k}")
    assert not bool(torch.isnan(y.t).any())


@pytest.mark.parametrize("fmt", list(KV))
@pytest.mark.parametrize("heads,q_heads,d,page,lens,news", [
    (2, 4, 64, 16, [40, 7, 0], [3, 7, 0]), (3, 3, 128, 64, [129, 200], [1, 90]),
    (24, 48, 64, 32, [300, 50], [280, 20])])
def test_cache_and_attention_guarded(fmt, heads, q_heads, d, page, lens, news):
    """Appending writes nothing outside the cache, nor any page that no
    sequence appends to; attention nothing outside its rows."""
    p = Problem(fmt, heads, d, page, lens, news, q_heads, seed=11, pad_rows=2)
    g = []
    for t in p.cache():
        x = Guarded(t.shape, t.dtype)
        x.t.view(torch.uint8).copy_(t.view(torch.uint8))
        g.append(x)
    cache = w4.KV8Cache(*[x.t for x in g])
    p.check_append(cache)  # compares whole buffers, other pages among them
    out = Guarded((p.qkv.shape[0], q_heads, d), torch.bfloat16)
    w4.kv8_attention(p.part(0, q_heads), cache, *p.batch(), out=out.t)
    for x, name in zip(g + [out], ("k codes", "v codes", "k scales", "v scales", "out")):
        x.check(name)
    rows = int(p.starts[-1])
    assert bool((out.t[rows:].view(torch.uint8) == 0x5A).all())


@pytest.mark.parametrize("heads,news", [(2, [1, 3, 40]), (24, [1, 3, 300])])
def test_bad_device_indexes_are_skipped_and_recorded(heads, news):
    """Page ids, lengths and offsets outside the buffers: recorded in the
    device error word, the other sequences unharmed, nothing written for them."""
    lens = [33, 20, 310]
    p = Problem("int8", heads, 64, 16, lens, news, heads, seed=5)
    cache = p.cache()
    good = p.check_attention(cache)
    q, (table, ln, starts, most) = p.part(0, heads), p.batch()

    def run(table=table, ln=ln, starts=starts):
        before = [t.view(torch.uint8).clone() for t in cache]
        w4.kv8_append(cache, q, q, table, ln, starts, most)
        changed = [not torch.equal(a, t.view(torch.uint8)) for a, t in zip(before, cache)]
        for a, t in zip(before, cache):
            t.view(torch.uint8).copy_(a)
        out = torch.full_like(good, 7.0)
        w4.kv8_attention(q, cache, table, ln, starts, most, out=out)
        torch.cuda.synchronize()
        code = w4.device_error(clear=True)
        assert code & 2 and not code & 1, code
        return out, changed

    def rows(b):
        return slice(int(p.starts[b]), int(p.starts[b + 1]))

    for bad in (-1, cache.k_codes.shape[0], 2 ** 31 - 1, -2 ** 31):
        t = table.clone()
        t[1, 0] = bad
        out, _ = run(table=t)
        assert torch.equal(out[rows(0)], good[rows(0)]) and torch.equal(out[rows(2)], good[rows(2)])
    for bad in (-1, 16 * table.shape[1] + 1, 2 ** 31 - 1):
        x = ln.clone()
        x[1] = bad
        out, _ = run(ln=x)
        assert torch.equal(out[rows(0)], good[rows(0)]) and torch.equal(out[rows(2)], good[rows(2)])
        assert bool((out[rows(1)] == 7.0).all())
    x = starts.clone()
    x[3] = q.shape[0] + 1  # the last sequence's rows run over the buffer
    out, _ = run(starts=x)
    assert torch.equal(out[rows(0)], good[rows(0)]) and bool((out[rows(2)] == 7.0).all())
    x = starts.clone()
    x[0] = -5
    out, _ = run(starts=x)
    assert torch.equal(out[rows(1)], good[rows(1)]) and torch.equal(out[rows(2)], good[rows(2)])
    everything, changed = run(ln=torch.full_like(ln, -1))
    assert bool((everything == 7.0).all()) and not any(changed)
    with pytest.raises(w4.W4Error) as e:  # the status that the C ABI gives for it
        w4.kv8_attention(q, cache, table, torch.full_like(ln, -1), starts, most)
        torch.cuda.synchronize()
        w4._check(w4.lib().w4_device_error(1, None), "w4_device_error")
    assert e.value.name == "W4_ERR_DEVICE_INDEX"


def test_pages_beyond_32_bit_offsets():
    """Pages whose byte offsets pass 2^32, through each kernel."""
    page, d = 128, 128
    for heads, q_heads, lens, news in ((8, 16, [500, 200], [1, 1]), (8, 16, [500, 200], [1, 9]),
                                       (24, 48, [300], [260])):
        p = Problem("int8", heads, d, page, lens, news, q_heads, seed=9)
        small = p.cache()
        pages = 2 ** 32 // (heads * page * d) + 40
        shift = pages - small.k_codes.shape[0]
        big = w4.kv8_cache(pages, heads, page, d, device=DEV)
        for b, s in zip(big, small):
            b[shift:] = s
        table, *rest = p.batch()
        high = torch.where(table >= 0, table + shift, table)
        for f in (lambda c, t: w4.kv8_append(c, p.part(q_heads, q_heads + heads),
                                             p.part(q_heads + heads, q_heads + 2 * heads), t, *rest),
                  lambda c, t: w4.kv8_attention(p.part(0, q_heads), c, t, *rest)):
            a, b = f(small, table), f(big, high)
            if a is not None:
                assert torch.equal(a, b)
        for b, s in zip(big, small):
            assert torch.equal(b[shift:].view(torch.uint8), s.view(torch.uint8))
            assert not bool(b[:shift].view(torch.uint8).any())
        del big


def test_more_than_32_bit_elements():
    """Outputs and inputs of more than 2^31 elements: the last rows equal those
    of a small call."""
    for fmt in FMTS:
        x = torch.randn(70000, 128, device=DEV).to(torch.bfloat16)
        w = torch.randn(40000, 128, device=DEV).to(torch.bfloat16)
        xq, wq = w4.fp4_quantize(x, fmt), w4.fp4_quantize(w, fmt)
        y = w4.fp4_linear(*xq, *wq, fmt)
        tail = w4.fp4_linear(*w4.fp4_quantize(x[69632:], fmt), *wq, fmt)  # a multiple of 128 rows
        assert torch.equal(y[69632:], tail)
        del y, tail
    big = torch.zeros(150000, 16384, dtype=torch.bfloat16, device=DEV)
    big[-300:] = torch.randn(300, 16384, device=DEV).to(torch.bfloat16)
    for fmt in FMTS:
        codes, scales, row = w4.fp4_quantize(big, fmt)
        start = 149888 // 128 * 128
        c2, s2, r2 = w4.fp4_quantize(big[start:], fmt)
        assert torch.equal(codes[start:], c2)
        assert torch.equal(scales[start // 128:, :, :16], s2[:, :, :16])  # rows 0, 32, 64, 96 ...
        assert row is None or torch.equal(row[start:], r2)
        del codes, scales


def test_two_streams_at_once():
    """The same operators on two streams, problems of different sizes
    interleaved: nothing is shared between the calls."""
    streams = [torch.cuda.Stream(DEV) for _ in range(2)]
    probs = []
    for i, (m, n, k, fmt) in enumerate(((1, 2048, 4096, "mx"), (600, 1024, 2048, "nv"))):
        (wc, ws, wr), _ = fp4_weight(n, k, fmt, seed=i)
        x = synth.normal_activations(m, k, seed=50 + i).to(DEV)
        p = Problem("int8", 4, 64, 16, [900, 40], [1, 1], 8, seed=i)
        probs.append((x, wc, ws, wr, fmt, p, p.cache(), p.part(0, 8), p.batch(False)))
    torch.cuda.synchronize()

    def one(x, wc, ws, wr, fmt, p, cache, q, batch):
        return w4.fp4_linear(*w4.fp4_quantize(x, fmt), wc, ws, wr, fmt), w4.kv8_attention(q, cache, *batch)

    want = [one(*a) for a in probs]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(20):
        for s, a, g in zip(streams, probs, got):
            with torch.cuda.stream(s):
                g.append(one(*a))
    torch.cuda.synchronize()
    for w, g in zip(want, got):
        for y, o in g:
            assert torch.equal(y, w[0]) and torch.equal(o, w[1])


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("fmt", FMTS)
def test_quantize_keeps_infinities_to_their_row(fmt, bad):
    x = synth.normal_activations(200, 512, seed=8)
    clean = w4.fp4_quantize(x.to(DEV), fmt)
    x[77, 100] = bad
    codes, scales, row = w4.fp4_quantize(x.to(DEV), fmt)
    keep = np.arange(200) != 77
    assert np.array_equal(codes.cpu().numpy()[keep], clean[0].cpu().numpy()[keep])
    blocks = 512 // (32 if fmt == "mx" else 16)
    r, b = np.meshgrid(np.arange(200)[keep], np.arange(blocks), indexing="ij")
    at = (r // 128, b // 4, (r % 32) * 16 + (r % 128) // 32 * 4 + b % 4)
    assert np.array_equal(scales.cpu().numpy()[at], clean[1].cpu().numpy()[at])
    if row is not None:
        assert np.array_equal(row.cpu().numpy()[keep], clean[2].cpu().numpy()[keep])


@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_append_keeps_infinities_to_their_page(fmt, bad):
    dtype = torch.int8 if fmt == "int8" else torch.float8_e4m3fn
    table = torch.arange(6, dtype=torch.int32, device=DEV).view(2, 3)
    lens = torch.tensor([40, 35], dtype=torch.int32, device=DEV)
    starts = torch.tensor([0, 40, 75], dtype=torch.int32, device=DEV)
    k = synth.normal_activations(75, 2 * 64, seed=9).view(75, 2, 64).to(DEV)
    v = synth.normal_activations(75, 2 * 64, seed=10).view(75, 2, 64).to(DEV)
    caches = []
    for spoilt in (False, True):
        if spoilt:  # sequence 0, token 20 (page 1), kv head 1
            k[20, 1, 5] = bad
            v[20, 1, 6] = bad
        cache = w4.kv8_cache(6, 2, 16, 64, dtype, DEV)
        w4.kv8_append(cache, k, v, table, lens, starts, 40)
        caches.append([c.view(torch.uint8).cpu() if c.element_size() == 1 else c.cpu() for c in cache])
    for a, b in zip(*caches):
        a[1, 1] = 0
        b[1, 1] = 0
        assert torch.equal(a, b)
    assert w4.device_error() == 0


FIRST_CALLS = """
import torch
import weight_only_int4_quantize_b200 as w4
w4.lib()
dev = "cuda:0"
torch.manual_seed(0)
stream = torch.cuda.Stream()
x = torch.randn(300, 512, device=dev).bfloat16()
w = torch.randn(384, 512, device=dev).bfloat16()
k = torch.randn(4, 2, 128, device=dev).bfloat16()
q = torch.randn(4, 4, 128, device=dev).bfloat16()
long_q = torch.randn(300, 4, 128, device=dev).bfloat16()
long_k = torch.randn(300, 2, 128, device=dev).bfloat16()
table = torch.arange(4 * 128, dtype=torch.int32, device=dev).view(4, 128)
lens = torch.tensor([2000, 7, 300, 1], dtype=torch.int32, device=dev)
one = torch.tensor([300], dtype=torch.int32, device=dev)
ends = torch.tensor([0, 300], dtype=torch.int32, device=dev)
cache, other = w4.kv8_cache(512, 2, 16, 128), w4.kv8_cache(512, 2, 16, 128)

def run(cache):
    W = w4.fp4_quantize(w, "nv")
    X = w4.fp4_quantize(x, "nv")
    y = w4.fp4_linear(*X, *W, "nv")
    z = w4.fp4_linear(*w4.fp4_quantize(x[:3], "mx"), *w4.fp4_quantize(w, "mx"), "mx")
    w4.kv8_append(cache, long_k, long_k, table[2:3], one, ends, 300)
    w4.kv8_append(cache, k, k, table, lens)
    return y, z, w4.kv8_attention(q, cache, table, lens), \
        w4.kv8_attention(long_q, cache, table[2:3], one, ends, 300)

torch.cuda.synchronize()
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph, stream=stream):
    got = run(cache)
graph.replay()
graph.replay()
torch.cuda.synchronize()
want = run(other)
torch.cuda.synchronize()
assert all(torch.equal(a, b) for a, b in zip(got, want))
assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(cache, other))
assert w4.device_error() == 0
print("same")
"""


def test_first_calls_of_a_process_may_be_captured():
    """No call needs a warm-up before it is captured into a graph, and a
    replayed append leaves what one call leaves."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_CALLS], cwd=root, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0 and r.stdout.strip().endswith("same"), r.stdout + r.stderr
