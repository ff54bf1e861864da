"""Host-side checks of the microscaled 4-bit and 8-bit KV cache entry points
(no GPU needed): refusals of the C ABI and of the binding, and pins of the
oracle that their GPU tests use."""
import ctypes
import itertools
import os
from fractions import Fraction

import numpy as np
import pytest
import torch

import weight_only_int4_quantize_b200 as w4
from oracle import lowp_oracle as L
from weight_only_int4_quantize_b200 import synth

A, B = 0x10000, 0x20000  # aligned fake device addresses: validation touches no device


@pytest.fixture(scope="module")
def lib():
    if not os.path.exists(w4.LIB_PATH):
        from weight_only_int4_quantize_b200 import build
        build.build()
    return w4.lib()


# -------------------------------------------------------------- refusals ----

def test_scale_bytes(lib):
    f = lib.w4_fp4_scale_bytes
    for r, k, fmt in itertools.product((1, 128, 129, 1000), (128, 384, 17408), ("mx", "nv")):
        assert f(r, k, w4.FP4_FORMATS[fmt][0]) == int(np.prod(w4.fp4_scale_shape(r, k, fmt)))
    assert f(0, 128, 0) == 0 and f(1, 100, 0) == 0 and f(1, 128, 2) == 0


def test_fp4_quantize_validation(lib):
    f = lib.w4_fp4_quantize
    assert f(None, 4, 128, 128, 0, A, A, None, None, None) == 1
    assert f(A, 4, 128, 128, 0, None, A, None, None, None) == 1
    assert f(A, 4, 128, 128, 0, A, A, A, None, None) == 1       # mx has no row scales
    assert f(A, 4, 128, 128, 1, A, A, None, None, None) == 1    # nv needs them
    assert f(A, 4, 128, 128, 2, A, A, None, None, None) == 4    # no such format
    assert f(A, 0, 128, 128, 0, A, A, None, None, None) == 2
    assert f(A, 4, 96, 128, 0, A, A, None, None, None) == 2     # K % 128
    assert f(A, 4, 128, 120, 0, A, A, None, None, None) == 2    # rows overlap
    assert f(A, 1 << 32, 128, 128, 0, A, A, None, None, None) == 2
    assert f(A + 2, 4, 128, 128, 0, A, A, None, None, None) == 3
    assert f(A, 4, 128, 132, 0, A, A, None, None, None) == 3    # rows off 16 bytes
    assert f(A, 4, 128, 128, 0, A, A, None, A + 8, None) == 3


def test_fp4_linear_validation(lib):
    f = lib.w4_fp4_linear
    mx = lambda **k: f(*[k.get(n, d) for n, d in (  # noqa: E731
        ("xc", A), ("xs", A), ("xr", None), ("m", 4), ("wc", A), ("ws", A), ("wr", None), ("n", 8),
        ("k", 128), ("fmt", 0), ("y", B), ("flags", 0), ("stream", None))])
    assert mx(xc=None) == 1 and mx(ws=None) == 1 and mx(y=None) == 1
    assert mx(xr=A) == 1 and mx(wr=A) == 1 and mx(fmt=1) == 1 and mx(fmt=1, xr=A) == 1
    assert mx(flags=1) == 1 and mx(flags=4) == 1
    assert mx(fmt=3) == 4
    assert mx(m=0) == 2 and mx(n=0) == 2 and mx(k=64) == 2 and mx(m=1 << 31) == 2
    assert mx(y=B + 8) == 3 and mx(fmt=1, xr=A + 4, wr=A) == 3


def _cache(**over):
    c = dict(k_codes=A, v_codes=A, k_scales=A, v_scales=A, num_pages=10, kv_heads=2, page_size=16,
             head_dim=64, format=0)
    c.update(over)
    return w4._KV8Cache(**c)


def test_kv8_validation(lib):
    def append(cache=None, null=False, **k):
        c = _cache(**(cache or {}))
        return lib.w4_kv8_append(None if null else ctypes.byref(c), *[k.get(n, d) for n, d in (
            ("k", A), ("ldk", 128), ("v", A), ("ldv", 128), ("rows", 5), ("table", A), ("pages", 4),
            ("lens", A), ("starts", A), ("batch", 3), ("most", 2), ("stream", None))])

    def attend(cache=None, null=False, **k):
        c = _cache(**(cache or {}))
        return lib.w4_kv8_attention(*[k.get(n, d) for n, d in (
            ("q", A), ("ldq", 256), ("rows", 5), ("heads", 4))], None if null else ctypes.byref(c),
            *[k.get(n, d) for n, d in (
                ("table", A), ("pages", 4), ("lens", A), ("starts", A), ("batch", 3), ("most", 2),
                ("scale", 1.0), ("out", B), ("stream", None))])

    for f in (append, attend):
        assert f(null=True) == 1 and f(table=None) == 1 and f(lens=None) == 1
        for name in ("k_codes", "v_codes", "k_scales", "v_scales"):
            assert f({name: None}) == 1 and f({name: A + 8}) == 3
        assert f({"format": 2}) == 4 and f({"head_dim": 96}) == 4
        for page in (0, 8, 24, 256, -16):
            assert f({"page_size": page}) == 4
        assert f({"num_pages": 0}) == 2 and f({"kv_heads": 0}) == 2
        assert f(pages=0) == 2 and f(pages=1 << 27) == 2
        assert f(batch=0) == 2 and f(most=0) == 2 and f(most=6) == 2 and f(rows=1 << 32) == 2
        assert f(starts=None) == 2                      # without starts: one row per sequence
        assert f(starts=None, rows=3, most=2) == 2
        assert f(table=A + 2) == 3 and f(lens=A + 1) == 3 and f(starts=A + 2) == 3
    assert append(k=None) == 1 and append(v=None) == 1
    assert append(ldk=120) == 2 and append(ldv=64) == 2
    assert append(ldk=132) == 3 and append(k=A + 8) == 3
    assert append(rows=1 << 30, most=1 << 30, batch=1 << 10) == 4   # units of a launch
    assert attend(q=None) == 1 and attend(out=None) == 1
    assert attend(scale=float("nan")) == 1 and attend(scale=float("inf")) == 1
    assert attend(heads=3) == 2 and attend(heads=0) == 2 and attend(ldq=248) == 2
    assert attend(ldq=260) == 3 and attend(out=B + 2) == 3


def test_binding_refuses_tensors(lib):
    x = torch.zeros(4, 128, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        w4.fp4_quantize(x)                              # not on a GPU
    with pytest.raises(ValueError):
        w4.fp4_quantize(x, "e2m1")
    with pytest.raises(ValueError):
        w4.fp4_scale_shape(1, 128, "fp4")
    with pytest.raises(TypeError):
        w4.fp4_linear(x, x, None, x, x, None)
    cache = w4.kv8_cache(4, 2, 16, 64, device="cpu")
    assert cache.k_codes.shape == (4, 2, 16, 64) and cache.v_codes.shape == (4, 2, 64, 16)
    with pytest.raises(TypeError):
        w4.kv8_cache(4, 2, 16, 64, dtype=torch.float16, device="cpu")
    q = torch.zeros(3, 4, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        w4.kv8_attention(q, cache, None, None)


def test_row_strides_refused(lib):
    """Only the first axis may be strided, and rows may not overlap; what
    passes these checks is refused for not lying on a GPU."""
    base = torch.zeros(6, 256, dtype=torch.bfloat16)
    for ok in (base, base[:, :128], base[:, 128:], base[2:3]):
        with pytest.raises(TypeError, match="CUDA"):
            w4.fp4_quantize(ok)
    for bad in (base.t(), base[:, ::2], base[:1].expand(6, 256)):
        with pytest.raises(ValueError):
            w4.fp4_quantize(bad)
    with pytest.raises(ValueError):
        w4.fp4_quantize(base[0])
    with pytest.raises(TypeError):
        w4.fp4_quantize(base.float())


def test_shape_mismatches_refused(lib):
    """The C ABI takes bare pointers: the binding refuses buffers of another
    size before it asks where they lie."""
    u8 = lambda *s: torch.zeros(s, dtype=torch.uint8)  # noqa: E731
    bf = lambda *s: torch.zeros(s, dtype=torch.bfloat16)  # noqa: E731
    xs, ws = u8(1, 1, 512), u8(2, 1, 512)
    with pytest.raises(TypeError, match="CUDA"):
        w4.fp4_linear(u8(4, 64), xs, None, u8(130, 64), ws, None, out=bf(4, 130))
    with pytest.raises(ValueError):
        w4.fp4_linear(u8(4, 64), xs, None, u8(130, 128), ws, None)         # K differs
    with pytest.raises(ValueError):
        w4.fp4_linear(u8(4, 64), xs, None, u8(130, 64), xs, None)          # scale tiles
    with pytest.raises(ValueError):
        w4.fp4_linear(u8(4, 64), xs, None, u8(130, 64), ws, torch.zeros(130))
    with pytest.raises(ValueError):
        w4.fp4_linear(u8(4, 64), u8(1, 2, 512), torch.zeros(3), u8(130, 64), u8(2, 2, 512),
                      torch.zeros(130), "nv")
    with pytest.raises(ValueError):
        w4.fp4_linear(u8(4, 64), u8(1, 2, 512), None, u8(130, 64), u8(2, 2, 512), None, "nv")
    with pytest.raises(ValueError):
        w4.fp4_linear(u8(4, 64), xs, None, u8(130, 64), ws, None, out=bf(4, 131))
    with pytest.raises(ValueError):
        w4.fp4_linear(u8(4, 128)[:, ::2], xs, None, u8(130, 64), ws, None)
    with pytest.raises(TypeError):
        w4.fp4_linear(u8(4, 64).char(), xs, None, u8(130, 64), ws, None)
    with pytest.raises(TypeError):
        w4.fp4_linear(u8(4, 64), xs, None, u8(130, 64), ws, None, flags="none")
    cache = w4.kv8_cache(4, 2, 16, 64, device="cpu")
    table, lens = torch.zeros(3, 2, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    starts, k = torch.zeros(4, dtype=torch.int32), bf(5, 2, 64)
    for f in (lambda c=cache, x=k, *a: w4.kv8_append(c, x, x, *a),
              lambda c=cache, x=k, *a: w4.kv8_attention(x, c, *a)):
        with pytest.raises(TypeError, match="CUDA"):
            f(cache, k, table, lens, starts, 2)
        with pytest.raises(ValueError):
            f(cache, k, table, lens, starts)                               # max_new missing
        with pytest.raises(ValueError):
            f(cache, k, table, lens, starts[:3], 2)
        with pytest.raises(ValueError):
            f(cache, k, table, lens[:2], starts, 2)
        with pytest.raises(ValueError):
            f(cache, k, table[0], lens, starts, 2)
        with pytest.raises(ValueError):
            f(cache, k, table, lens, None, 2)
        with pytest.raises(TypeError):
            f(cache, k, table.long(), lens, starts, 2)
        with pytest.raises(TypeError):
            f(cache, k.float(), table, lens, starts, 2)
        with pytest.raises(ValueError):
            f(cache, k[:, :, :32], table, lens, starts, 2)
        with pytest.raises(ValueError):
            f(cache._replace(v_codes=cache.k_codes), k, table, lens, starts, 2)
        with pytest.raises(ValueError):
            f(cache._replace(k_scales=cache.k_scales[:3]), k, table, lens, starts, 2)
        with pytest.raises(TypeError):
            f(cache._replace(k_codes=cache.k_codes.float()), k, table, lens, starts, 2)
        with pytest.raises(TypeError):
            f(list(cache), k, table, lens, starts, 2)
    with pytest.raises(ValueError):
        w4.kv8_append(cache, k, k[:4], table, lens, starts, 2)
    with pytest.raises(ValueError):
        w4.kv8_append(cache, k[:, :1], k[:, :1], table, lens, starts, 2)
    with pytest.raises(ValueError):
        w4.kv8_attention(k, cache, table, lens, starts, 2, out=k[:4])


def test_missing_extension_fails_loudly(lib, monkeypatch):
    import sys
    monkeypatch.setattr(w4, "_TENSORS", None)
    monkeypatch.delattr(w4, "_tensors", raising=False)
    monkeypatch.setitem(sys.modules, w4.__name__ + "._tensors", None)
    with pytest.raises(RuntimeError, match="no fallback"):
        w4.fp4_quantize(torch.zeros(1, 128, dtype=torch.bfloat16))


# ----------------------------------------------------------- oracle pins ----

def test_oracle_grids():
    assert list(L.E2M1) == [0, 0.5, 1, 1.5, 2, 3, 4, 6]
    bytes_ = torch.arange(127, dtype=torch.uint8)
    assert np.array_equal(bytes_.view(torch.float8_e4m3fn).double().numpy(), L.E4M3)


def _rational_nearest(a, grid):
    """Nearest grid value by exact comparison of distances, ties to the even index."""
    best = min(range(len(grid)), key=lambda i: (abs(a - grid[i]), i % 2))
    return best if a < grid[-1] else len(grid) - 1


@pytest.mark.parametrize("fmt", ["mx", "nv"])
def test_oracle_fp4_against_rationals(fmt):
    g = torch.Generator().manual_seed(1)
    x = torch.randn(4, 128, generator=g) * 2.0 ** torch.randint(-6, 7, (4, 1), generator=g)
    x[0, :40] = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, -0.0]).repeat(4)
    x[1, 16:48] = 0
    x = x.to(torch.bfloat16)
    codes, byte, row, value = L.fp4_quantize(synth.bits(x), fmt)
    e2m1 = [Fraction(float(v)) for v in L.E2M1]
    e4m3 = [Fraction(float(v)) for v in L.E4M3]
    blk = L.BLOCK[fmt]
    for r in range(4):
        xs = [Fraction(float(v)) for v in x[r]]
        f = Fraction(1)
        if fmt == "nv":
            top, f = max(abs(v) for v in xs), Fraction(1, 2 ** 126)
            while top > 2688 * f:
                f *= 2
        assert Fraction(float(row[r])) == f
        for b in range(128 // blk):
            part = xs[b * blk: (b + 1) * blk]
            top = max(abs(v) for v in part)
            if fmt == "mx":
                e = -127
                while e < 127 and top >= Fraction(2) ** (e + 3):
                    e += 1
                assert byte[r, b] == e + 127
                s = Fraction(2) ** e
            else:
                c = _rational_nearest(top / f / 6, e4m3)
                assert byte[r, b] == c
                s = e4m3[c] * f
            for i, v in enumerate(part):
                c = _rational_nearest(abs(v) / s, e2m1) if s else 0
                assert codes[r, b * blk + i] & 7 == c
                want = e2m1[c] * s * (-1 if v < 0 else 1)
                assert Fraction(float(value[r, b * blk + i])) == want
    assert np.array_equal(L.fp4_values(codes, byte, row, fmt), value)


def test_oracle_scale_tiles_are_a_permutation():
    rows, blocks = 256, 8
    tiles = np.arange(rows * blocks).reshape(2, 2, 512)
    i, j = np.arange(rows)[:, None], np.arange(blocks)[None, :]
    assert sorted(L.fp4_scale_byte(tiles, i, j).ravel()) == list(range(rows * blocks))
    # rows 0, 32, 64, 96 of a tile are the four words of its first 16 bytes
    assert [int(L.fp4_scale_byte(tiles, r, 0)) for r in (0, 32, 64, 96, 1)] == [0, 4, 8, 12, 16]


@pytest.mark.parametrize("fmt", ["int8", "e4m3"])
def test_oracle_append_against_rationals(fmt):
    rng = np.random.RandomState(3)
    k, v = rng.randn(2, 9, 1, 4) * 3
    k = torch.from_numpy(k).to(torch.bfloat16).double().numpy()
    v = torch.from_numpy(v * 40).to(torch.bfloat16).double().numpy()
    zero = np.zeros((3, 1, 16, 4), np.uint8)
    table = np.array([[2, 0]])
    cache = (zero, zero.transpose(0, 1, 3, 2).copy(), np.zeros((3, 1)), np.zeros((3, 1)))
    cache = L.kv_append(*cache, k[:6], v[:6], table, [6], [0, 6], 16, fmt)
    kc, vc, ks, vs = L.kv_append(*cache, k[6:], v[6:], table, [9], [0, 3], 16, fmt)
    grid = ([Fraction(i) for i in range(128)] if fmt == "int8" else
            [Fraction(float(x)) for x in L.E4M3])
    q = Fraction(127 if fmt == "int8" else 448)

    def up(t):
        e = 0
        while t * Fraction(2) ** e < 128:
            e += 1
        while t * Fraction(2) ** e >= 256:
            e -= 1
        n = t * Fraction(2) ** e
        return Fraction(-(-n.numerator // n.denominator)) / Fraction(2) ** e

    for x, codes, scales in ((k, kc, ks), (v, vc.transpose(0, 1, 3, 2), vs)):
        x = [[Fraction(float(a)) for a in row] for row in x[:, 0]]
        s0 = up(max(abs(a) for row in x[:6] for a in row) / q)
        s1 = max(s0, up(max(abs(a) for row in x[6:] for a in row) / q))
        assert Fraction(float(scales[2, 0])) == s1
        got = L.kv_decode(np.ascontiguousarray(codes[2, 0, :9]), fmt)
        for t, row in enumerate(x):
            for c, a in enumerate(row):
                m = grid[_rational_nearest(abs(a) / (s0 if t < 6 else s1), grid)]
                if t < 6 and s1 > s0:
                    m = grid[_rational_nearest(m * s0 / s1, grid)]
                assert abs(Fraction(float(got[t, c]))) == m
                assert got[t, c] == 0 or (got[t, c] < 0) == (a < 0)
        assert np.all(codes[[0, 1]] == 0) and np.all(codes[2, 0, 9:] == 0)


def test_oracle_attention_closed_forms():
    """Equal keys average the values seen; a page's scale multiplies its
    values; one far larger key takes all; a token before position 0 gets 0."""
    d, page = 4, 16
    kc = np.zeros((2, 1, page, d), np.uint8)
    vc = np.zeros((2, 1, d, page), np.uint8)
    vc[:, 0, 0, :] = np.arange(32).reshape(2, page).astype(np.uint8)
    one = np.ones((2, 1))
    vs = np.array([[1.0], [2.0]])
    q = np.ones((3, 2, d))
    o, w, _ = L.kv_attention(q, kc, vc, one, vs, np.array([[0, 1]]), [18], [0, 3], page, "int8", 0.5)
    for i, seen in enumerate((16, 17, 18)):
        vals = [float(j) if j < 16 else 2.0 * j for j in range(seen)]
        assert np.allclose(o[i, :, 0], np.mean(vals), rtol=1e-14)
    kc[0, 0, 5] = 100
    o, _, _ = L.kv_attention(q, kc, vc, one, vs, np.array([[0, 1]]), [18], [0, 3], page, "int8", 0.5)
    assert np.allclose(o[:, :, 0], 5.0, rtol=1e-12)
    o, _, _ = L.kv_attention(q, kc, vc, one, vs, np.array([[0, 1]]), [2], [0, 3], page, "int8", 0.5)
    assert np.all(o[0] == 0) and np.allclose(o[1, :, 0], 0.0) and np.allclose(o[2, :, 0], 0.5)
