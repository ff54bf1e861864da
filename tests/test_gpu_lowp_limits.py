"""GPU tests of the microscaled and 8-bit KV cache operators at the ends of
what their contracts allow.

Appending is bit-exact against the binary64 oracle, attention within the bound
that test_gpu_lowp.py derives (its allowance of 1e-30 replaced by half of
bf16's smallest spacing, 2^-134).
"""
import numpy as np
import pytest
import torch

import weight_only_int4_quantize_b200 as w4
from oracle import lowp_oracle as L
from tests.test_gpu_lowp import DEV, KV, Problem
from weight_only_int4_quantize_b200 import synth

pytestmark = [pytest.mark.gpu,
              pytest.mark.skipif(not torch.cuda.is_available(), reason="needs a CUDA GPU")]


@pytest.fixture(autouse=True)
def no_device_error():
    yield
    torch.cuda.synchronize()
    assert w4.device_error(clear=True) == 0


# ------------------------------------------------------- foreign cache scales ----

def foreign_scales(p, seed, low, high):
    """Scales of 24 significant bits, log-uniform between low and high."""
    r = np.random.RandomState(seed)
    for name in ("ks", "vs"):
        s = np.exp(r.uniform(np.log(low), np.log(high), getattr(p, name).shape))
        setattr(p, name, s.astype(np.float32).astype(np.float64))


@pytest.mark.parametrize("fmt", list(KV))
@pytest.mark.parametrize("heads,d,page,lens,news", [
    (8, 128, 128, [100, 228, 64, 1000], [50, 60, 1, 30]), (4, 64, 16, [9, 31, 200, 17], [1, 3, 11, 8]),
    (2, 128, 64, [40] * 6, [1] * 6), (3, 64, 32, [70, 31, 96], [35, 30, 90])])
def test_append_into_pages_of_foreign_scales(fmt, heads, d, page, lens, news):
    """Scales that this operator did not write have up to 24 significant bits:
    quotients come closer to a rounding border than with its own 8-bit ones.
    Half of the scales are larger than the new tokens need, so they stay and
    the new codes are quotients by them; half are smaller, so the earlier codes
    are products with them."""
    p = Problem(fmt, heads, d, page, lens, news, q_heads=heads, seed=sum(lens) + d)
    need = 4.5 / L.QMAX[fmt]  # about the largest of some thousand normal values
    foreign_scales(p, d + page, need / 8, need * 8)
    p.check_append()


@pytest.mark.parametrize("fmt", list(KV))
def test_append_near_ties_of_foreign_scales(fmt):
    """Scales chosen so that a new token's quotient misses a border by one
    unit in the last place of the scale, on either side."""
    heads = 16
    p = Problem(fmt, heads, 64, 16, [5], [1], q_heads=heads, seed=3)
    r = np.random.RandomState(5)
    x = r.randint(128, 256, (heads, 64)) / 128.0
    border = {"int8": r.randint(40, 120, heads) + 0.5,
              "e4m3": (r.randint(8, 16, heads) + 0.5) * 8}[fmt]
    page = p.table[0, 0]
    for name in ("ks", "vs"):
        s = (x[:, 0] / border).astype(np.float32)
        s = np.where(np.arange(heads) % 2 == 0, np.nextafter(s, np.float32(0)),
                     np.nextafter(s, np.float32(9)))
        getattr(p, name)[page] = s.astype(np.float64)
    x[:, 1:] = np.minimum(x[:, 1:], x[:, :1])
    p.qkv = torch.from_numpy(np.tile(x.reshape(-1), 3)[None]).to(torch.bfloat16)
    p.check_append()


@pytest.mark.parametrize("fmt", list(KV))
@pytest.mark.parametrize("scale", [1e-45, 9.2e-41, 1e-39, 1.3e-38, 3e38])
def test_append_foreign_scales_at_the_ends_of_the_range(fmt, scale):
    """Scales under 2^-126 (their reciprocal is no binary32 number) and next
    to the largest number: with new tokens of zeros and of ordinary values."""
    for zero in (True, False):
        p = Problem(fmt, 2, 64, 32, [20, 40], [7, 1], q_heads=2, seed=4)
        p.ks[:] = p.vs[:] = np.float64(np.float32(scale))
        if zero:
            p.qkv.zero_()
        p.check_append()


# ------------------------------------------------------------ attention limits ----

def attention_error(p, scale=None):
    """Largest error of the kernel in units of its bound, which allows 2^-134
    beside the relative terms, and the reference."""
    got = w4.kv8_attention(p.part(0, p.q_heads), p.cache(), *p.batch(), scale=scale)
    torch.cuda.synchronize()
    sc = float(np.float32(p.d ** -0.5 if scale is None else scale))
    rows = int(p.starts[-1])
    ref, weight, reach = L.kv_attention(p.host(0, p.q_heads), p.kc, p.vc, p.ks, p.vs, p.table, p.lens,
                                        p.starts, p.page, p.fmt, sc)
    delta = (p.d / 16 + 24) * 2.0 ** -23 * reach[:rows]
    bound = (2.0 ** -8 * np.abs(ref[:rows]) + (2.0 ** -11 + 2.0 ** -18 + 2 * delta) * weight[:rows] +
             max(p.lens) * 2.0 ** -34 * p.vs.max() * L.QMAX[p.fmt] + 2.0 ** -134)
    err = np.abs(got.cpu().double().numpy()[:rows] - ref[:rows])
    assert not np.any(np.isnan(err))
    return float(np.max(err / bound)), ref[:rows]


KERNELS = [  # heads, q_heads, d, lens, news: the rows kernel with 8 and 16 rows, the tcgen05 kernel
    (2, 4, 128, [700, 33], [1, 1]), (2, 4, 64, [300, 90], [1, 9]), (24, 48, 64, [400], [300]),
    (24, 48, 128, [400, 290], [200, 290])]


@pytest.mark.parametrize("fmt", list(KV))
@pytest.mark.parametrize("heads,q_heads,d,lens,news", KERNELS)
@pytest.mark.parametrize("exponent", [-120, 0, 100, 125])
def test_attention_values_at_the_ends_of_the_range(fmt, heads, q_heads, d, lens, news, exponent):
    """Values whose largest lie next to 2^126: the outputs are averages of
    them, so as finite.  Values near 2^-113, and ordinary ones."""
    p = Problem(fmt, heads, d, 32, lens, news, q_heads, seed=21)
    r = np.random.RandomState(exponent & 15)
    top = 2.0 ** (exponent if exponent < 100 else exponent - (6 if fmt == "int8" else 8))
    p.vs = np.where(r.rand(*p.vs.shape) < 0.5, top, top / 2)
    worst, ref = attention_error(p)
    assert np.all(np.isfinite(ref)) and np.any(ref != 0)
    assert worst <= 1


@pytest.mark.parametrize("fmt", list(KV))
@pytest.mark.parametrize("heads,q_heads,d,lens,news", KERNELS)
def test_attention_values_of_the_smallest_scale_appended(fmt, heads, q_heads, d, lens, news):
    """Pages whose value scale is 2^-126, the smallest that appending writes:
    the outputs are ordinary bf16 numbers of 8 significant bits."""
    p = Problem(fmt, heads, d, 32, lens, news, q_heads, seed=21)
    p.vs[:] = 2.0 ** -126
    worst, ref = attention_error(p)
    assert np.any(np.abs(ref) > 2.0 ** -124)
    assert worst <= 1


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("heads,q_heads,d,lens,news", KERNELS)
def test_attention_of_a_query_that_is_not_finite(heads, q_heads, d, lens, news, bad):
    """It gives NaN, not zeros, for its own token and head, and changes no
    other output."""
    p = Problem("int8", heads, d, 32, lens, news, q_heads, seed=23)
    clean = w4.kv8_attention(p.part(0, q_heads), p.cache(), *p.batch())
    q = p.part(0, q_heads).clone()
    token, head = int(p.starts[1]) - 1, q_heads - 1
    q[token, head, 5] = bad
    got = w4.kv8_attention(q, p.cache(), *p.batch())
    torch.cuda.synchronize()
    assert bool(torch.isnan(got[token, head]).all())
    got[token, head] = clean[token, head]
    assert torch.equal(got, clean)


@pytest.mark.parametrize("fmt", list(KV))
@pytest.mark.parametrize("heads,q_heads,d,lens,news", KERNELS)
def test_attention_value_scales_under_the_smallest_normal(fmt, heads, q_heads, d, lens, news):
    """Value scales that another quantizer left under 2^-126: 1 / scale is no
    binary32 number, but the outputs are ordinary bf16 subnormals."""
    p = Problem(fmt, heads, d, 32, lens, news, q_heads, seed=22)
    p.vs[:] = float(np.float32(2.0 ** -131))
    worst, ref = attention_error(p)
    assert np.any(np.abs(ref) > 2.0 ** -130)
    assert worst <= 1


@pytest.mark.parametrize("fmt", list(KV))
@pytest.mark.parametrize("heads,q_heads,d,lens,news", KERNELS)
@pytest.mark.parametrize("exponent", [10, 20, 30])
def test_attention_beside_a_page_of_far_larger_value_scale(fmt, heads, q_heads, d, lens, news, exponent):
    """A page that is hardly attended but whose value scale is 2^10 to 2^30
    times the others': the outputs stay within the stated bound, whose term
    n 2^-34 V is then the larger one."""
    p = Problem(fmt, heads, d, 32, lens, news, q_heads, seed=24)
    p.qkv[:, : q_heads * d] = p.qkv[:, : q_heads * d].abs() * 4
    low = {"int8": 0x84, "e4m3": 0xFA}[fmt]  # -124, -320
    for b in range(len(lens)):
        p.kc[p.table[b, 0]] = low
        p.ks[p.table[b, 0]] = p.ks.max()
        p.vs[p.table[b, 0]] = p.vs.max()
    for b in range(len(lens)):
        p.vs[p.table[b, 0]] *= 2.0 ** exponent
    worst, _ = attention_error(p)
    assert worst <= 1


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("side", ["ks", "vs"])
@pytest.mark.parametrize("heads,q_heads,d,lens,news", KERNELS)
def test_attention_keeps_a_spoilt_page_to_its_sequence_and_head(heads, q_heads, d, lens, news, side, bad):
    """A page of one kv head whose scale is not finite, as appending an infinity
    leaves it: the other heads' and sequences' outputs keep their bits."""
    lens, news = (list(lens) + [150])[:2], (list(news) + [100])[:2]
    p = Problem("e4m3", heads, d, 32, lens, news, q_heads, seed=25)
    clean = w4.kv8_attention(p.part(0, q_heads), p.cache(), *p.batch())
    getattr(p, side)[p.table[0, 1], heads - 1] = bad
    got = w4.kv8_attention(p.part(0, q_heads), p.cache(), *p.batch())
    group, rows = q_heads // heads, int(p.starts[1])
    assert torch.equal(got[rows:], clean[rows:])
    assert torch.equal(got[:rows, : q_heads - group], clean[:rows, : q_heads - group])
    # the last token sees the page
    assert bool(torch.isnan(got[rows - 1, q_heads - group:]).all())


LONG_CONTEXTS = [  # heads, q_heads, d, page, lens, news
    (1, 1, 64, 16, [3000], [1]), (8, 16, 128, 64, [9000], [1]), (8, 16, 64, 32, [32768], [1]),
    (2, 8, 128, 128, [32768], [1]), (1, 4, 128, 128, [70000], [1]), (1, 1, 64, 64, [70001], [1]),
    (2, 4, 128, 16, [9000, 70, 1], [1, 1, 1]), (4, 4, 64, 32, [64, 17, 20000, 0], [1, 1, 1, 0]),
    (2, 8, 128, 64, [9000, 700], [9, 1]), (4, 16, 64, 64, [40, 12345], [9, 12]),
    (16, 16, 128, 64, [5000, 31], [1, 1])]


@pytest.mark.parametrize("fmt", list(KV))
@pytest.mark.parametrize("heads,q_heads,d,page,lens,news", LONG_CONTEXTS)
def test_attention_over_long_contexts(fmt, heads, q_heads, d, page, lens, news):
    """Few problems and many key tiles: clusters of up to 16 CTAs (more than 8
    are not portable sizes), CTAs of twelve warps, several tiles for each warp;
    short and empty sequences beside a long one, whose clusters have CTAs
    without a tile."""
    p = Problem(fmt, heads, d, page, lens, news, q_heads, seed=sum(lens) + d, pad_rows=1)
    p.check_attention()
    p.ks = p.ks * 4
    p.vs = p.vs * 2.0 ** np.random.RandomState(d).randint(-4, 5, p.vs.shape)
    p.check_attention()


@pytest.mark.parametrize("fmt", list(KV))
@pytest.mark.parametrize("batch,heads,q_heads,d,page", [(64, 8, 16, 128, 64), (32, 4, 4, 64, 16),
                                                        (8, 8, 16, 64, 64)])
def test_append_and_attention_without_a_pause(fmt, batch, heads, q_heads, d, page):
    """Steps whose appends change the scale of every page, each kernel started
    while the one before it runs: the same bits as with a wait between them."""
    g = torch.Generator().manual_seed(batch)
    table = torch.randperm(3 * batch, generator=g).int().view(batch, 3).to(DEV)
    have, steps = page - 9, 6
    first = torch.randn(batch * have, heads, d, generator=g).to(torch.bfloat16).to(DEV) * 0.01
    new = [(torch.randn(batch, heads, d, generator=g) * 0.01 * 1.7 ** (i + 1)).to(torch.bfloat16).to(DEV)
           for i in range(steps)]
    q = torch.randn(batch, q_heads, d, generator=g).to(torch.bfloat16).to(DEV)
    lens = [torch.full((batch,), have + i, dtype=torch.int32, device=DEV) for i in range(steps + 1)]
    starts = torch.arange(0, batch * have + 1, have, dtype=torch.int32, device=DEV)
    empty = w4.kv8_cache(3 * batch, heads, page, d, KV[fmt], DEV)
    w4.kv8_append(empty, first, first, table, lens[0], starts, have)

    def run(cache, pause):
        for a, b in zip(cache, empty):
            a.copy_(b)
        out = []
        for i in range(steps):
            w4.kv8_append(cache, new[i], new[i], table, lens[i + 1])
            pause()
            out.append(w4.kv8_attention(q, cache, table, lens[i + 1]))
            pause()
        return out

    calm, busy = (w4.KV8Cache(*[torch.empty_like(t) for t in empty]) for _ in range(2))
    want = run(calm, torch.cuda.synchronize)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        got = run(busy, lambda: None)
    for _ in range(20):
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))
        assert all(torch.equal(a.view(torch.uint8), b.view(torch.uint8)) for a, b in zip(busy, calm))


@pytest.mark.parametrize("d", [64, 128])
def test_tensor_core_kernels_on_two_streams(d):
    """The kernels that allocate tensor memory at the same time: prompt
    attention on one stream, the 4-bit linear's two kernels and the int4
    prefill on another, with the bits of calls that have the GPU to
    themselves."""
    p = Problem("int8", 24, d, 32, [600, 333], [600, 300], 48, seed=26)
    cache, q, batch = p.cache(), p.part(0, 48), p.batch()
    linears = []
    for m, n, k, fmt in ((5, 2048, 2048, "mx"), (100, 1024, 2048, "nv"), (700, 2048, 1024, "nv")):
        w = w4.fp4_quantize(synth.normal_weight(n, k, 0.02, seed=m).to(DEV), fmt)
        linears.append((synth.normal_activations(m, k, seed=n).to(DEV), w, fmt))
    packed = w4.quantize_pack(synth.normal_weight(2048, 1024, 0.02, seed=8).to(DEV), False)
    x = synth.normal_activations(300, 1024, seed=9).to(DEV)

    def attend():
        return [w4.kv8_attention(q, cache, *batch)]

    def multiply():
        return [w4.fp4_linear(*w4.fp4_quantize(a, fmt), *w, fmt) for a, w, fmt in linears] + \
            [w4.w4a16_linear(x, *packed, flags=w4.LINEAR_FORCE_GEMM | w4.LINEAR_PDL)]

    work = [(torch.cuda.Stream(DEV), attend), (torch.cuda.Stream(DEV), multiply)]
    want = [f() for _, f in work]
    torch.cuda.synchronize()
    got = [[], []]
    for _ in range(15):
        for (stream, f), g in zip(work, got):
            with torch.cuda.stream(stream):
                g.append(f())
    torch.cuda.synchronize()
    for w, runs in zip(want, got):
        assert all(torch.equal(a, b) for r in runs for a, b in zip(r, w))


# ------------------------------------------------------------ long predecessors ----

@pytest.fixture(scope="module")
def slow_kernel():
    """A call whose kernel runs for longer than a wait's limit of one second
    on 60 SMs and lets its dependents start at once: attention over a long
    sequence whose pages are all the same one."""
    heads, page, d = 60, 128, 64
    cache = w4.kv8_cache(1, heads, page, d, device=DEV)
    q = torch.randn(128, heads, d, generator=torch.Generator().manual_seed(1)).to(torch.bfloat16).to(DEV)
    starts = torch.tensor([0, 128], dtype=torch.int32, device=DEV)

    def call(pages):
        table = torch.zeros(1, pages, dtype=torch.int32, device=DEV)
        lens = torch.tensor([pages * page], dtype=torch.int32, device=DEV)
        out = torch.empty_like(q)
        a, b = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)

        def run(dependents=lambda: None):
            a.record()
            w4.kv8_attention(q, cache, table, lens, starts, 128, out=out)
            got = dependents()
            b.record()
            torch.cuda.synchronize()
            return a.elapsed_time(b) / 1e3, got
        return run

    call(16384)()
    seconds, _ = call(16384)()
    return call(min(2 ** 23, int(16384 * 1.6 / seconds)))


@pytest.mark.parametrize("fmt", ["mx", "nv"])
@pytest.mark.parametrize("flags", [0, w4.LINEAR_STATIC_WEIGHTS])
def test_linear_waits_for_a_long_predecessor(slow_kernel, fmt, flags):
    """The linear is resident while the kernel in front of it runs, and its
    waits' limit does not count that time."""
    calls = []
    for m, n, k in ((5, 256, 2048), (300, 512, 1024)):
        w = w4.fp4_quantize(synth.normal_weight(n, k, 0.02, seed=n).to(DEV), fmt)
        x = w4.fp4_quantize(synth.normal_activations(m, k, seed=m).to(DEV), fmt)
        calls.append((*x, *w, fmt, flags))
    want = [w4.fp4_linear(*c) for c in calls]
    seconds, got = slow_kernel(lambda: [w4.fp4_linear(*c) for c in calls])
    assert seconds > 1.05
    assert w4.device_error(clear=True) == 0
    for a, b in zip(got, want):
        assert torch.equal(a, b)


@pytest.mark.parametrize("symmetric", [True, False])
@pytest.mark.parametrize("flags", [w4.LINEAR_PDL, w4.LINEAR_PDL | w4.LINEAR_STATIC_WEIGHTS])
def test_int4_linear_waits_for_a_long_predecessor(slow_kernel, symmetric, flags):
    """The same for the int4 linear's programmatic dependent launches: prefill
    (its K has more stages than its ring) and both decode kernels."""
    w = w4.quantize_pack(synth.normal_weight(256, 2048, 0.02, seed=3).to(DEV), symmetric)
    calls = []
    for m, kind in ((64, w4.LINEAR_FORCE_GEMM), (4, w4.LINEAR_DECODE_STREAM),
                    (4, w4.LINEAR_DECODE_TILED)):
        calls.append((synth.normal_activations(m, 2048, seed=m).to(DEV), *w, flags | kind))
    want = [w4.w4a16_linear(*c) for c in calls]
    for c, y in zip(calls, want):
        seconds, got = slow_kernel(lambda: w4.w4a16_linear(*c))
        assert seconds > 1.05
        assert w4.device_error(clear=True) == 0
        assert torch.equal(got, y)
