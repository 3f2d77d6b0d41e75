"""8-bit quantisation and products against float64.

Codes and scales are exact, and so are products of them; a product's sum is fp32.  An
fp32 addition that rounds, or cuts off, loses less than 2^-23 of its result, which no
partial sum has above S = sum |x w|: K additions lose less than K 2^-23 S.  A bf16
result is off by 2^-8 of itself more.  Where the values are small whole numbers
times powers of two that fp32 adds up exactly, results have to be equal.
"""
import numpy as np
import pytest
import torch

from host_latent_cache_gb300 import ess
from oracle import row_cache as R

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from host_latent_cache_gb300 import build as B
    B.build()
    assert torch.cuda.is_available()
    ess.load()


@pytest.fixture()
def P():
    from host_latent_cache_gb300 import products
    return products


# ------------------------------------------------------------------ quantisation

def bf16(x):
    return torch.from_numpy(np.asarray(x, dtype=np.float32)).to(torch.bfloat16)


def code_values(codes):
    raw = codes.view(torch.uint8).cpu().numpy().astype(np.int64)
    full = np.concatenate([R.E4M3, [np.nan]])
    return full[raw & 127] * np.where(raw & 128, -1.0, 1.0)


def want_quant(x, square):
    """(values of the codes / scale, scales) of float64 x."""
    n, dim = x.shape
    high = 128 if square else 1
    pad = np.pad(np.abs(x), ((0, -n % high), (0, -dim % 128)))
    amax = pad.reshape(-(-n // high), high, -1, 128).max(axis=(1, 3)).astype(np.float32)
    e = np.maximum(R.power_at_least(amax / np.float32(448.0)), -126)
    scale = 2.0 ** e
    full = np.repeat(np.repeat(scale, high, axis=0)[:n], 128, axis=1)[:, :dim]
    return np.sign(x) * R.E4M3[R.nearest_code(np.abs(x) / full, R.E4M3)], scale


@pytest.mark.parametrize("square", [False, True])
@pytest.mark.parametrize("n,dim", [(1, 8), (3, 120), (5, 128), (130, 136), (257, 4096), (1, 16384),
                                   (1000, 128), (700, 264), (128, 384)])
def test_quant(P, n, dim, square):
    rng = np.random.default_rng(n * 7 + dim + square)
    x = bf16(rng.normal(size=(n, dim)) * 2.0 ** rng.integers(-20, 20, size=(n, 1)))
    x[n // 2, : dim // 2] = 0
    if n > 2:
        x[0] = 0
    codes, scales = P.quant_q8(x.cuda(), square=square)
    v, s = want_quant(x.float().numpy().astype(np.float64), square)
    assert np.array_equal(scales.cpu().numpy().astype(np.float64), s)
    assert np.array_equal(code_values(codes), v)


@pytest.mark.parametrize("square", [False, True])
def test_quant_of_a_view_and_of_far_values(P, square):
    rng = np.random.default_rng(5)
    wide = bf16(rng.normal(size=(40, 320)) * 2.0 ** rng.integers(-100, 100, size=(40, 320)))
    wide[3, 70] = float("inf")
    wide[4, 70] = float("-inf")
    wide[5, 70] = float("nan")
    wide[6, 64:200] = 2.0 ** -133       # subnormal in bf16
    x = wide.cuda()[:, 64:264]
    codes, scales = P.quant_q8(x, square=square)
    xs = wide[:, 64:264].float().numpy().astype(np.float64)
    got, sc = code_values(codes), scales.cpu().numpy().astype(np.float64)
    if square:   # an infinity anywhere in the block: scale 1
        assert sc[0, 0] == 1.0
        fine = np.isfinite(xs[:, :128])
        v = np.clip(xs[:, :128], -448, 448)
        v = np.sign(v) * R.E4M3[R.nearest_code(np.abs(np.where(fine, v, 0)), R.E4M3)]
        assert np.array_equal(got[:, :128][fine], v[fine])
    else:
        assert sc[3, 0] == sc[4, 0] == 1.0 and sc[6, 0] == 2.0 ** -126
        rows = [i for i in range(40) if i not in (3, 4, 5)]
        v, s = want_quant(xs[rows], False)
        assert np.array_equal(sc[rows], s) and np.array_equal(got[rows], v)
    assert got[3, 6] == 448 and got[4, 6] == -448 and np.isnan(got[5, 6])


def test_quant_is_what_the_norm_gives(P):
    """norm_q8 of rows whose norm is 1 quantises the same values."""
    from host_latent_cache_gb300.rows import norm_q8
    rng = np.random.default_rng(8)
    x = bf16(np.sign(rng.normal(size=(9, 256)))).cuda()
    gamma = bf16(rng.normal(size=256)).cuda()
    a, b, _ = norm_q8(x, gamma, 0.0)
    c, d = P.quant_q8((x.float() * gamma.float()).to(torch.bfloat16))
    assert torch.equal(a.view(torch.uint8), c.view(torch.uint8)) and torch.equal(b, d)


def test_quant_refusals(P):
    x = torch.zeros(4, 256, dtype=torch.bfloat16, device="cuda")
    for bad in (x.float(), x.cpu(), x[0], x.t(), None):
        with pytest.raises(ValueError):
            P.quant_q8(bad)
    for kw in (dict(codes=torch.empty(4, 256, device="cuda")), dict(scales=torch.empty(4, 3, device="cuda"))):
        with pytest.raises(ValueError):
            P.quant_q8(x, **kw)
    with pytest.raises(RuntimeError):
        P.quant_q8(x[:, :12].contiguous())          # not a multiple of 8
    with pytest.raises(RuntimeError):
        P.quant_q8(torch.zeros(4, 257, dtype=torch.bfloat16, device="cuda")[:, 1:])   # misaligned
    codes, scales = P.quant_q8(x[:0])
    assert codes.shape == (0, 256) and scales.shape == (0, 2)


# ------------------------------------------------------------------ products

def whole(rng, n, dim):
    """Codes that are whole numbers from -3 to 3, as float64 and e4m3."""
    v = rng.integers(-3, 4, size=(n, dim)).astype(np.float64)
    return v, torch.from_numpy(v.astype(np.float32)).to(E4M3)


def scales_of(rng, shape, lo, hi):
    s = 2.0 ** rng.integers(lo, hi + 1, size=shape)
    return s, torch.from_numpy(s.astype(np.float32))


def spread(s, high, n, dim):
    return np.repeat(np.repeat(s, high, axis=0)[:n], 128, axis=1)[:, :dim]


SHAPES = [(1, 16, 1), (2, 128, 128), (4, 4096, 1600), (16, 4096, 257), (17, 48, 129), (32, 1024, 2432),
          (33, 528, 640), (64, 640, 300), (65, 1040, 257), (128, 2048, 512), (129, 256, 300),
          (333, 4112, 1601), (300, 528, 9800), (257, 128, 9801), (600, 1040, 5000), (1000, 16, 2500),
          (513, 4096, 4096), (65, 528, 4000), (200, 1040, 4100), (1024, 272, 1601), (256, 4096, 9728)]


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n,ins,outs", SHAPES)
def test_products_of_whole_numbers_are_exact(P, n, ins, outs, dtype):
    rng = np.random.default_rng(n + ins + outs)
    g = -(-ins // 128)
    x, xc = whole(rng, n, ins)
    w, wc = whole(rng, outs, ins)
    # |x w| <= 9 * 2^4 in steps of 2^-4: 4112 of them stay below 2^24 steps
    xs, xsd = scales_of(rng, (n, g), -2, 2)
    ws, wsd = scales_of(rng, (-(-outs // 128), g), -2, 2)
    weight = P.Weight8(wc.cuda(), wsd.cuda())
    got = weight.product(xc.cuda(), xsd.cuda(), dtype=dtype)
    assert weight.poll() == ess.ESS_OK
    want = (x * spread(xs, 1, n, ins)) @ (w * spread(ws, 128, outs, ins)).T
    assert np.abs(want).max() < 2 ** 19
    want = torch.from_numpy(want.astype(np.float32)).to(dtype)
    assert torch.equal(got.cpu(), want)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("tiles", [30, 37, 45, 57, 73, 90, 140, 300])
@pytest.mark.parametrize("n", [15, 16, 31, 64])
def test_k_in_any_number_of_parts(P, n, tiles, dtype):
    """From eight parts to one, as there are more tiles; each CTA's sums have their place."""
    rng = np.random.default_rng(n + tiles)
    ins, outs = 2048, 128 * tiles - 3
    x, xc = whole(rng, n, ins)
    w, wc = whole(rng, outs, ins)
    ws, wsd = scales_of(rng, (tiles, 16), -2, 2)
    xs, xsd = scales_of(rng, (n, 16), -2, 2)
    weight = P.Weight8(wc.cuda(), wsd.cuda())
    got = [weight.product(xc.cuda(), xsd.cuda(), dtype=dtype) for _ in range(3)]
    assert weight.poll() == ess.ESS_OK
    want = (x * spread(xs, 1, n, ins)) @ (w * spread(ws, 128, outs, ins)).T
    want = torch.from_numpy(want.astype(np.float32)).to(dtype)
    assert all(torch.equal(g.cpu(), want) for g in got)


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n,ins,outs", [(3, 4096, 300), (40, 16384, 200), (200, 2064, 700), (400, 1024, 5000),
                                        (9, 144, 70), (70, 16384, 4100), (300, 4112, 9800)])
def test_products_of_quantised_values(P, n, ins, outs, dtype):
    rng = np.random.default_rng(n)
    x = bf16(rng.normal(size=(n, ins)) * 2.0 ** rng.integers(-6, 6, size=(n, 1)))
    w = bf16(rng.normal(size=(outs, ins)) * 2.0 ** rng.integers(-6, 6, size=(outs, 1)))
    codes, scales = P.quant_q8(x.cuda())
    weight = P.Weight8.of(w.cuda())
    got = weight.product(codes, scales, dtype=dtype)
    assert weight.poll() == ess.ESS_OK
    xv = code_values(codes) * spread(scales.cpu().numpy().astype(np.float64), 1, n, ins)
    wv = code_values(weight.codes) * spread(weight.scales.cpu().numpy().astype(np.float64), 128, outs, ins)
    want, size = xv @ wv.T, np.abs(xv) @ np.abs(wv).T
    tol = ins * 2.0 ** -23 * size
    if dtype is torch.bfloat16:
        tol = tol + 2.0 ** -8 * np.abs(want)
    err = np.abs(got.double().cpu().numpy() - want)
    assert (err <= tol).all(), float((err / tol).max())
    if dtype is torch.float32:   # sums of 1024 products a time: see the header
        assert np.linalg.norm(err) <= 2e-6 * np.linalg.norm(want)


@pytest.mark.parametrize("n,outs", [(5, 200), (200, 200), (300, 9800), (100, 4200)])
def test_a_nan_code_reaches_its_row_and_column_only(P, n, outs):
    rng = np.random.default_rng(n)
    _, xc = whole(rng, n, 256)
    _, wc = whole(rng, outs, 256)
    xc.view(torch.uint8)[n // 2, 255] = 0x7F
    wc.view(torch.uint8)[outs - 1, 0] = 0xFF
    one = lambda r: torch.ones(r, 2, device="cuda")
    got = P.Weight8(wc.cuda(), one(-(-outs // 128))).product(xc.cuda(), one(n)).cpu()
    nan = torch.isnan(got)
    want = torch.zeros_like(nan)
    want[n // 2] = True
    want[:, outs - 1] = True
    assert torch.equal(nan, want)


@pytest.mark.parametrize("n", [3, 100, 300])
def test_scales_at_both_ends(P, n):
    outs = 9800 if n == 300 else 130
    xc = torch.ones(n, 256).to(E4M3).cuda()
    wc = torch.ones(outs, 256).to(E4M3).cuda()
    xs = torch.tensor([2.0 ** -126, 2.0 ** 127]).repeat(n, 1).cuda()
    ws = torch.tensor([2.0 ** 120, 2.0 ** -125]).repeat(-(-outs // 128), 1).cuda()
    weight = P.Weight8(wc, ws)
    got = weight.product(xc, xs, dtype=torch.float32)
    assert weight.poll() == ess.ESS_OK
    assert (got == 128 * (2.0 ** -6 + 4)).all()


@pytest.mark.parametrize("where", ["x", "w"])
@pytest.mark.parametrize("n", [1, 70, 300])
@pytest.mark.parametrize("scale", [1.5, -1.0, 0.0, float("inf"), float("nan"), 2.0 ** -130])
def test_other_scales_are_reported(P, n, where, scale):
    outs = 9800 if n == 300 else 130
    xc, wc = torch.ones(n, 640).to(E4M3).cuda(), torch.ones(outs, 640).to(E4M3).cuda()
    xs, ws = torch.ones(n, 5, device="cuda"), torch.ones(-(-outs // 128), 5, device="cuda")
    (xs if where == "x" else ws)[-1, 4] = scale
    weight = P.Weight8(wc, ws)
    got = weight.product(xc, xs, dtype=torch.float32)
    assert weight.poll() == ess.ESS_ERR_DEVICE_CHECK
    assert weight.poll() == ess.ESS_OK
    if abs(scale) in (1.5, 1.0):   # the exponent alone
        assert (got == 640).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n,outs,stride,first", [(7, 130, 576, 3), (300, 200, 209, 1), (300, 9800, 9808, 8),
                                                 (300, 9800, 9801, 1), (300, 9795, 10000, 16), (40, 64, 64, 0),
                                                 (100, 4200, 4208, 8), (100, 4196, 4200, 4), (100, 4198, 4201, 2)])
def test_into_a_view(P, n, outs, stride, first, dtype):
    rng = np.random.default_rng(n + outs)
    x, xc = whole(rng, n, 272)
    w, wc = whole(rng, outs, 272)
    weight = P.Weight8(wc.cuda(), torch.ones(-(-outs // 128), 3, device="cuda"))
    buf = torch.full((n * stride + outs + first,), 7.0, dtype=dtype, device="cuda")
    view = buf[first:first + n * stride].view(n, stride)[:, :outs]
    out = weight.product(xc.cuda(), torch.ones(n, 3, device="cuda"), out=view)
    assert out is view
    want = torch.from_numpy((x @ w.T).astype(np.float32)).to(dtype)
    assert torch.equal(view.cpu(), want)
    view.fill_(7.0)
    assert (buf == 7.0).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("stride", [33000, 33001])
def test_offsets_past_32_bits(P, stride, dtype):
    """Values, codes and results whose places pass 2^31 elements."""
    n, outs, ins = 66000, 32993, 16
    rng = np.random.default_rng(3)
    x, xc = whole(rng, n, ins)
    w, wc = whole(rng, outs, ins)
    one = lambda r: torch.ones(r, 1, device="cuda")
    weight = P.Weight8(wc.cuda(), one(-(-outs // 128)))
    out = torch.full((n, stride), 7.0, dtype=dtype, device="cuda")
    weight.product(xc.cuda(), one(n), out=out[:, :outs])
    assert weight.poll() == ess.ESS_OK
    assert (out[:, outs:] == 7.0).all()
    for rows in (slice(0, 70), slice(n // 2, n // 2 + 70), slice(n - 70, n)):
        want = torch.from_numpy((x[rows] @ w.T).astype(np.float32)).to(dtype)
        assert torch.equal(out[rows, :outs].cpu(), want)
    if dtype is torch.bfloat16 and stride == 33000:
        wide = out[:, :outs - outs % 8]          # large values, in a view of wide rows
        for square in (False, True):
            codes, scales = P.quant_q8(wide, square=square)
            at = n - n % 128 - 256               # whole blocks near the end
            c, s = P.quant_q8(wide[at:].contiguous(), square=square)
            assert torch.equal(codes[at:].view(torch.uint8), c.view(torch.uint8))
            assert torch.equal(scales[at // 128 if square else at:], s)
            del codes, scales


def test_a_product_repeats_its_bits(P):
    x = torch.randn(70, 4096, device="cuda").to(torch.bfloat16)
    weight = P.Weight8.of(torch.randn(700, 4096, device="cuda").to(torch.bfloat16))
    codes, scales = P.quant_q8(x)
    for dtype in (torch.bfloat16, torch.float32):
        first = weight.product(codes, scales, dtype=dtype)
        assert all(torch.equal(first, weight.product(codes, scales, dtype=dtype)) for _ in range(20))


def test_streams_and_graphs(P):
    """Products on two streams at once, and captured ones replayed on changed inputs, are
    the eager ones."""
    w = torch.randn(10000, 1024, device="cuda").to(torch.bfloat16)
    weights = [P.Weight8.of(w), P.Weight8.of(w[:600])]
    xs = [torch.randn(n, 1024, device="cuda").to(torch.bfloat16) for n in (300, 20)]
    quant = [P.quant_q8(x) for x in xs]
    want = [weight.product(*q) for weight, q in zip(weights, quant)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = [[], []]
    for _ in range(20):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(weights[i].product(*quant[i]))
    torch.cuda.synchronize()
    assert all(torch.equal(o, want[i]) for i in range(2) for o in got[i])

    for i in range(2):
        x = xs[i].clone()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            out = weights[i].product(*P.quant_q8(x))
        for factor in (1.0, 3.0):
            x.copy_(xs[i] * factor)
            out.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(out, weights[i].product(*P.quant_q8(x)))
    assert all(weight.poll() == ess.ESS_OK for weight in weights)


def test_the_row_cache_takes_a_wide_products_columns(P):
    """A projection's result, of which the last 576 columns are cache rows, norm ahead of it."""
    from host_latent_cache_gb300.rows import RowCache, norm_q8
    rng = np.random.default_rng(1)
    h = bf16(rng.normal(size=(37, 512))).cuda()
    weight = P.Weight8.of(bf16(rng.normal(size=(1600, 512)) / 22).cuda())
    codes, scales, _ = norm_q8(h, torch.ones(512, dtype=torch.bfloat16, device="cuda"))
    out = weight.product(codes, scales)
    cache = RowCache(torch.zeros(64, 1152, dtype=torch.uint8, device="cuda"), "bf16")
    slots = torch.randperm(64, device="cuda")[:37]
    cache.write(out[:, 1024:], slots)
    assert torch.equal(cache.read(slots), out[:, 1024:])
    assert cache.poll() == ess.ESS_OK and weight.poll() == ess.ESS_OK


def test_product_refusals(P):
    codes = torch.zeros(3, 256, device="cuda").to(E4M3)
    scales = torch.ones(3, 2, device="cuda")
    good = P.Weight8(torch.zeros(130, 256, device="cuda").to(E4M3), torch.ones(2, 2, device="cuda"))
    for c, s in ((codes.float(), scales), (codes, scales[:, :1]), (codes, scales.double()), (codes.cpu(), scales),
                 (codes[:, :128].contiguous(), scales), (codes.t(), scales), (None, scales), (codes, None)):
        with pytest.raises(ValueError):
            good.product(c, s)
    for out in (torch.empty(3, 129, device="cuda"), torch.empty(3, 130, device="cuda", dtype=torch.float16),
                torch.empty(130, 3, device="cuda").t(), torch.empty(1, 130, device="cuda").expand(3, 130)):
        with pytest.raises(ValueError):
            good.product(codes, scales, out=out)
    with pytest.raises(ValueError):
        good.product(codes, scales, dtype=torch.float16)
    for c, s in ((torch.zeros(130, 264, device="cuda").to(E4M3), torch.ones(2, 3, device="cuda")),
                 (torch.zeros(130, 256, device="cuda").to(E4M3), torch.ones(2, 3, device="cuda")),
                 (torch.zeros(130, 256, device="cuda"), torch.ones(2, 2, device="cuda"))):
        with pytest.raises(ValueError):
            P.Weight8(c, s)
    assert good.product(codes[:0], scales[:0]).shape == (0, 130)
