"""The device row cache's writes and reads, and the 8-bit norm, against float64.

Tolerances count the roundings of the definitions.  y goes through three fp32
roundings (r, x * r, * gamma), at most 3 * 2^-24 relative with r itself within
2^-24 of its root: 2^-22.  A bf16 output adds half a step, 2^-8 of the value.  A
code is the nearest level of a value that far off: it lies within half of the
gap between the levels on either side, plus 2^-22 of the value.  The rotation
adds the errors of a sine and a cosine (2^-22 with the angle's) times both
values of the pair, and fp32 roundings of the two products: 2^-20 of |a| + |b|.
"""
import numpy as np
import pytest
import torch

from host_latent_cache_gb300 import ess
from host_latent_cache_gb300 import workloads as W
from oracle import compact_row as X
from oracle import row_cache as R

pytestmark = pytest.mark.gpu
Y_REL = 2.0 ** -22
BF16_HALF = 2.0 ** -8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from host_latent_cache_gb300 import build as B
    B.build()
    assert torch.cuda.is_available()
    ess.load()


def rows_mod():
    from host_latent_cache_gb300 import rows
    return rows


def f64(t):
    return t.detach().float().cpu().numpy().astype(np.float64)


FREQ = [10000.0 ** (-i / 32.0) for i in range(32)]


def check_codes(values, scale, y, levels):
    """values = code * scale is a nearest level of y within Y_REL of it."""
    u, a = np.abs(values) / scale, np.abs(y) / scale
    i = np.searchsorted(levels, u)
    assert np.array_equal(levels[np.minimum(i, len(levels) - 1)], u), "not a level of the format"
    up = levels[np.minimum(i + 1, len(levels) - 1)] - u
    down = u - levels[np.maximum(i - 1, 0)]
    slack = Y_REL * a + 1e-300
    ok = np.where(a >= u, (a - u <= up / 2 + slack) | (i == len(levels) - 1),
                  u - a <= down / 2 + slack)
    assert ok.all(), f"{(~ok).sum()} codes are not the nearest"
    same = np.sign(values) == np.sign(y)
    assert (same | (values == 0)).all()


def check_scales(exps, y, size, top, lo=-126, hi=126):
    want = np.clip(R.block_exps(y, size, top), lo, hi)
    off = exps != want
    if off.any():   # only next to a power of two, where Y_REL decides
        pad = -(-y.shape[1] // size) * size - y.shape[1]
        a = np.abs(np.pad(y, ((0, 0), (0, pad)))).reshape(y.shape[0], -1, size).max(2)[off] / top
        near = np.abs(a / 2.0 ** np.round(np.log2(a)) - 1.0)
        assert (near <= 2 * Y_REL).all() and (np.abs(exps - want)[off] == 1).all()


def check_rows(got, fmt, y, rope, rope_tol):
    v = R.row_values(got, fmt)
    assert (np.abs(v[:, 512:] - rope) <= rope_tol).all(), np.abs(v[:, 512:] - rope).max()
    if fmt == "bf16":
        assert (np.abs(v[:, :512] - y) <= (BF16_HALF + Y_REL) * np.abs(y)).all()
    elif fmt == "compact":
        scale = np.ascontiguousarray(got[:, 512:528]).view(np.float32).astype(np.float64)
        check_scales(np.log2(scale).astype(np.int64), y, 128, 448.0)
        check_codes(v[:, :512], np.repeat(scale, 128, axis=1), y, R.E4M3)
    else:
        e = got[:, 256:272].astype(np.int64) - 127
        check_scales(e, y, 32, 6.0, R.MIN_EXP, R.MAX_EXP)
        check_codes(v[:, :512], np.repeat(2.0 ** e, 32, axis=1), y, R.E2M1)


def make_rows(n, g, stride=576, scale=1.0):
    x = (scale * torch.randn(n, stride, generator=g, device="cuda")).to(torch.bfloat16)
    return x[:, stride - 576:]


@pytest.mark.parametrize("fmt", ["bf16", "compact", "q4"])
@pytest.mark.parametrize("n,stride,norm,rope", [
    (1, 576, True, "adjacent"), (7, 576, True, "halves"), (8, 584, False, "adjacent"),
    (65, 1600, True, None), (333, 2176, False, None), (2050, 640, True, "halves"),
], ids=lambda v: str(v))
def test_write(fmt, n, stride, norm, rope):
    rows = rows_mod()
    g = torch.Generator(device="cuda").manual_seed(n * 7 + stride)
    kv = make_rows(n, g, stride, scale=0.7)
    total = n + 70
    cache_rows = torch.full((total, R.ROW_BYTES[fmt]), 0xA5, dtype=torch.uint8, device="cuda")
    cache = rows.RowCache(cache_rows, fmt)
    slots = torch.randperm(total, generator=g, device="cuda")[:n].contiguous()
    if n > 5:
        slots[n // 2] = -1
        slots[3] = -(1 << 40)
    gamma = (0.5 + torch.rand(512, generator=g, device="cuda")).to(torch.bfloat16) if norm else None
    pos = torch.randint(0, 1 << 20, (n,), generator=g, device="cuda", dtype=torch.int32)
    cache.write(kv, slots, gamma=gamma, eps=1e-5, pos=pos if rope else None,
                inv_freq=FREQ if rope else None, pairs=rope or "adjacent")
    assert cache.poll() == ess.ESS_OK
    x = f64(kv)
    y = R.rms_norm(x[:, :512], f64(gamma), 1e-5) if norm else x[:, :512]
    k = x[:, 512:]
    if rope:
        k2 = R.rotate(k, pos.cpu().numpy(), FREQ, rope == "halves")
        other = np.abs(np.roll(k, 32, axis=1)) if rope == "halves" else \
            np.abs(k.reshape(n, 32, 2)[:, :, ::-1].reshape(n, 64))
        tol = BF16_HALF * np.abs(k2) + 2.0 ** -20 * (np.abs(k) + other)
    else:
        k2, tol = k, np.zeros_like(k)
    s = slots.cpu().numpy()
    keep = s >= 0
    got = cache_rows.cpu().numpy()
    check_rows(got[s[keep]], fmt, y[keep], k2[keep], tol[keep])
    rest = np.ones(total, bool)
    rest[s[keep]] = False
    assert (got[rest] == 0xA5).all(), "a row that no token names was changed"


def test_frequencies_that_change_in_place():
    rows = rows_mod()
    g = torch.Generator(device="cuda").manual_seed(31)
    kv, slots = make_rows(4, g), torch.arange(4, device="cuda")
    pos = torch.arange(1, 5, dtype=torch.int32, device="cuda")
    freq = torch.tensor(FREQ, dtype=torch.float64)
    cache = rows.RowCache(torch.zeros(4, 1152, dtype=torch.uint8, device="cuda"), "bf16")
    cache.write(kv, slots, pos=pos, inv_freq=freq)
    freq *= 0.5
    cache.write(kv, slots, pos=pos, inv_freq=freq)
    got = cache.rows.clone()
    cache.write(kv, slots, pos=pos, inv_freq=[f * 0.5 for f in FREQ])
    assert torch.equal(got, cache.rows)


@pytest.mark.parametrize("pairs", ["adjacent", "halves"])
def test_angles_of_far_positions(pairs):
    """Positions up to 2^31 under frequencies up to 1000 and below 0, against angles
    reduced in 70 decimal digits.  Angles near a quarter turn make values near 0,
    where only the rotation's own error is left."""
    from decimal import Decimal, getcontext
    getcontext().prec = 70
    turn = 2 * Decimal("3.14159265358979323846264338327950288419716939937510582097494459230781640628620899")
    rows = rows_mod()
    g = torch.Generator(device="cuda").manual_seed(51)
    freq = [1000.0 ** (1 - i / 12) * (-1) ** (i % 3) for i in range(32)]
    pos = torch.cat([2 ** 31 - 1 - torch.randint(0, 1 << 20, (200,), generator=g, device="cuda"),
                     torch.randint(-2 ** 31, 2 ** 31, (200,), generator=g, device="cuda")]).int()
    kv = make_rows(400, g)
    kv[::2, 512:] = 0                    # pairs (1, 0)
    one = slice(512, 576, 2) if pairs == "adjacent" else slice(512, 544)
    kv[::2, one] = 1
    buf = torch.zeros(400, 1152, dtype=torch.uint8, device="cuda")
    rows.RowCache(buf, "bf16").write(kv, torch.arange(400, device="cuda"), pos=pos, inv_freq=freq, pairs=pairs)
    f = [Decimal(x) for x in freq]
    angle = np.array([[float((int(p) * x) % turn) for x in f] for p in pos.cpu().tolist()])
    z = np.cos(angle) + 1j * np.sin(angle)
    k = f64(kv)[:, 512:]
    a, b = (k[:, 0::2], k[:, 1::2]) if pairs == "adjacent" else (k[:, :32], k[:, 32:])
    out = (a + 1j * b) * z
    got = R.row_values(buf.cpu().numpy(), "bf16")[:, 512:]
    ga, gb = (got[:, 0::2], got[:, 1::2]) if pairs == "adjacent" else (got[:, :32], got[:, 32:])
    slack = 2.0 ** -20 * (np.abs(a) + np.abs(b))
    assert (np.abs(ga - out.real) <= BF16_HALF * np.abs(out.real) + slack).all()
    assert (np.abs(gb - out.imag) <= BF16_HALF * np.abs(out.imag) + slack).all()


def test_compact_rows_are_those_of_the_host_encoder():
    rows = rows_mod()
    g = torch.Generator(device="cuda").manual_seed(5)
    kv = make_rows(300, g, scale=2.0)
    kv[3, :128] = 0
    kv[4] = 0
    buf = torch.zeros(300, 656, dtype=torch.uint8, device="cuda")
    rows.RowCache(buf, "compact").write(kv, torch.arange(300, device="cuda"))
    want = ess.ess_compact_rows(kv.contiguous().view(torch.int16).cpu().numpy().view(np.uint16))
    assert np.array_equal(buf.cpu().numpy(), want)


def test_q4_rows_are_those_of_the_oracle():
    rows = rows_mod()
    g = torch.Generator(device="cuda").manual_seed(6)
    kv = make_rows(300, g, scale=3.0)
    kv[3, :64] = 0
    kv[4] = 0
    kv[5, 10] = 1e9          # past the largest scale: saturates
    kv[6, :512] *= 1e-7      # below the smallest scale
    kv[7, :32] = torch.tensor([6, 5, 3.5, 2.5, 1.75, 1.25, 0.75, 0.25] * 4)   # ties
    kv[8, 0], kv[8, 40] = float("inf"), float("nan")
    buf = torch.zeros(300, 400, dtype=torch.uint8, device="cuda")
    rows.RowCache(buf, "q4").write(kv, torch.arange(300, device="cuda"))
    got = buf.cpu().numpy()
    x = f64(kv)
    keep = np.arange(300) != 8
    packed, exps = R.q4_encode(x[keep, :512])
    assert np.array_equal(got[keep, :256], packed) and np.array_equal(got[keep, 256:272], exps)
    assert np.array_equal(got[:, 272:], kv[:, 512:].contiguous().view(torch.uint8).cpu().numpy())
    v = R.row_values(got[8:9], "q4")[0]
    assert v[0] == 6.0 and got[8, 256] == 127            # an infinity saturates at scale 1
    assert abs(v[40]) == 6.0 * 2.0 ** (int(got[8, 257]) - 127)


@pytest.mark.parametrize("fmt", ["bf16", "compact", "q4"])
@pytest.mark.parametrize("n", [1, 9, 1000])
def test_read(fmt, n):
    rows = rows_mod()
    rng = np.random.default_rng(n)
    total = 1500
    raw = rng.integers(0, 256, (total, R.ROW_BYTES[fmt]), dtype=np.uint8)
    rope = rng.normal(size=(total, 64)).astype(np.float32)
    tail = torch.from_numpy(rope).to(torch.bfloat16).view(torch.uint8).numpy()
    if fmt == "bf16":
        vals = torch.from_numpy(rng.normal(size=(total, 576)).astype(np.float32)).to(torch.bfloat16)
        raw = vals.view(torch.uint8).numpy().copy()
    elif fmt == "compact":
        raw[:, :512][(raw[:, :512] & 127) == 127] = 0    # no NaN codes
        raw[:, 512:528] = (2.0 ** rng.integers(-20, 20, (total, 4))).astype(np.float32).view(np.uint8)
        raw[:, 528:] = tail
    else:
        raw[:, 272:] = tail   # every exponent byte: those outside the format read as its ends
    cache = rows.RowCache(torch.from_numpy(raw).cuda(), fmt)
    slots = torch.from_numpy(rng.integers(0, total, n)).cuda()
    if n > 3:
        slots[2] = slots[1]        # the same row twice
        slots[0] = -5
    out = torch.full((n, 576), 7.0, dtype=torch.bfloat16, device="cuda")
    got = f64(cache.read(slots, out=out))
    assert cache.poll() == ess.ESS_OK
    s = slots.cpu().numpy()
    want = R.row_values(raw[np.maximum(s, 0)], fmt) * (s >= 0)[:, None]
    assert np.array_equal(got, want)


def test_slots_past_the_cache_are_reported_and_skipped():
    rows = rows_mod()
    buf = torch.full((10, 400), 3, dtype=torch.uint8, device="cuda")
    guard = buf.clone()
    cache = rows.RowCache(buf, "q4")
    kv = torch.ones(3, 576, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([10, 1 << 40, -1], device="cuda")
    cache.write(kv, slots)
    assert cache.poll() == ess.ESS_ERR_DEVICE_CHECK and cache.poll() == ess.ESS_OK
    assert torch.equal(buf, guard)
    out = cache.read(slots)
    assert cache.poll() == ess.ESS_ERR_DEVICE_CHECK
    assert not out.any()


def test_errors_on_another_stream_are_kept():
    """An error that lands while a poll on another stream runs is that poll's or the
    next one's."""
    rows = rows_mod()
    cache = rows.RowCache(torch.zeros(10, 400, dtype=torch.uint8, device="cuda"), "q4")
    kv = torch.ones(1, 576, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([99], device="cuda")
    side = torch.cuda.Stream()
    busy = torch.ones(4000, 4000, dtype=torch.bfloat16, device="cuda")
    out = busy @ busy
    torch.cuda.synchronize()
    for i in range(600):
        n = 520 + 168 * (i % 20)                    # 3 to 60 us ahead of the write
        with torch.cuda.stream(side):
            torch.mm(busy[:n, :n], busy[:n, :n], out=out[:n, :n])
            cache.write(kv, slots)
        first = cache.poll()
        side.synchronize()
        second = cache.poll()
        assert ess.ESS_ERR_DEVICE_CHECK in (first, second), i
        assert cache.poll() == ess.ESS_OK


def test_a_new_cache_may_be_used_on_any_stream():
    """The status word is clear before the constructor returns, whatever the
    stream it ran on still has to do."""
    rows = rows_mod()
    kv = torch.ones(1, 576, dtype=torch.bfloat16, device="cuda")
    slots = torch.tensor([99], device="cuda")
    buf = torch.zeros(10, 400, dtype=torch.uint8, device="cuda")
    big = torch.ones(8192, 8192, dtype=torch.bfloat16, device="cuda")
    out = big @ big
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(20):
        torch.mm(big, big, out=out)
    cache = rows.RowCache(buf, "q4")
    with torch.cuda.stream(side):
        cache.write(kv, slots)
    side.synchronize()
    torch.cuda.synchronize()
    assert cache.poll() == ess.ESS_ERR_DEVICE_CHECK


def test_offsets_past_32_bits():
    rows = rows_mod()
    n_rows = (5 << 30) // 400        # a cache of 5 GiB
    buf = torch.zeros(n_rows, 400, dtype=torch.uint8, device="cuda")
    cache = rows.RowCache(buf, "q4")
    kv = make_rows(4, torch.Generator(device="cuda").manual_seed(1))
    slots = torch.tensor([n_rows - 1, 0, (1 << 32) // 400 + 1, n_rows // 2], device="cuda")
    cache.write(kv, slots)
    got = buf[slots].cpu().numpy()
    packed, exps = R.q4_encode(f64(kv)[:, :512])
    assert np.array_equal(got[:, :256], packed) and np.array_equal(got[:, 256:272], exps)
    back = f64(cache.read(slots))
    assert np.array_equal(back, R.row_values(got, "q4"))
    assert cache.poll() == ess.ESS_OK


@pytest.mark.parametrize("dim", [8, 64, 128, 136, 256, 520, 1000, 1024, 2048, 2056, 4096, 5120, 8192,
                                 16384])
@pytest.mark.parametrize("n,res", [(1, True), (13, False), (130, True)])
def test_norm(dim, n, res):
    rows = rows_mod()
    g = torch.Generator(device="cuda").manual_seed(dim + n)
    x = torch.randn(n, dim + 8, generator=g, device="cuda").to(torch.bfloat16)[:, 8:]
    r = (2 * torch.randn(n, dim, generator=g, device="cuda")).to(torch.bfloat16) if res else None
    gamma = (0.5 + torch.rand(dim, generator=g, device="cuda")).to(torch.bfloat16)
    if n > 10:
        x[5] = 0
        if res:
            r[5] = 0
    codes, scales, out = rows.norm_q8(x, gamma, 1e-6, residual=r)
    # h is rounded to fp32 once: the oracle takes the same sum
    h = (x.float() + r.float() if res else x.float()).cpu().numpy().astype(np.float64)
    y, _ = R.norm_quant(h, f64(gamma), 1e-6)
    s = f64(scales)
    assert s.shape == (n, -(-dim // 128))
    check_scales(np.log2(s).astype(np.int64), y, 128, 448.0)
    wide = np.repeat(s, 128, axis=1)[:, :dim]
    check_codes(f64(codes) * wide, wide, y, R.E4M3)
    if res:
        assert torch.equal(out, (x.float() + r.float()).to(torch.bfloat16))
    else:
        assert out is None


def far_rows(dim, g):
    """Rows of every size that bf16 has, and rows in which a few values are far
    larger than all the others."""
    power = torch.cat([torch.arange(-120, 121, device="cuda"), torch.tensor([-30, -50, -50, 20, -60], device="cuda")])
    x = torch.randn(len(power), dim, generator=g, device="cuda", dtype=torch.float64)
    x = (x + 0.25 * x.sign()) * torch.exp2(power.double())[:, None]   # no value far below its row's
    x[-5, dim // 2] = 2.0 ** 60
    x[-4, dim - 1] = 2.0 ** 30
    x[-3, 0] = 2.0 ** 41
    x[-2, dim - 8:] *= 2.0 ** 90
    x[-1, dim // 2:] *= 2.0 ** 15
    return x.to(torch.bfloat16)


@pytest.mark.parametrize("fmt", ["bf16", "compact", "q4"])
@pytest.mark.parametrize("eps", [0.0, 1e-6, 1e-25])
def test_written_rows_of_any_size(fmt, eps):
    """As test_write: r and y are within their tolerance at every size."""
    rows = rows_mod()
    g = torch.Generator(device="cuda").manual_seed(41)
    x = far_rows(512, g)
    n = x.shape[0]
    kv = torch.zeros(n, 576, dtype=torch.bfloat16, device="cuda")
    kv[:, :512] = x
    gamma = (0.5 + torch.rand(512, generator=g, device="cuda")).to(torch.bfloat16)
    buf = torch.zeros(n, R.ROW_BYTES[fmt], dtype=torch.uint8, device="cuda")
    rows.RowCache(buf, fmt).write(kv, torch.arange(n, device="cuda"), gamma=gamma, eps=eps)
    zero = np.zeros((n, 64))
    check_rows(buf.cpu().numpy(), fmt, R.rms_norm(f64(x), f64(gamma), eps), zero, zero)


@pytest.mark.parametrize("dim", [64, 128, 256, 1000, 1024, 4096, 16384])
@pytest.mark.parametrize("eps", [0.0, 1e-6])
def test_norms_of_any_size(dim, eps):
    rows = rows_mod()
    g = torch.Generator(device="cuda").manual_seed(dim)
    x = far_rows(dim, g)
    gamma = (0.5 + torch.rand(dim, generator=g, device="cuda")).to(torch.bfloat16)
    codes, scales, _ = rows.norm_q8(x, gamma, eps)
    y, _ = R.norm_quant(f64(x), f64(gamma), eps)
    s = f64(scales)
    check_scales(np.log2(s).astype(np.int64), y, 128, 448.0)
    wide = np.repeat(s, 128, axis=1)[:, :dim]
    check_codes(f64(codes) * wide, wide, y, R.E4M3)


def test_an_infinity_and_a_nan_stay_in_their_row():
    rows = rows_mod()
    for dim in (128, 512, 4096):
        x = torch.ones(6, dim, dtype=torch.bfloat16, device="cuda")
        x[1, 5], x[2, dim - 1] = float("inf"), float("-inf")
        x[3, 7] = float("nan")
        x[4, 3], x[4, dim - 2] = float("inf"), float("nan")
        gamma = torch.ones(dim, dtype=torch.bfloat16, device="cuda")
        codes = rows.norm_q8(x, gamma)[0].float()
        assert (codes[[0, 5]] == codes[0, 0]).all() and codes[0, 0] > 0
        for i, at in ((1, 5), (2, dim - 1)):
            bad = torch.zeros(dim, dtype=torch.bool, device="cuda")
            bad[at] = True
            assert torch.isnan(codes[i][bad]).all() and (codes[i][~bad] == 0).all()
        assert torch.isnan(codes[3:5]).all()
    kv = torch.ones(3, 576, dtype=torch.bfloat16, device="cuda")
    kv[1, 100] = float("inf")
    buf = torch.zeros(3, 1152, dtype=torch.uint8, device="cuda")
    cache = rows.RowCache(buf, "bf16")
    cache.write(kv, torch.arange(3, device="cuda"), gamma=torch.ones(512, dtype=torch.bfloat16, device="cuda"))
    out = cache.read(torch.arange(3, device="cuda"))
    assert torch.isnan(out[1, 100]) and out[1].isnan().sum() == 1 and out[1, :512].nan_to_num(0).eq(0).all()
    assert out[0].eq(out[2]).all() and not out[0].isnan().any()


def test_norm_in_place_and_rows_apart():
    rows = rows_mod()
    g = torch.Generator(device="cuda").manual_seed(9)
    x = torch.randn(40, 512, generator=g, device="cuda").to(torch.bfloat16)
    r = torch.randn(40, 1024, generator=g, device="cuda").to(torch.bfloat16)
    gamma = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    want = rows.norm_q8(x, gamma, residual=r[:, :512])
    right = r[:, 512:].clone()
    got = rows.norm_q8(x, gamma, residual=r[:, :512], residual_out=r[:, :512])
    assert torch.equal(got[0].view(torch.uint8), want[0].view(torch.uint8))
    assert torch.equal(got[1], want[1])
    assert torch.equal(r[:, :512], want[2]) and torch.equal(r[:, 512:], right)
    x2 = x.clone()
    back = rows.norm_q8(x2, gamma, residual=right.contiguous(), residual_out=x2)
    assert torch.equal(back[2], x2) and torch.equal(x2, (x.float() + right.float()).bfloat16())


def test_a_captured_write_replays_on_new_inputs():
    rows = rows_mod()
    g = torch.Generator(device="cuda").manual_seed(11)
    kv = make_rows(33, g)
    slots = torch.arange(33, device="cuda")
    gamma = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    pos = torch.arange(33, device="cuda", dtype=torch.int32)
    buf = torch.zeros(64, 400, dtype=torch.uint8, device="cuda")
    cache = rows.RowCache(buf, "q4")
    out = torch.zeros(33, 576, dtype=torch.bfloat16, device="cuda")
    run = lambda: (cache.write(kv, slots, gamma=gamma, pos=pos, inv_freq=FREQ), cache.read(slots, out=out))
    run()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        run()
    for step in range(3):
        kv.copy_(make_rows(33, g))
        pos += 100
        slots.copy_((torch.arange(33, device="cuda") * 5 + step) % 64)
        graph.replay()
        torch.cuda.synchronize()
        a, b = buf.clone(), out.clone()
        run()
        assert torch.equal(a, buf) and torch.equal(b, out)
    assert cache.poll() == ess.ESS_OK


@pytest.mark.parametrize("call", [
    lambda c, r: c.write(torch.zeros(2, 576, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda")),
    lambda c, r: c.write(torch.zeros(2, 576, dtype=torch.bfloat16), torch.zeros(2, dtype=torch.int64, device="cuda")),
    lambda c, r: c.write(torch.zeros(3, 576, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda")),
    lambda c, r: c.write(torch.zeros(2, 576, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, dtype=torch.int32, device="cuda")),
    lambda c, r: c.write(torch.zeros(2, 576, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda"), inv_freq=[1.0] * 32),
    lambda c, r: c.write(torch.zeros(2, 576, dtype=torch.bfloat16, device="cuda"), torch.zeros(2, dtype=torch.int64, device="cuda"), pairs="both"),
    lambda c, r: c.write(torch.zeros(576, 2, dtype=torch.bfloat16, device="cuda").t(), torch.zeros(2, dtype=torch.int64, device="cuda")),
    lambda c, r: c.read(torch.zeros(4, dtype=torch.int64, device="cuda")[::2]),
    lambda c, r: r.RowCache(torch.zeros(4, 401, dtype=torch.uint8, device="cuda"), "q4"),
    lambda c, r: r.RowCache(torch.zeros(4, 400, dtype=torch.uint8, device="cuda"), "q5"),
    lambda c, r: r.norm_q8(torch.zeros(2, 128, device="cuda"), torch.ones(128, dtype=torch.bfloat16, device="cuda")),
    lambda c, r: r.norm_q8(torch.zeros(2, 128, dtype=torch.bfloat16, device="cuda"), torch.ones(64, dtype=torch.bfloat16, device="cuda")),
])
def test_what_the_kernels_do_not_take_is_refused(call):
    rows = rows_mod()
    cache = rows.RowCache(torch.zeros(8, 400, dtype=torch.uint8, device="cuda"), "q4")
    with pytest.raises(ValueError):
        call(cache, rows)


def test_misaligned_rows_are_refused():
    rows = rows_mod()
    cache = rows.RowCache(torch.zeros(8, 400, dtype=torch.uint8, device="cuda"), "q4")
    kv = torch.zeros(2 * 577, dtype=torch.bfloat16, device="cuda")[1:1153].view(2, 576)
    with pytest.raises(ess.EssError):
        cache.write(kv, torch.zeros(2, dtype=torch.int64, device="cuda"))
    odd = torch.zeros(2, 579, dtype=torch.bfloat16, device="cuda")[:, :576]
    with pytest.raises(ess.EssError):
        cache.write(odd, torch.zeros(2, dtype=torch.int64, device="cuda"))


@pytest.mark.parametrize("how", ["eager", "one graph", "graph of the norm", "graph of the indexer",
                                 "host step"])
def test_an_indexer_right_behind_the_norm_that_makes_its_keys(how):
    """A prompt's keys normed straight into the bound keys, and the indexer next on
    the stream: it scores those keys, as one that starts after everything is done."""
    from host_latent_cache_gb300.session import Session
    rows = rows_mod()
    cfg = W.v32_32k().replace(batch=2, T=32768, k=512, C=2048, mtp=1, mla_heads=16, layers=1)
    ld = W.gen_layer(cfg)
    sess = Session(cfg, [ld])
    keys = sess.keys[0].view(torch.uint8).view(torch.float8_e4m3fn).view(-1, 128)
    scale = sess.scale[0].view(-1, 1)
    n = keys.shape[0]
    gamma = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    g = torch.Generator(device="cuda").manual_seed(21)
    raws = [torch.randn(n, 128, generator=g, device="cuda").to(torch.bfloat16) for _ in range(4)]
    raw = torch.empty_like(raws[0])
    q, enc, qm = W.QueryStream(cfg).next()
    w = W.head_weights(cfg, ld.w)
    qd, wd, qmd = sess.device_inputs(enc, w, qm)
    norm = lambda: rows.norm_q8(raw, gamma, codes=keys, scales=scale)

    def done():                     # the scores, or the output of a step
        torch.cuda.synchronize()
        return (out if how == "host step" else sess.scores).clone()
    if how == "host step":
        host = [ess.HostBuffer(a.shape, a.dtype) for a in (enc.view(np.uint8), w, qm)]
        for h, a in zip(host, (enc.view(np.uint8), w, qm)):
            h.array[...] = a
        out_host = ess.HostBuffer((2, 1, 16, 512), np.float32)
        out = None

        def index():
            nonlocal out
            ess.ess_pool_reset(sess.pool, 0)
            torch.cuda.synchronize()
            norm()
            ess.ess_step_host(sess.pool, 0, *host, out_host)
            torch.cuda.synchronize()
            out = torch.from_numpy(out_host.array.copy())
    else:
        index = lambda: sess.scores_only(0, qd, wd)

    want = []
    for r in raws:
        raw.copy_(r)
        norm()
        torch.cuda.synchronize()
        index()
        want.append(done())
    assert not torch.equal(want[0], want[1])
    graph = torch.cuda.CUDAGraph()
    if "graph" in how:
        index()                     # one after the last norm: the next need not wait
        with torch.cuda.graph(graph):
            if how != "graph of the indexer":
                norm()
            if how != "graph of the norm":
                sess.scores_only(0, qd, wd, torch.cuda.current_stream())
        index()
    for i in range(24):
        raw.copy_(raws[i % 4])
        torch.cuda.synchronize()
        if how in ("eager", "graph of the indexer"):
            norm()
        if "graph" in how:
            graph.replay()
        if how in ("eager", "graph of the norm", "host step"):
            index()
        assert torch.equal(done(), want[i % 4]), i
    assert sess.poll() == ess.ESS_OK
    sess.close()


def test_raw_rows_through_the_norms_into_a_decode_step():
    """The producers beside the step that eats them: norm_q8 makes the indexer
    key and its scale, a bf16 cache write the latent row, ess_append takes
    both, and a step attends to them; the appended host rows equal what went in."""
    from host_latent_cache_gb300.session import Session
    rows = rows_mod()
    cfg = W.v32_32k().replace(batch=2, T=1024, k=256, C=512, mtp=1, mla_heads=16, layers=1,
                              T_per_req=[130, 959], grow=4)
    ld = W.gen_layer(cfg)
    sess = Session(cfg, [ld])
    g = torch.Generator(device="cuda").manual_seed(3)
    qs = W.QueryStream(cfg)
    gk = torch.ones(128, dtype=torch.bfloat16, device="cuda")
    gl = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    made = []
    for step in range(3):
        raw_key = torch.randn(2, 128, generator=g, device="cuda").to(torch.bfloat16)
        raw = make_rows(2, g)
        codes, scales, _ = rows.norm_q8(raw_key, gk)
        latent = torch.empty(2, 1152, dtype=torch.uint8, device="cuda")
        pos = torch.tensor([130 + step, 959 + step], dtype=torch.int32, device="cuda")
        rows.RowCache(latent, "bf16").write(raw, torch.arange(2, device="cuda"), gamma=gl, pos=pos,
                                            inv_freq=FREQ)
        sess.append(0, latent, codes, scales)
        made.append(latent.clone())
        q, enc, qm = qs.next()
        out = sess.step(0, *sess.device_inputs(enc, W.head_weights(cfg, ld.w), qm))
        torch.cuda.synchronize()
        assert sess.poll() == ess.ESS_OK
        assert torch.isfinite(out).all()
        key = sess.keys[0][1, 959 + step].view(torch.uint8)
        assert torch.equal(key, codes[1].view(torch.uint8))
        assert sess.scale[0][1, 959 + step] == scales[1, 0]
    page = int(ld.page_table[1, 959 // 64])     # token 959 completed its page
    host = sess.host[0].array.reshape(2, W.t_max_of(cfg), 576)[1, page * 64 + 63].view(np.uint16)
    assert np.array_equal(host, made[0][1].cpu().numpy().view(np.uint16))
    sess.close()
