"""Rotation of queries and cache rows by positions on one or more axes, against float64.

The sine and cosine move either value of a pair (a, b) by at most 2^-20 (|a| + |b|), the
products and their sum in fp32 by 2^-22 of that, and bf16 by 2^-8 of the result.
"""
import numpy as np
import pytest
import torch

from host_latent_cache_gb300 import ess
from oracle import row_cache as R

pytestmark = pytest.mark.gpu
FREQ = [10000.0 ** (-i / 32.0) for i in range(32)]


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from host_latent_cache_gb300 import build as B
    B.build()
    assert torch.cuda.is_available()
    ess.load()


def sections(rng, axes):
    return [int(a) for a in rng.integers(0, axes, size=32)]


def want_turned(k, pos, freq, halves, axis):
    """k float64 [n][64], pos [axes][n]."""
    per_axis = [R.rotate(k, p, freq, halves) for p in pos]
    out = np.empty_like(per_axis[0])
    for i in range(32):
        for at in ((i, i + 32) if halves else (2 * i, 2 * i + 1)):
            out[:, at] = per_axis[axis[i]][:, at]
    return out


def bound(k, want, halves):
    a = np.abs(k)
    pair = a[:, :32] + a[:, 32:] if halves else a[:, 0::2] + a[:, 1::2]
    pair = np.concatenate([pair, pair], 1) if halves else np.repeat(pair, 2, axis=1)
    return (2.0 ** -20 + 2.0 ** -22) * pair + 2.0 ** -8 * np.abs(want) + 2.0 ** -134


def positions(rng, axes, n):
    p = rng.integers(0, 200000, size=(axes, n))
    p.flat[:: 5] = rng.integers(-(1 << 31), (1 << 31), size=p.flat[:: 5].shape)
    return p.astype(np.int32)


@pytest.mark.parametrize("pairs", ["adjacent", "halves"])
@pytest.mark.parametrize("n,heads,axes", [(1, 1, 1), (3, 1, 3), (8, 128, 1), (37, 5, 2), (130, 16, 3), (5, 4, 4),
                                          (1000, 7, 3), (20000, 3, 3)])
def test_rotate(n, heads, axes, pairs):
    from host_latent_cache_gb300.rows import rotate
    rng = np.random.default_rng(n + heads)
    x = torch.from_numpy(rng.normal(size=(n, heads, 64)).astype(np.float32)).to(torch.bfloat16)
    pos, axis = positions(rng, axes, n), sections(rng, axes)
    dev = torch.from_numpy(pos).cuda()
    got = rotate(x.cuda(), dev if axes > 1 else dev[0], FREQ, pairs=pairs, axes=axis if axes > 1 else None)
    for h in (0, heads // 2, heads - 1):
        k = x[:, h].double().numpy()
        want = want_turned(k, pos, FREQ, pairs == "halves", axis if axes > 1 else [0] * 32)
        err = np.abs(got[:, h].double().cpu().numpy() - want)
        assert (err <= bound(k, want, pairs == "halves")).all()


@pytest.mark.parametrize("pairs", ["adjacent", "halves"])
def test_views_and_places(pairs):
    """Out of one view, into another, in place, and one head repeated for several."""
    from host_latent_cache_gb300.rows import rotate
    n, heads = 50, 6
    q = torch.randn(n, heads, 192, device="cuda").to(torch.bfloat16)
    pos = torch.arange(n, device="cuda", dtype=torch.int32)
    want = rotate(q[:, :, 128:].contiguous(), pos, FREQ, pairs=pairs)
    into = torch.full((n, heads, 576), 5.0, dtype=torch.bfloat16, device="cuda")
    assert rotate(q[:, :, 128:], pos, FREQ, pairs=pairs, out=into[:, :, 512:]).data_ptr() == into[:, :, 512:].data_ptr()
    assert torch.equal(into[:, :, 512:], want) and (into[:, :, :512] == 5.0).all()
    swapped = torch.zeros(heads, n, 64, dtype=torch.bfloat16, device="cuda")
    rotate(q[:, :, 128:], pos, FREQ, pairs=pairs, out=swapped.transpose(0, 1))
    assert torch.equal(swapped.transpose(0, 1), want)
    same = q.clone()
    rotate(same[:, :, 128:], pos, FREQ, pairs=pairs, out=same[:, :, 128:])
    assert torch.equal(same[:, :, 128:], want) and torch.equal(same[:, :, :128], q[:, :, :128])
    one = q[:, :1, 128:]
    assert torch.equal(rotate(one.expand(n, heads, 64), pos, FREQ, pairs=pairs),
                       rotate(one.contiguous(), pos, FREQ, pairs=pairs).expand(n, heads, 64))


def test_offsets_past_32_bits():
    from host_latent_cache_gb300.rows import rotate
    n, heads = 300000, 64
    wide = torch.zeros(n, heads, 128, dtype=torch.bfloat16, device="cuda")   # 2.4e9 values
    wide[-5:] = torch.randn(5, heads, 128, device="cuda").to(torch.bfloat16)
    pos = torch.arange(n, device="cuda", dtype=torch.int32)
    want = rotate(wide[-5:, :, 64:].contiguous(), pos[-5:].contiguous(), FREQ)
    left = wide[-5:, :, :64].clone()
    rotate(wide[:, :, 64:], pos, FREQ, out=wide[:, :, 64:])
    assert torch.equal(wide[-5:, :, 64:], want) and torch.equal(wide[-5:, :, :64], left)
    assert not wide[:-5].any()


def test_the_inverse_is_by_the_negative_frequencies():
    """To bf16's two roundings: each off by 2^-8 of a value below |(a, b)|."""
    from host_latent_cache_gb300.rows import rotate
    x = torch.randn(100, 8, 64, device="cuda").to(torch.bfloat16)
    pos = torch.arange(100, device="cuda", dtype=torch.int32) * 999
    back = rotate(rotate(x, pos, FREQ), pos, [-f for f in FREQ]).double()
    size = torch.linalg.norm(x.double().unflatten(2, (32, 2)), dim=3).repeat_interleave(2, 2)
    assert ((back - x.double()).abs() <= (3 * 2.0 ** -8 + 2.0 ** -17) * size).all()


@pytest.mark.parametrize("fmt", ["bf16", "compact", "q4"])
@pytest.mark.parametrize("pairs", ["adjacent", "halves"])
def test_cache_rows_turn_as_queries_do(fmt, pairs):
    from host_latent_cache_gb300.rows import RowCache, rotate
    rng = np.random.default_rng(3)
    n, axes = 70, 3
    kv = torch.randn(n, 600, device="cuda").to(torch.bfloat16)[:, 24:]
    pos, axis = torch.from_numpy(positions(rng, axes, n)).cuda(), sections(rng, axes)
    cache = RowCache(torch.zeros(128, ess.ess_row_bytes(["bf16", "compact", "q4"].index(fmt)), dtype=torch.uint8,
                                 device="cuda"), fmt)
    slots = torch.randperm(128, device="cuda")[:n]
    gamma = torch.rand(512, device="cuda").to(torch.bfloat16)
    cache.write(kv, slots, gamma=gamma, pos=pos, inv_freq=FREQ, pairs=pairs, axes=axis)
    got = cache.read(slots)
    turned = rotate(kv[:, None, 512:], pos, FREQ, pairs=pairs, axes=axis)[:, 0]
    assert torch.equal(got[:, 512:], turned)
    # one axis for all pairs is the plain call, bit for bit
    plain = RowCache(torch.zeros_like(cache.rows), fmt)
    plain.write(kv, slots, gamma=gamma, pos=pos[1].contiguous(), inv_freq=FREQ, pairs=pairs)
    cache.write(kv, slots, gamma=gamma, pos=pos, inv_freq=FREQ, pairs=pairs, axes=[1] * 32)
    assert torch.equal(cache.rows, plain.rows)
    assert cache.poll() == ess.ESS_OK


def test_a_replayed_rotation_follows_its_inputs():
    from host_latent_cache_gb300.rows import rotate
    x = torch.randn(30, 4, 64, device="cuda").to(torch.bfloat16)
    pos = torch.zeros(2, 30, device="cuda", dtype=torch.int32)
    axis = [0, 1] * 16
    rotate(x, pos, FREQ, axes=axis)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = rotate(x, pos, FREQ, axes=axis)
    for p in (0, 77):
        pos.fill_(p)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, rotate(x, pos, FREQ, axes=axis))
    assert not torch.equal(out, x)


def test_refusals():
    from host_latent_cache_gb300.rows import RowCache, rotate
    x = torch.zeros(4, 2, 64, dtype=torch.bfloat16, device="cuda")
    pos = torch.zeros(4, dtype=torch.int32, device="cuda")
    three = torch.zeros(3, 4, dtype=torch.int32, device="cuda")
    for args, kw in (((x.float(), pos, FREQ), {}), ((x[0], pos, FREQ), {}), ((x[:, :, :32], pos, FREQ), {}),
                     ((x, pos.long(), FREQ), {}), ((x, pos[:3], FREQ), {}), ((x, pos, FREQ[:31]), {}),
                     ((x, three, FREQ), {}), ((x, pos, FREQ), dict(axes=[0] * 32)),
                     ((x, three, FREQ), dict(axes=[0] * 31)), ((x, three, FREQ), dict(axes=[3] * 32)),
                     ((x, three, FREQ), dict(axes=[-1] * 32)), ((x, pos, FREQ), dict(pairs="thirds")),
                     ((x, pos, FREQ), dict(out=x.float())), ((x.transpose(1, 2), pos, FREQ), {})):
        with pytest.raises(ValueError):
            rotate(*args, **kw)
    with pytest.raises(RuntimeError):   # rows that overlap
        rotate(x, pos, FREQ, out=torch.zeros(1, 2, 64, dtype=torch.bfloat16, device="cuda").expand(4, 2, 64))
    with pytest.raises(RuntimeError):   # not 16-byte aligned
        rotate(torch.zeros(4, 2, 65, dtype=torch.bfloat16, device="cuda")[:, :, 1:], pos, FREQ)
    with pytest.raises(RuntimeError):
        rotate(x, pos, [float("nan")] * 32)
    assert rotate(x[:0], pos[:0], FREQ).shape == (0, 2, 64)
    cache = RowCache(torch.zeros(8, 1152, dtype=torch.uint8, device="cuda"), "bf16")
    kv, slots = torch.zeros(4, 576, dtype=torch.bfloat16, device="cuda"), torch.arange(4, device="cuda")
    with pytest.raises(ValueError):
        cache.write(kv, slots, pos=three, inv_freq=FREQ)
    with pytest.raises(ValueError):
        cache.write(kv, slots, axes=[0] * 32)
    with pytest.raises(ValueError):
        cache.write(kv, slots, pos=three, inv_freq=FREQ, axes=[5] * 32)
