"""Long sums of 8-bit products: bf16 results of more than 65536 values are made of short sums,
as the tensor core cuts off what it adds.

Values of one sign show it.  A short sum of 1024 values has fewer than 1024 additions that lose
less than 2^-23 of it, 2^-13 in all; the K / 1024 sums are added up with a rounding of 2^-24
each; and bf16 rounds to 2^-8 at most, either way.  The mean of m such roundings is within six
times 2^-8 / sqrt(3 m).
"""
import math

import pytest
import torch

from host_latent_cache_gb300 import ess
from host_latent_cache_gb300.products import E4M3, Weight8

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from host_latent_cache_gb300 import build as B
    B.build()


def codes_of(g, rows, ins, most):
    return torch.randint(0, most, (rows, ins), generator=g, device="cuda", dtype=torch.uint8).view(E4M3)


def product_in_64_bits(x, w):
    total = torch.zeros(x.shape[0], w.shape[0], dtype=torch.float64, device="cuda")
    for i in range(0, x.shape[1], 1 << 18):
        at = slice(i, i + (1 << 18))
        total += x[:, at].double() @ w[:, at].double().T
    return total


def ones(rows, ins):
    return torch.ones(rows, -(-ins // 128), device="cuda")


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32], ids=["bf16", "fp32"])
@pytest.mark.parametrize("n,outs,ins", [(3, 200, 1 << 22), (20, 200, 1 << 22), (60, 200, (1 << 22) + 16),
                                        (300, 4000, 1 << 17), (300, 4000, 65536 + 16), (100, 200, 1 << 20)])
def test_long_sums_of_one_sign(n, outs, ins, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    x, w = codes_of(g, n, ins, 120), codes_of(g, outs, ins, 120)
    weight = Weight8(w, ones(-(-outs // 128), ins))
    got = weight.product(x, ones(n, ins), dtype=dtype).double()
    assert weight.poll() == ess.ESS_OK
    off = got / product_in_64_bits(x, w) - 1
    half = 2.0 ** -8 if dtype is torch.bfloat16 else 2.0 ** -24
    short = 2.0 ** -13 + ins / 1024 * 2.0 ** -24
    assert off.abs().max() <= half + short, float(off.abs().max())
    assert abs(off.mean()) <= short + 6 * half / math.sqrt(3 * n * outs), float(off.mean())


@pytest.mark.parametrize("n,outs,ins,stride", [(5, 300, 66048, 300), (16, 4700, 65552, 4701), (31, 129, 131072, 200),
                                               (64, 640, 66064, 640), (300, 4100, 65664, 4100), (300, 4096, 65600, 4096),
                                               (257, 4103, 65552, 4200)])
def test_long_sums_of_whole_numbers_are_exact(n, outs, ins, stride):
    """Sums of whole numbers below 2^24, with scales, into rows of any stride."""
    g = torch.Generator(device="cuda")
    g.manual_seed(outs)
    value = lambda rows: torch.randint(-3, 4, (rows, ins), generator=g, device="cuda").float().to(E4M3)
    power = lambda rows: torch.exp2(torch.randint(-1, 1, (rows, -(-ins // 128)), generator=g, device="cuda").float())
    x, w, xs, ws = value(n), value(outs), power(n), power(-(-outs // 128))
    weight = Weight8(w, ws)
    buf = torch.full((n, stride), 7.0, dtype=torch.bfloat16, device="cuda")
    weight.product(x, xs, out=buf[:, :outs])
    assert weight.poll() == ess.ESS_OK
    full = x.float() * xs.repeat_interleave(128, 1)[:, :ins]
    part = w.float() * ws.repeat_interleave(128, 0)[:outs].repeat_interleave(128, 1)[:, :ins]
    want = product_in_64_bits(full, part)
    assert want.abs().max() < 2 ** 22          # in quarters
    assert torch.equal(buf[:, :outs], want.float().to(torch.bfloat16)) and (buf[:, outs:] == 7.0).all()
