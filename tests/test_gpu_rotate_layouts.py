"""Rotations into every layout whose rows keep apart give the dense result's bits."""
import pytest
import torch

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("n,heads,row,head", [
    (5, 3, 192, 64), (5, 3, 64, 320), (2, 2, 64, 128), (9, 1, 64, 0), (1, 9, 0, 64), (4, 8, 8 * 576, 576),
    (4, 8, 576, 4 * 576), (30, 2, 200, 64), (7, 3, 72 * 3, 72), (7, 3, 72, 72 * 7),
])
def test_layouts(n, heads, row, head):
    from host_latent_cache_gb300 import build as B
    from host_latent_cache_gb300.rows import rotate
    B.build()
    g = torch.Generator(device="cuda")
    g.manual_seed(n)
    x = torch.randn(n, heads, 64, generator=g, device="cuda").to(torch.bfloat16)
    pos = torch.randint(0, 1 << 20, (n,), generator=g, device="cuda", dtype=torch.int32)
    freq = [10000.0 ** (-i / 32.0) for i in range(32)]
    buf = torch.full((n * row + heads * head + 64,), 5.0, dtype=torch.bfloat16, device="cuda")
    out = torch.as_strided(buf, (n, heads, 64), (row, head, 1))
    rotate(x, pos, freq, out=out)
    assert torch.equal(out, rotate(x, pos, freq))
    out.fill_(5.0)
    assert (buf == 5.0).all()
