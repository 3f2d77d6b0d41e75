"""Chunk attention with a million units and more: a query token with a list each.  A list of
one token gives that token's values, exactly, and its score."""
import pytest
import torch

from host_latent_cache_gb300 import ess

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("total", [1 << 20, (1 << 21) + 77])
def test_lists_of_more_than_a_million_queries(total):
    from host_latent_cache_gb300 import build as B
    from host_latent_cache_gb300.rows import RowCache
    B.build()
    g = torch.Generator(device="cuda")
    g.manual_seed(total)
    n_rows = 640
    raw = torch.randint(0, 256, (n_rows, 400), generator=g, device="cuda", dtype=torch.uint8)
    raw[:, 256:272] = torch.randint(120, 130, (n_rows, 16), generator=g, device="cuda", dtype=torch.uint8)
    raw[:, 272:] = torch.randn(n_rows, 64, generator=g, device="cuda").to(torch.bfloat16).view(torch.uint8)
    cache = RowCache(raw, "q4")
    # more tokens than rows: pages named again and again
    table = torch.randint(0, n_rows // 64, (3, total // 64), generator=g, device="cuda", dtype=torch.int32)
    # (more new tokens than the request has: the first 999 of the second see nothing)
    cu = torch.tensor([0, 600, total - 5, total], dtype=torch.int32, device="cuda")
    T = torch.tensor([640, total - 605 - 999, 5], dtype=torch.int32, device="cuda")
    at = torch.arange(total, device="cuda")
    b = (at >= 600).long() + (at >= total - 5).long()
    sees = (T[b] - (cu[b + 1] - cu[b]) + (at - cu[b]) + 1).clamp(min=0)
    pick = torch.minimum((torch.rand(total, generator=g, device="cuda").double() * sees).long(), (sees - 1).clamp(min=0))
    tokens = torch.where(sees > 0, pick, -1).to(torch.int32).view(total, 1)
    q = torch.empty(total, 1, 576, dtype=torch.bfloat16, device="cuda").normal_(generator=g)
    out, lse = cache.attend_chunk(q, cu, table, T, 1 / 24, tokens=tokens)
    assert cache.poll() == ess.ESS_OK
    slots = torch.where(sees > 0, table[b, pick // 64].long() * 64 + pick % 64, -1)
    for i in range(0, total, 1 << 18):
        some = slice(i, i + (1 << 18))
        rows = cache.read(slots[some].contiguous())
        assert torch.equal(out[some, 0], rows[:, :512])
        z = (q[some, 0].double() * rows.double()).sum(1) / 24
        # 576 products added up in fp32: at most 576 * 2^-24 of their magnitudes, and lse's own roundings
        tol = (q[some, 0].double() * rows.double()).abs().sum(1) / 24 * 576 * 2 ** -24 + 2 ** -20 * (1 + z.abs())
        live = slots[some] >= 0
        assert ((lse[some, 0].double() - z).abs() <= tol)[live].all()
        assert (lse[some, 0][~live] == -float("inf")).all()
