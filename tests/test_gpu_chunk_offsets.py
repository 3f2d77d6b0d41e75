"""Offsets of chunks that fall and rise again: a query row belongs to one request, or to none."""
import numpy as np
import pytest
import torch

from host_latent_cache_gb300 import ess
from test_gpu_chunk import Chunks, _lib   # noqa: F401  (the fixture builds the library)

pytestmark = pytest.mark.gpu


def accepted(cu, total):
    """The requests that have queries: in range, and behind the end of every one before."""
    end, keep = 0, []
    for lo, hi in zip(cu[:-1], cu[1:]):
        fine = 0 <= lo <= hi <= total
        keep.append(fine and (lo == hi or lo >= end))
        if fine and hi > lo:
            end = max(end, hi)
    return keep


@pytest.mark.parametrize("listed", [False, True], ids=["dense", "listed"])
@pytest.mark.parametrize("heads", [16, 128])
@pytest.mark.parametrize("cu", [
    [0, 40, 0, 40], [0, 20, 10, 30], [0, 20, 10, 30, 50], [30, 50, 0, 20, 20, 40], [0, 20, 5, 10, 30, 60],
    [0, 99, 20, 40], [-3, 30, 10, 60], [0, 25, 25, 3, 25, 40], [0, 60] * 20, [0, 1, 0, 60, 0, 60],
], ids=lambda v: "_".join(map(str, v[:6])))
def test_offsets_that_fall_and_rise(cu, heads, listed):
    total, batch = 60, len(cu) - 1
    T = [3000 if b == batch - 1 else 200 + 7 * b for b in range(batch)]
    c = Chunks(batch + heads, [(0, t) for t in T], heads, gap=total)
    keep = accepted(cu, total)
    assert sum(keep) < batch
    c.requests = [(hi - lo if k else 0, t) for lo, hi, k, t in zip(cu[:-1], cu[1:], keep, T)]
    c.cu = np.array(cu, dtype=np.int32)
    c.dev_cu = torch.from_numpy(c.cu).cuda()
    tokens = c.lists(300) if listed else None
    out = torch.full((total, heads, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((total, heads), 3.0, device="cuda")
    c.attend(tokens, out=out, lse=lse)
    assert c.cache.poll() == ess.ESS_ERR_DEVICE_CHECK
    c.check(out, lse, tokens, some=0.4)
    written = np.zeros(total, dtype=bool)
    for b in range(batch):
        if keep[b]:
            assert not written[cu[b]:cu[b + 1]].any()
            written[cu[b]:cu[b + 1]] = True
    stays = torch.from_numpy(~written)
    assert (out.cpu()[stays] == 3.0).all() and (lse.cpu()[stays] == 3.0).all()
    first = out.clone()
    c.attend(tokens, out=out, lse=lse)
    assert torch.equal(out, first)


def test_thousands_of_requests_for_the_same_rows():
    """Of 8000 requests for the same 300 query tokens the first has them."""
    c = Chunks(1, [(0, 70), (0, 70)], 8, gap=300)
    batch = 8000
    cu = np.tile(np.array([0, 300], dtype=np.int32), batch // 2 + 1)[: batch + 1]
    c.dev_cu, c.cu = torch.from_numpy(cu).cuda(), cu[:3]
    c.T = torch.full((batch,), 70, dtype=torch.int32, device="cuda")
    c.dev_table = c.dev_table[:1].repeat(batch, 1).contiguous()
    c.requests = [(300, 70)]
    out, lse = c.attend()
    assert c.cache.poll() == ess.ESS_ERR_DEVICE_CHECK
    c.check(out, lse, some=0.2)


def test_many_requests_inside_one():
    """Of 3000 requests the first 101 have their rows, and those behind, which start inside the
    101st, have none."""
    total = 700
    cu = list(range(101)) + [700] + [100 + i % 500 for i in range(2897)] + [699, 700]
    batch = len(cu) - 1
    c = Chunks(2, [(0, 70), (0, 70)], 16, gap=total)
    keep = accepted(cu, total)
    assert sum(keep[:101]) == 101 and not any(hi > lo and k for lo, hi, k in zip(cu[101:], cu[102:], keep[101:]))
    c.cu = np.array(cu, dtype=np.int32)
    c.dev_cu = torch.from_numpy(c.cu).cuda()
    c.T = torch.full((batch,), 70, dtype=torch.int32, device="cuda")
    c.dev_table = c.dev_table[:1].repeat(batch, 1).contiguous()
    c.table = c.table[:1].repeat(batch, axis=0)
    c.requests = [(hi - lo if k else 0, 70) for lo, hi, k in zip(cu[:-1], cu[1:], keep)]
    out, lse = c.attend()
    assert c.cache.poll() == ess.ESS_ERR_DEVICE_CHECK
    c.check(out, lse, some=0.2)
