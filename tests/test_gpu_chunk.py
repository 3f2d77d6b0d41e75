"""Attention of chunks of new tokens over the 4-bit device row cache against float64.

The tolerance is that of the attention with a few query tokens (test_gpu_cache_mla): with
A = sum p |v| / sum p and dz = 576 * 2^-24 of a score's summed magnitudes, an output is
off by at most (2 dz + 2^-11 + 2^-18) A + 2^-32 sum |v|, and by bf16's 2^-8 of itself.
"""
import numpy as np
import pytest
import torch

from host_latent_cache_gb300 import ess
from oracle import row_cache as R

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from host_latent_cache_gb300 import build as B
    B.build()
    assert torch.cuda.is_available()
    ess.load()


class Chunks:
    """Ragged requests (new tokens, tokens) over random 4-bit rows behind a shuffled page
    table, with `gap` tokens of q after the last request that belong to none."""

    def __init__(self, seed, requests, heads, page=64, gap=0, qscale=0.5, max_pages=None):
        from host_latent_cache_gb300 import rows
        rng = np.random.default_rng(seed)
        self.requests, self.heads, self.page, self.rng = requests, heads, page, rng
        batch = len(requests)
        per = max_pages or max(1, -(-max(T for _, T in requests) // page))
        n_pages = batch * per + 3
        y = rng.normal(size=(n_pages * page, 512)) * (0.5 + rng.random(512))
        packed, exps = R.q4_encode(y)
        rope = torch.from_numpy(rng.normal(size=(n_pages * page, 64)).astype(np.float32)).to(torch.bfloat16)
        self.raw = np.concatenate([packed, exps, rope.view(torch.uint8).numpy()], axis=1)
        self.table = rng.permutation(n_pages)[: batch * per].reshape(batch, per).astype(np.int32)
        self.cu = np.concatenate([[0], np.cumsum([n for n, _ in requests])]).astype(np.int32)
        self.total = int(self.cu[-1]) + gap
        q = torch.from_numpy((qscale * rng.normal(size=(self.total, heads, 576))).astype(np.float32))
        self.q = q.to(torch.bfloat16).cuda()
        self.scale = 1.0 / 24.0
        self.cache = rows.RowCache(torch.from_numpy(self.raw).cuda(), "q4", page=page)
        self.T = torch.tensor([T for _, T in requests], dtype=torch.int32, device="cuda")
        self.dev_cu = torch.from_numpy(self.cu).cuda()
        self.dev_table = torch.from_numpy(self.table).cuda()

    def attend(self, tokens=None, **kw):
        tok = None if tokens is None else torch.from_numpy(tokens).cuda()
        return self.cache.attend_chunk(self.q, self.dev_cu, self.dev_table, self.T, self.scale, tokens=tok, **kw)

    def lists(self, k, short=False):
        """k tokens that each query may see, in any order, with holes."""
        out = np.full((self.total, k), -1, dtype=np.int32)
        for b, (n, T) in enumerate(self.requests):
            for i in range(n):
                sees = max(0, T - n + i + 1)
                some = self.rng.permutation(sees)[: self.rng.integers(0, k + 1) if short else k]
                row = self.cu[b] + i
                out[row, : some.size] = some
                if some.size > 4:
                    out[row, 2] = -1
        return out

    def check(self, out, lse, tokens=None, skip=(), some=None):
        out, lse = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
        q = self.q.float().cpu().numpy().astype(np.float64)
        for b, (n, T) in enumerate(self.requests):
            t_all = np.arange(T)
            values = R.row_values(self.raw[self.table[b, t_all // self.page].astype(np.int64) * self.page
                                           + t_all % self.page], "q4") if T else np.zeros((0, 576))
            for i in range(n):
                if some and i not in (0, n - 1) and self.rng.random() > some:
                    continue
                row, sees = self.cu[b] + i, max(0, T - n + i + 1)
                if tokens is None:
                    t = np.arange(sees)
                else:
                    t = tokens[row][: min(tokens.shape[1], sees)].astype(np.int64)
                    t = t[(t >= 0) & (t < sees)]
                t = np.array([x for x in t if (b, int(x)) not in skip], dtype=np.int64)
                got, gl = out[row], lse[row]
                if t.size == 0:
                    assert (got == 0).all() and (gl == -np.inf).all(), (b, i)
                    continue
                k = values[t]
                want, wl, size = R.attention(q[row], k, self.scale, np.ones((self.heads, t.size), bool))
                dz = (576 * 2.0 ** -24) * (np.abs(q[row]) @ np.abs(k).T).max(axis=1) * self.scale
                tol = (2 * dz[:, None] + 2.0 ** -11 + 2.0 ** -18) * size + 2.0 ** -8 * np.abs(want) \
                    + 2.0 ** -32 * np.abs(k[:, :512]).sum(axis=0)
                err = np.abs(got - want)
                assert (err <= tol).all(), (b, i, float((err / tol).max()))
                assert (np.abs(gl - wl) <= dz + 2.0 ** -20 * (1 + np.abs(wl))).all(), (b, i)


@pytest.mark.parametrize("requests,heads", [
    ([(1, 1)], 1), ([(1, 500)], 128), ([(16, 16)], 16), ([(5, 4096)], 16), ([(129, 129)], 128),
    ([(200, 300), (1, 1), (0, 700), (64, 64), (3, 1000)], 20), ([(33, 1025), (130, 130)], 128),
    ([(7, 7), (128, 128), (127, 256), (0, 0)], 33), ([(300, 2000)], 8), ([(0, 5), (0, 0), (2, 90)], 96),
    ([(1, 130)] * 40, 7), ([(3, 200), (0, 9)] * 30, 64), ([(900, 900)], 1), ([(2, 20000)], 128),
], ids=lambda v: str(v).replace(" ", "")[:24])
def test_dense(requests, heads):
    c = Chunks(len(requests) + heads, requests, heads)
    out, lse = c.attend()
    assert c.cache.poll() == ess.ESS_OK
    c.check(out, lse, some=0.3)


@pytest.mark.parametrize("page", [1, 7, 16, 100, 256])
def test_page_sizes(page):
    c = Chunks(page, [(40, 513), (3, 130), (3, 3)], 24, page=page)
    out, lse = c.attend()
    assert c.cache.poll() == ess.ESS_OK
    c.check(out, lse, some=0.3)


@pytest.mark.parametrize("requests,heads,k", [
    ([(20, 1000), (3, 3), (0, 50), (1, 700)], 128, 256), ([(50, 600)], 16, 512), ([(9, 5000)], 128, 2048),
    ([(40, 40)], 8, 64), ([(90, 300), (100, 100)], 100, 1), ([(1, 1)], 5, 7),
], ids=lambda v: str(v).replace(" ", "")[:24])
@pytest.mark.parametrize("short", [False, True], ids=["full", "short"])
def test_listed(requests, heads, k, short):
    c = Chunks(heads + k, requests, heads)
    tokens = c.lists(k, short)
    out, lse = c.attend(tokens)
    assert c.cache.poll() == ess.ESS_OK
    c.check(out, lse, tokens, some=0.5)


def test_rows_of_no_request_stay():
    c = Chunks(3, [(5, 70), (0, 3), (60, 200)], 40, gap=9)
    out = torch.full((c.total, 40, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((c.total, 40), 3.0, device="cuda")
    got, gl = c.attend(out=out, lse=lse)
    assert got is out and gl is lse and c.cache.poll() == ess.ESS_OK
    c.check(out, lse)
    assert (out[-9:] == 3.0).all() and (lse[-9:] == 3.0).all()


@pytest.mark.parametrize("heads", [127, 128])
def test_results_that_are_not_32_byte_aligned(heads):
    c = Chunks(19, [(70, 400), (3, 3)], heads)
    want, _ = c.attend()
    buf = torch.zeros(c.total * heads * 512 + 8, dtype=torch.bfloat16, device="cuda")
    got, _ = c.attend(out=buf[8:].view(c.total, heads, 512))
    assert torch.equal(got, want) and (buf[:8] == 0).all()


def test_requests_may_start_behind_the_first_row():
    c = Chunks(5, [(6, 90), (40, 400)], 33, gap=7)
    c.cu = c.cu + 7
    c.dev_cu = torch.from_numpy(c.cu).cuda()
    out = torch.full((c.total, 33, 512), 3.0, dtype=torch.bfloat16, device="cuda")
    out, lse = c.attend(out=out)
    assert c.cache.poll() == ess.ESS_OK
    c.check(out, lse)
    assert (out[:7] == 3.0).all()


@pytest.mark.parametrize("requests,heads,k", [
    ([(1, 3)] * 2000, 1, 0), ([(2, 2), (0, 1), (1, 70)] * 900, 2, 0), ([(900, 1200), (1100, 1100)], 5, 8),
    ([(2500, 2600)], 16, 0),
], ids=["2000", "2700", "listed", "long"])
def test_more_units_than_threads(requests, heads, k):
    c = Chunks(len(requests) + k, requests, heads)
    tokens = c.lists(k) if k else None
    out, lse = c.attend(tokens)
    assert c.cache.poll() == ess.ESS_OK
    c.check(out, lse, tokens, some=0.02 if len(requests) < 9 else 0.3)


def test_threads_on_one_stream():
    """Calls of several threads, with the other attention among them, share a workspace."""
    import threading
    c, d = Chunks(17, [(60, 900), (20, 20)], 64), Chunks(18, [(4, 700), (4, 1500)], 64)
    other = lambda: d.cache.attend(d.q.view(2, 4, 64, 576), d.dev_table, d.T, d.scale)
    want, want_other = c.attend()[0], other()[0]
    torch.cuda.synchronize()
    got, bad = [], []

    def work(f, w):
        try:
            for _ in range(20):
                got.append((f()[0], w))
        except Exception as e:   # noqa: BLE001
            bad.append(e)
    threads = [threading.Thread(target=work, args=a) for a in ((c.attend, want), (other, want_other)) * 2]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    assert not bad and len(got) == 80 and all(torch.equal(o, w) for o, w in got)


@pytest.mark.parametrize("listed", [False, True], ids=["dense", "listed"])
def test_rows_past_4_gb(listed):
    from host_latent_cache_gb300.rows import RowCache
    c = Chunks(20, [(30, 300), (70, 128)], 24)
    tokens = c.lists(64) if listed else None
    want, lse = c.attend(tokens)
    small = c.cache.rows
    extra = 11_000_000 // 64                      # pages ahead of them, 4.4 GB
    big = torch.zeros(extra * 64 + small.shape[0], 400, dtype=torch.uint8, device="cuda")
    big[extra * 64:] = small
    c.cache = RowCache(big, "q4", page=64)
    c.dev_table = c.dev_table + extra
    got, gl = c.attend(tokens)
    assert torch.equal(got, want) and torch.equal(gl, lse) and c.cache.poll() == ess.ESS_OK


def test_more_queries_than_tokens():
    """The first queries then have no token at all."""
    c = Chunks(4, [(10, 4), (300, 150), (2, 0)], 128)
    out, lse = c.attend()
    assert c.cache.poll() == ess.ESS_OK
    c.check(out, lse)


def test_it_agrees_with_the_attention_of_a_few_query_tokens():
    """The same roundings: to the join's order of fp32 sums, off by 2^-20 of A."""
    c = Chunks(6, [(4, 3000), (4, 129), (4, 4)], 128)
    a, la = c.attend()
    b, lb = c.cache.attend(c.q.view(3, 4, 128, 576), c.dev_table, c.T, c.scale)
    assert torch.allclose(la.view(3, 4, 128), lb, rtol=0, atol=2 ** -18)
    err = (a.view(3, 4, 128, 512).float() - b.float()).abs()
    assert (err <= 2.0 ** -7 * b.float().abs() + 2.0 ** -10).all()


@pytest.mark.parametrize("listed", [False, True], ids=["dense", "listed"])
def test_bad_offsets_lengths_tokens_and_pages(listed):
    # a page outside the cache
    c = Chunks(9, [(20, 300), (20, 300)], 16)
    tokens = c.lists(64) if listed else None
    c.table[1, 1] = 1 << 20
    c.dev_table = torch.from_numpy(c.table).cuda()
    out, lse = c.attend(tokens)
    assert c.cache.poll() == ess.ESS_ERR_DEVICE_CHECK
    c.table[1, 1] = 0
    c.check(out, lse, tokens, skip={(1, t) for t in range(64, 128)}, some=0.5)
    # lengths below zero and past the table
    for bad in (-5, 301 + 64):
        c = Chunks(9, [(20, 300), (20, 300)], 16)
        c.T[0] = bad
        out, lse = c.attend()
        assert c.cache.poll() == ess.ESS_ERR_DEVICE_CHECK
        c.requests = [(20, 0 if bad < 0 else 320), (20, 300)]
        c.check(out, lse, some=0.5)
    # offsets that fall, are negative or pass the end: those requests have no queries
    for cu, left in (([0, 20, 10], [(20, 300), (0, 300)]), ([-1, 20, 40], [(0, 300), (20, 300)]),
                     ([0, 20, 41], [(20, 300), (0, 300)]), ([0, 1 << 30, 1 << 31 - 1], [(0, 300), (0, 300)])):
        c = Chunks(9, [(20, 300), (20, 300)], 16)
        c.dev_cu = torch.tensor(cu, dtype=torch.int32, device="cuda")
        out = torch.full((40, 16, 512), 3.0, dtype=torch.bfloat16, device="cuda")
        out, lse = c.attend(out=out)
        assert c.cache.poll() == ess.ESS_ERR_DEVICE_CHECK
        c.requests = left
        c.cu = np.array([0, 20, 40], dtype=np.int32)
        c.check(out, lse, some=0.5)
        for b in range(2):
            if left[b][0] == 0:
                assert (out[20 * b:20 * b + 20] == 3.0).all()
    # a listed token past its query's
    if listed:
        c = Chunks(10, [(20, 300)], 16)
        tokens = c.lists(64)
        tokens[5, 7] = 300 - 20 + 5 + 1
        out, lse = c.attend(tokens)
        assert c.cache.poll() == ess.ESS_ERR_DEVICE_CHECK
        c.check(out, lse, tokens)


def test_masked_tokens_may_hold_anything():
    """A later token's NaN and infinity reach no earlier query."""
    c = Chunks(11, [(30, 100)], 16)
    rope = c.raw[:, 272:].view(np.uint16)
    for t, bits in ((99, 0x7FC0), (98, 0x7F80)):
        rope[c.table[0, t // 64].astype(np.int64) * 64 + t % 64] = bits
    clean, _ = c.attend()
    c.cache.rows.copy_(torch.from_numpy(c.raw))
    out, lse = c.attend()
    assert torch.equal(out[:28], clean[:28]) and torch.isfinite(lse[:28]).all()
    assert torch.isnan(out[29]).all()


@pytest.mark.parametrize("qscale", [1e-30, 1e-3, 300.0, 1e4])
def test_query_sizes(qscale):
    c = Chunks(12, [(20, 400)], 32, qscale=qscale)
    out, lse = c.attend()
    assert c.cache.poll() == ess.ESS_OK
    c.check(out, lse)


def test_streams_workspaces_and_graphs():
    c, d = Chunks(13, [(100, 2000), (30, 30)], 128), Chunks(14, [(17, 5000)], 16)
    want = [x.attend() for x in (c, d)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(2)]
    got = []
    for _ in range(10):
        for s, x in zip(streams, (c, d)):
            with torch.cuda.stream(s):
                got.append(x.attend())
    torch.cuda.synchronize()
    for i, (o, l) in enumerate(got):
        assert torch.equal(o, want[i % 2][0]) and torch.equal(l, want[i % 2][1])
    ws = c.cache.chunk_workspace()
    o, l = c.attend(workspace=ws)
    assert torch.equal(o, want[0][0]) and torch.equal(l, want[0][1])
    # captured: lengths, offsets and queries are read when the graph runs
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = c.attend()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(out, want[0][0])
    c.requests = [(40, 1500), (90, 200)]
    c.cu = np.array([0, 40, 130], dtype=np.int32)
    c.dev_cu.copy_(torch.from_numpy(c.cu))
    c.T.copy_(torch.tensor([1500, 200], dtype=torch.int32))
    graph.replay()
    torch.cuda.synchronize()
    c.check(out, lse, some=0.2)
    assert c.cache.poll() == ess.ESS_OK


def test_empty_arguments():
    c = Chunks(15, [(4, 60)], 8)
    out, lse = c.attend(np.zeros((4, 0), dtype=np.int32))
    assert (out == 0).all() and (lse == -float("inf")).all()
    empty = torch.zeros(1, 0, dtype=torch.int32, device="cuda")
    out, lse = c.cache.attend_chunk(c.q, c.dev_cu, empty, torch.zeros_like(c.T), c.scale)
    assert (out == 0).all() and (lse == -float("inf")).all() and c.cache.poll() == ess.ESS_OK
    out, lse = c.cache.attend_chunk(c.q[:0], torch.zeros_like(c.dev_cu), c.dev_table, c.T, c.scale)
    assert out.shape == (0, 8, 512)
    none = torch.zeros(0, dtype=torch.int32, device="cuda")
    out, lse = c.cache.attend_chunk(c.q, torch.zeros(1, dtype=torch.int32, device="cuda"), empty[:0], none, c.scale)
    assert out.shape == (4, 8, 512)


def test_refusals():
    c = Chunks(16, [(4, 60)], 8)
    other = {"q": [c.q.float(), c.q[0], c.q[:, :, :512], c.q.transpose(0, 1)], "cu": [c.dev_cu.long(), c.dev_cu[:1]],
             "T": [c.T.long(), c.T.cpu()], "page_table": [c.dev_table.long(), c.dev_table[0]]}
    good = dict(q=c.q, cu=c.dev_cu, page_table=c.dev_table, T=c.T, sm_scale=c.scale)
    for name, bad in other.items():
        for value in bad:
            with pytest.raises(ValueError):
                c.cache.attend_chunk(**{**good, name: value})
    for kw in (dict(tokens=c.dev_table), dict(out=torch.empty(4, 8, 512, device="cuda")),
               dict(lse=torch.empty(4, 9, device="cuda")), dict(workspace=torch.empty(8, device="cuda"))):
        with pytest.raises(ValueError):
            c.cache.attend_chunk(**good, **kw)
    with pytest.raises(RuntimeError):
        c.cache.attend_chunk(**good, workspace=c.cache.chunk_workspace()[:256])
    with pytest.raises(RuntimeError):
        c.cache.attend_chunk(**{**good, "sm_scale": -1.0})
