"""Attention over the 4-bit device row cache against float64.

The tolerance follows from the kernel's roundings.  A score is an fp32 sum of
576 exact products: off by at most 576 * 2^-24 of the sum of their magnitudes
(dz, after the scale, in nats), so a weight is off by dz relative, the weights'
sum too, and the fp16 numerator by 2^-11 more.  The numerators are scaled so that
the largest is 2^7 or more, and fp16's steps below 2^-14 are 2^-24: small ones are
off by up to 2^-25 / 2^7 of the largest, which is at most the sum.  With
A = sum p |v| / sum p an output is off by at most
(2 dz + 2^-11 + 2^-18) A + 2^-32 sum |v|, and its bf16 rounding by 2^-8 of itself.
The 2^-18 covers the exponential's own error and fp32 sums.
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


class Case:
    """A cache of random 4-bit rows behind a shuffled page table, with queries."""

    def __init__(self, seed, lens, ways, heads, page=64, max_pages=None, extra=3, qscale=0.5):
        from host_latent_cache_gb300 import rows
        rng = np.random.default_rng(seed)
        self.lens, self.ways, self.heads, self.page = list(lens), ways, heads, page
        self.batch = len(self.lens)
        per = max_pages or max(1, -(-max(self.lens) // page))
        n_pages = self.batch * per + extra
        y = rng.normal(size=(n_pages * page, 512)) * (0.5 + rng.random(512))
        packed, exps = R.q4_encode(y)
        rope = torch.from_numpy(rng.normal(size=(n_pages * page, 64)).astype(np.float32)).to(torch.bfloat16)
        self.raw = np.concatenate([packed, exps, rope.view(torch.uint8).numpy()], axis=1)
        self.table = rng.permutation(n_pages)[: self.batch * per].reshape(self.batch, per).astype(np.int32)
        q = torch.from_numpy((qscale * rng.normal(size=(self.batch, ways, heads, 576))).astype(np.float32))
        self.q = q.to(torch.bfloat16).cuda()
        self.scale = 1.0 / 24.0
        self.rng = rng
        self.cache = rows.RowCache(torch.from_numpy(self.raw).cuda(), "q4", page=page)
        self.T = torch.tensor(self.lens, dtype=torch.int32, device="cuda")
        self.dev_table = torch.from_numpy(self.table).cuda()

    def attend(self, tokens=None, **kw):
        tok = None if tokens is None else torch.from_numpy(tokens).cuda()
        return self.cache.attend(self.q, self.dev_table, self.T, self.scale, tokens=tok, **kw)

    def rows_of(self, b, t):
        return R.row_values(self.raw[self.table[b, t // self.page].astype(np.int64) * self.page
                                     + t % self.page], "q4")

    def check(self, out, lse, tokens=None, skip=()):
        out, lse = out.float().cpu().numpy().astype(np.float64), lse.cpu().numpy().astype(np.float64)
        q = self.q.float().cpu().numpy().astype(np.float64)
        for b, T in enumerate(self.lens):
            for m in range(self.ways):
                if tokens is None:
                    t = np.arange(max(0, T - (self.ways - 1) + m))
                else:
                    t = tokens[b, m][: min(tokens.shape[2], T)].astype(np.int64)
                    t = t[(t >= 0) & (t < T)]
                t = np.array([x for x in t if (b, int(x)) not in skip], dtype=np.int64) if skip else t
                got, gl = out[b, m], lse[b, m]
                if t.size == 0:
                    assert (got == 0).all() and (gl == -np.inf).all(), (b, m)
                    continue
                k = self.rows_of(b, t)
                want, wl, size = R.attention(q[b, m], k, self.scale, np.ones((self.heads, t.size), bool))
                dz = (576 * 2.0 ** -24) * (np.abs(q[b, m]) @ np.abs(k).T).max(axis=1) * self.scale
                tol = (2 * dz[:, None] + 2.0 ** -11 + 2.0 ** -18) * size + 2.0 ** -8 * np.abs(want) \
                    + 2.0 ** -32 * np.abs(k[:, :512]).sum(axis=0)
                err = np.abs(got - want)
                assert (err <= tol).all(), (b, m, float((err / tol).max()))
                assert (np.abs(gl - wl) <= dz + 2.0 ** -20 * (1 + np.abs(wl))).all(), (b, m)


@pytest.mark.parametrize("lens,ways,heads", [
    ([1], 1, 1), ([2], 1, 16), ([127, 128, 129], 1, 128), ([4096], 1, 16), ([0, 1, 63, 700], 1, 20),
    ([5, 0, 1, 1000], 4, 128), ([64, 65], 2, 64), ([300, 2, 257], 3, 33), ([2500, 31, 640], 1, 96),
    ([1, 1, 1, 1, 1], 2, 7), ([3000] * 7, 1, 128), ([20000], 1, 128),
], ids=lambda v: str(v).replace(" ", "")[:24])
def test_dense(lens, ways, heads):
    c = Case(sum(lens) + heads, lens, ways, heads)
    out, lse = c.attend()
    assert c.cache.poll() == ess.ESS_OK
    c.check(out, lse)


@pytest.mark.parametrize("page", [1, 7, 16, 100, 256])
def test_page_sizes(page):
    c = Case(page, [513, 130, 3], 2, 24, page=page)
    out, lse = c.attend()
    assert c.cache.poll() == ess.ESS_OK
    c.check(out, lse)


@pytest.mark.parametrize("lens,ways,heads,k", [
    ([1000, 3, 0], 1, 128, 256), ([4000, 2000], 2, 16, 512), ([5000], 4, 128, 2048), ([40], 1, 8, 64),
    ([300, 300], 1, 128, 1),
], ids=lambda v: str(v).replace(" ", "")[:24])
def test_listed_tokens(lens, ways, heads, k):
    c = Case(k, lens, ways, heads)
    tok = np.full((len(lens), ways, k), 12345678, dtype=np.int32)   # entries past min(k, T) are not read
    for b, T in enumerate(lens):
        for m in range(ways):
            n = min(k, T)
            tok[b, m, :n] = c.rng.permutation(T)[:n]
            if n > 4:
                tok[b, m, c.rng.integers(0, n, n // 4)] = -1        # holes anywhere
    if lens[0] == 1000:
        tok[0, 0, :256] = -7                                        # a list that holds nothing
    out, lse = c.attend(tok)
    assert c.cache.poll() == ess.ESS_OK
    c.check(out, lse, tok)


def test_a_listed_token_counts_as_often_as_it_is_listed():
    c = Case(5, [10], 1, 4)
    tok = np.array([[[3, 3, 3, 5]]], dtype=np.int32)
    out, lse = c.attend(tok)
    c.check(out, lse, tok)


def test_peaked_and_rising_scores():
    """Running maxima that keep growing along the tokens, and single tokens that take it all."""
    c = Case(8, [3000], 1, 64, qscale=6.0)
    k = c.rows_of(0, np.arange(3000))
    q = c.q.float().cpu().numpy()
    order = np.argsort(k @ q[0, 0, 0])                  # ascending scores of head 0
    tok = order.astype(np.int32).reshape(1, 1, -1)
    for t in (tok, tok[:, :, ::-1].copy()):
        out, lse = c.attend(t)
        c.check(out, lse, t)


class Rising(Case):
    """A Case whose scores rise by `step` nats with every tile of 128 tokens, in
    a saw-tooth of `period` tiles, for the heads that `rises` picks: the first RoPE
    value of token t is the tile's number in its period, the queries' is
    step / scale (both exact in bf16)."""

    def __init__(self, seed, lens, ways, heads, step=6, period=60, rises=lambda h: True):
        from host_latent_cache_gb300 import rows
        super().__init__(seed, lens, ways, heads)
        for b, T in enumerate(self.lens):
            t = np.arange(T)
            at = self.table[b, t // 64].astype(np.int64) * 64 + t % 64
            tooth = torch.from_numpy((t // 128 % period).astype(np.float32)).to(torch.bfloat16)
            self.raw[at, 272:274] = tooth.view(torch.uint8).numpy().reshape(-1, 2)
        self.cache = rows.RowCache(torch.from_numpy(self.raw).cuda(), "q4")
        for h in range(heads):
            self.q[:, :, h, 512] = step / self.scale if rises(h) else 0.0


@pytest.mark.parametrize("lens,ways,heads,rises", [
    ([800] * 76, 1, 128, lambda h: True), ([800] * 76, 1, 128, lambda h: h % 3 == 0),
    ([1500] * 40, 2, 64, lambda h: h != 17), ([3000, 40, 9000, 1], 1, 20, lambda h: True),
], ids=["all", "some", "two-ways", "few-heads"])
def test_maxima_that_grow_from_tile_to_tile(lens, ways, heads, rises):
    """Pairs hold several tiles of a segment and rescale O at nearly each; every
    one of a pair's rows, and both halves of the dims, follow."""
    c = Rising(40 + len(lens), lens, ways, heads, rises=rises)
    out, lse = c.attend()
    assert c.cache.poll() == ess.ESS_OK
    c.check(out, lse)
    for _ in range(20):
        again = c.attend()
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)


def test_a_long_request_whose_maxima_grow():
    c = Rising(45, [60000], 1, 128, period=25)       # six tiles a pair
    out, lse = c.attend()
    c.check(out, lse)
    for _ in range(20):
        again = c.attend()
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)


def test_listed_tokens_whose_maxima_grow():
    c = Rising(46, [7000] * 8, 1, 128)
    tok = np.stack([np.sort(c.rng.permutation(7000)[:6000]) for _ in range(8)]).astype(np.int32)[:, None]
    out, lse = c.attend(tok)                         # five tiles a pair
    assert c.cache.poll() == ess.ESS_OK
    c.check(out, lse, tok)
    down = np.ascontiguousarray(tok[:, :, ::-1])     # and maxima that never grow
    c.check(*c.attend(down), down)
    for _ in range(20):
        again = c.attend(tok)
        assert torch.equal(again[0], out) and torch.equal(again[1], lse)


def test_what_lies_behind_the_last_token_does_not_matter():
    c = Case(9, [70, 129], 2, 16, max_pages=5)
    want = c.attend()
    rows = c.cache.rows.clone()
    used = torch.zeros(rows.shape[0], dtype=torch.bool, device="cuda")
    for b, T in enumerate(c.lens):
        t = np.arange(T)
        used[torch.from_numpy(c.table[b, t // 64].astype(np.int64) * 64 + t % 64).cuda()] = True
    rows[~used] = 0xFF                                  # NaN in k^R, the largest codes and exponents
    from host_latent_cache_gb300.rows import RowCache
    table = c.dev_table.clone()
    table[0, 2:] = 1 << 30                              # pages past the last token are not read
    table[1, 3:] = -9
    cache = RowCache(rows, "q4")
    got = cache.attend(c.q, table, c.T, c.scale)
    assert cache.poll() == ess.ESS_OK
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_infinite_and_nan_queries_stay_in_their_row():
    c = Case(10, [200, 200], 1, 16)
    want, _ = c.attend()
    c.q[0, 0, 3, 5] = float("nan")
    c.q[1, 0, 15, 0] = float("inf")
    out, lse = c.attend()
    bad = torch.zeros(2, 1, 16, dtype=torch.bool, device="cuda")
    bad[0, 0, 3] = bad[1, 0, 15] = True
    assert torch.equal(out[~bad], want[~bad])
    assert torch.isnan(out[bad]).all()


def test_device_checks():
    c = Case(11, [100, 200], 1, 8)
    tok = np.full((2, 1, 50), -1, dtype=np.int32)
    tok[0, 0, :3] = [5, 100, 7]                          # 100 is past the request's last token
    tok[1, 0, :2] = [199, 0]
    out, lse = c.attend(tok)
    assert c.cache.poll() == ess.ESS_ERR_DEVICE_CHECK
    c.check(out, lse, tok)
    c.dev_table[1, 1] = 1 << 30                          # a page outside the cache: its tokens are left out
    out, lse = c.attend()
    assert c.cache.poll() == ess.ESS_ERR_DEVICE_CHECK
    c.check(out, lse, skip={(1, t) for t in range(64, 128)})
    c.dev_table[1, 1] = int(c.table[1, 1])
    for bad, as_if in ((-3, 0), (1 << 20, 256)):         # a length outside its range is clamped
        c.T[1] = bad
        c.lens[1] = as_if
        out, lse = c.attend()
        assert c.cache.poll() == ess.ESS_ERR_DEVICE_CHECK
        c.check(out, lse)


def test_runs_are_the_same_and_a_workspace_may_be_dirty():
    c = Case(12, [5000, 17, 900], 2, 128)
    ws = c.cache.workspace(3, 2, 128)
    ws.fill_(0xFF)
    a = c.attend(workspace=ws)
    b = c.attend()
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_captured_calls_follow_the_lengths():
    c = Case(13, [700, 300], 1, 128, max_pages=12)
    out = torch.empty(2, 1, 128, 512, dtype=torch.bfloat16, device="cuda")
    lse = torch.empty(2, 1, 128, device="cuda")
    ws = c.cache.workspace(2, 1, 128)
    c.attend(out=out, lse=lse, workspace=ws)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        c.attend(out=out, lse=lse, workspace=ws)
    for lens in ([700, 300], [1, 768], [0, 0], [64, 640]):
        c.lens = lens
        c.T.copy_(torch.tensor(lens, dtype=torch.int32))
        graph.replay()
        torch.cuda.synchronize()
        c.check(out, lse)
    assert c.cache.poll() == ess.ESS_OK


def test_many_short_requests():
    """More requests than threads that scan their lengths, runs of empty ones
    among them, and more than fit the pairs evenly."""
    lens = [(7 * i * i) % 150 if i % 5 else 0 for i in range(1700)]
    lens[100:200] = [0] * 100
    c = Case(18, lens, 1, 8, page=16)
    out, lse = c.attend()
    assert c.cache.poll() == ess.ESS_OK
    c.check(out, lse)
    lens = [0] * 40 + [1000] + [0] * 900
    c = Case(19, lens, 2, 100)
    out, lse = c.attend()
    c.check(out, lse)


def test_no_request_has_a_token():
    c = Case(20, [1, 1, 1], 1, 128)
    c.lens = [0, 0, 0]
    c.T.zero_()
    out, lse = c.attend()
    c.check(out, lse)
    assert c.cache.poll() == ess.ESS_OK


@pytest.mark.parametrize("fill", [0xFF, 0x7F])
@pytest.mark.parametrize("heads,ways", [(128, 1), (7, 2), (128, 4)])
def test_empty_requests_over_a_dirty_workspace(fill, heads, ways):
    """Nothing of an empty request is in the workspace, whatever it held."""
    c = Case(30, [1] * 9, ways, heads)
    c.lens = [0, 0, 1, 0, 0, 1, 0, 0, 0]
    c.T.copy_(torch.tensor(c.lens, dtype=torch.int32))
    ws = c.cache.workspace(9, ways, heads)
    ws.fill_(fill)
    out, lse = c.attend(workspace=ws)
    c.check(out, lse)


def test_rows_past_32_bits_of_offset():
    from host_latent_cache_gb300.rows import RowCache
    n_rows = (5 << 30) // 400 // 64 * 64            # a cache of 5 GiB
    rows = torch.zeros(n_rows, 400, dtype=torch.uint8, device="cuda")
    c = Case(21, [300, 70], 1, 128)
    last = n_rows // 64 - 1
    table = torch.tensor([[last, 3, last - 7, last // 2, 0], [last - 1, 5, 6, 7, 8]],
                         dtype=torch.int32, device="cuda")
    for b in range(2):
        for p in range(5):
            at, frm = int(table[b, p]) * 64, int(c.table[b, p]) * 64
            rows[at:at + 64] = c.cache.rows[frm:frm + 64]
    cache = RowCache(rows, "q4")
    out, lse = cache.attend(c.q, table, c.T, c.scale)
    assert cache.poll() == ess.ESS_OK
    c.check(out, lse)


def test_queries_of_any_scale():
    """Each query row is brought to fp16's range by its own power of two."""
    c = Case(22, [400], 1, 64)
    q = c.q.float()
    for h in range(64):
        q[0, 0, h] *= 2.0 ** (h - 30)               # 2^-30 .. 2^33
    q[0, 0, 40:, 512:] *= 2.0 ** -20                # and a RoPE part far below the rest
    q[0, 0, 3] = 0
    c.q = q.to(torch.bfloat16)
    out, lse = c.attend()
    c.check(out, lse)


def test_scales_far_below_one():
    """A scale whose product with a row's power of two is below fp32's range:
    every token weighs the same."""
    c = Case(24, [300, 3], 2, 16)
    c.q = (c.q.float() * 2.0 ** -115).to(torch.bfloat16)
    c.scale = 2.0 ** -60
    out, lse = c.attend()
    c.check(out, lse)


def test_scales_far_above_one():
    """A scale near fp32's end, alone or with a row's power of two: scores of 0 still
    weigh every token the same."""
    c = Case(34, [300, 3], 2, 16)
    c.q[:, :, ::2] = 0
    for scale, q in ((3e38, None), (2.0 ** 100, 2.0 ** 60)):
        if q:                                       # c2 past the range; rows orthogonal to the tokens
            c.q.zero_()
            c.q[:, :, ::2, 575] = q
            c.raw[:, 398:400] = 0
            c.cache.rows.copy_(torch.from_numpy(c.raw))
        out, lse = c.cache.attend(c.q, c.dev_table, c.T, scale)
        for b, T in enumerate(c.lens):
            for m in range(2):
                n = T - 1 + m
                v = torch.from_numpy(c.rows_of(b, np.arange(n))[:, :512])
                want, size = v.mean(0), v.abs().mean(0)
                got = out[b, m, ::2].double().cpu()
                assert ((got - want).abs() <= 2.0 ** -8 * want.abs() + (2.0 ** -11 + 2.0 ** -18) * size).all()
                assert ((lse[b, m, ::2].double().cpu() - np.log(n)).abs() <= 2.0 ** -20 * (1 + np.log(n))).all()


def test_short_requests_with_queries_of_many_scales():
    """Requests of one tile each, several to a pair: each one's row scales
    follow those of the one before at once."""
    lens = [1 + (11 * i) % 128 for i in range(400)]
    c = Case(23, lens, 1, 64, page=16)
    q = c.q.float() * 2.0 ** ((torch.arange(400 * 64, device="cuda") * 13) % 41 - 30).view(400, 1, 64, 1)
    c.q = q.to(torch.bfloat16)
    out, lse = c.attend()
    assert c.cache.poll() == ess.ESS_OK
    c.check(out, lse)


def test_two_streams_beside_one_another():
    a, b = Case(14, [6000] * 3, 1, 128), Case(15, [4000] * 4, 2, 64)
    want = a.attend(), b.attend()
    torch.cuda.synchronize()
    sa, sb = torch.cuda.Stream(), torch.cuda.Stream()
    for _ in range(5):
        with torch.cuda.stream(sa):
            ga = a.attend()
        with torch.cuda.stream(sb):
            gb = b.attend()
    torch.cuda.synchronize()
    for g, w in zip((ga, gb), want):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


def test_one_cache_on_two_streams():
    """Calls on one cache beside one another, with other queries and lengths, both
    long enough that their outputs go through the workspace."""
    c = Case(31, [6000, 5000, 7000], 1, 128)
    q2, T2 = c.q.roll(1, 2), c.T.flip(0).contiguous()
    table2 = c.dev_table.flip(0).contiguous()
    calls = [lambda: c.cache.attend(c.q, c.dev_table, c.T, c.scale),
             lambda: c.cache.attend(q2, table2, T2, c.scale)]
    want = [f() for f in calls]
    torch.cuda.synchronize()
    assert not torch.equal(want[0][0], want[1][0])
    before = len(c.cache._ws)
    streams = [torch.cuda.Stream() for _ in calls]
    got = [[], []]
    for _ in range(40):
        for i in range(2):
            with torch.cuda.stream(streams[i]):
                got[i].append(calls[i]())
    torch.cuda.synchronize()
    assert len(c.cache._ws) == before + 2
    for w, results in zip(want, got):
        for out, lse in results:
            assert torch.equal(out, w[0]) and torch.equal(lse, w[1])


def test_arguments_are_refused():
    c = Case(16, [50], 1, 4)
    ok = dict(q=c.q, page_table=c.dev_table, T=c.T, sm_scale=c.scale)
    for change in (dict(q=c.q.float()), dict(q=c.q[..., :575]), dict(q=c.q.cpu()),
                   dict(T=c.T.long()), dict(T=c.T.repeat(2)), dict(page_table=c.dev_table.long()),
                   dict(page_table=c.dev_table[0]), dict(tokens=c.T), dict(out=c.q),
                   dict(q=c.q.transpose(1, 2).expand(1, 4, 3, 576))):
        with pytest.raises(ValueError):
            c.cache.attend(**{**ok, **change})
    for change in (dict(sm_scale=0.0), dict(sm_scale=float("nan")), dict(q=c.q.expand(1, 1, 4, 576).repeat(1, 5, 1, 1)),
                   dict(workspace=c.cache.workspace(1, 1, 4)[:0])):
        with pytest.raises(ess.EssError):
            c.cache.attend(**{**ok, **change})
    from host_latent_cache_gb300.rows import RowCache
    with pytest.raises(ess.EssError):
        RowCache(torch.zeros(64, 656, dtype=torch.uint8, device="cuda"), "compact").attend(**ok)


def test_empty_batches_lists_and_tables():
    c = Case(32, [70, 3], 2, 16)
    out, lse = c.cache.attend(c.q[:0], c.dev_table[:0], c.T[:0], c.scale)
    assert out.shape == (0, 2, 16, 512) and lse.shape == (0, 2, 16)
    empty = torch.empty(0, 2, 7, dtype=torch.int32, device="cuda")
    assert c.cache.attend(c.q[:0], c.dev_table[:0], c.T[:0], c.scale, tokens=empty)[0].numel() == 0
    none = np.zeros((2, 2, 0), dtype=np.int32)
    c.check(*c.attend(none), none)
    got = torch.full_like(c.q[..., :512], 7).contiguous()
    c.lens = [0, 0]
    c.T.zero_()
    c.check(*c.cache.attend(c.q, c.dev_table[:, :0].contiguous(), c.T, c.scale, out=got))
    assert not got.any() and c.cache.poll() == ess.ESS_OK
    c.T[1] = 5                                      # a token, and no page for it
    out, lse = c.cache.attend(c.q, c.dev_table[:, :0].contiguous(), c.T, c.scale)
    assert c.cache.poll() == ess.ESS_ERR_DEVICE_CHECK
    assert not out.any() and (lse == -float("inf")).all()


def test_sizes_past_32_bits_are_refused():
    """Not taken modulo 2^32: a list of 2^32 + 5 entries is not one of five."""
    from host_latent_cache_gb300 import rows
    c = Case(33, [50], 1, 4)
    tok = torch.empty(1, 1, (1 << 32) + 5, dtype=torch.int32, device="cuda")
    with pytest.raises(ValueError):
        c.cache.attend(c.q, c.dev_table, c.T, c.scale, tokens=tok)
    with pytest.raises(ValueError):
        c.cache.attend(c.q, tok[0], c.T, c.scale)
    wide = tok.view(torch.bfloat16)[0, :, :(1 << 32) + 128]
    with pytest.raises(ValueError):
        rows.norm_q8(wide, wide[0])


def test_threads_at_once():
    """Threads that share the cache and its stream, each with its own request."""
    import threading
    c = Case(26, [5000, 900], 1, 128)
    qs = [c.q.roll(i, 2) for i in range(4)]
    want = [c.cache.attend(q, c.dev_table, c.T, c.scale) for q in qs]
    got = [[] for _ in qs]

    def run(i):
        for _ in range(30):
            got[i].append(c.cache.attend(qs[i], c.dev_table, c.T, c.scale))
    threads = [threading.Thread(target=run, args=(i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert len(g) == 30
        for o, l in g:
            assert torch.equal(o, w[0]) and torch.equal(l, w[1])


def test_two_captured_graphs_beside_one_another():
    """Without a workspace of the caller's each graph has one of its own."""
    a, b = Case(27, [6000] * 3, 1, 128), Case(28, [4000] * 4, 2, 64)
    q2 = a.q.roll(1, 2)
    want = [a.attend(), a.cache.attend(q2, a.dev_table, a.T, a.scale), b.attend()]
    graphs, got = [], []
    for x, q in ((a, a.q), (a, q2), (b, b.q)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            got.append(x.cache.attend(q, x.dev_table, x.T, x.scale))
        graphs.append(g)
    streams = [torch.cuda.Stream() for _ in graphs]
    torch.cuda.synchronize()
    for _ in range(5):
        for g, s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        eager = a.attend()
    torch.cuda.synchronize()
    for g, w in zip(got + [eager], want + [want[0]]):
        assert torch.equal(g[0], w[0]) and torch.equal(g[1], w[1])


def test_one_workspace_serves_every_batch():
    c = Case(29, [70] * 6, 1, 16)
    for n in (1, 6, 3, 2):
        c.lens = [70] * n
        c.check(*c.cache.attend(c.q[:n], c.dev_table[:n], c.T[:n], c.scale))
    assert len(c.cache._ws) == 1


def test_caches_on_one_stream_share_a_workspace():
    """A model's layers hold one workspace between them, and give it up together."""
    import gc
    from host_latent_cache_gb300 import rows
    from host_latent_cache_gb300.rows import RowCache
    gc.collect()
    rows.release_workspaces()
    cases = [Case(60 + i, [5000 - 900 * i, 300], 1, 128) for i in range(3)]
    want = [c.attend(workspace=c.cache.workspace(2, 1, 128)) for c in cases]
    size = cases[0].cache.workspace(2, 1, 128).numel()
    layers = [(c, RowCache(c.cache.rows, "q4")) for c in cases for _ in range(8)]
    torch.cuda.synchronize()
    before = torch.cuda.memory_allocated()
    got = [layer.attend(c.q, c.dev_table, c.T, c.scale) for c, layer in layers]
    outs = sum(o.untyped_storage().nbytes() + l.untyped_storage().nbytes() for o, l in got)
    used = torch.cuda.memory_allocated() - before
    assert size <= used < outs + 2 * size
    for i, (out, lse) in enumerate(got):
        assert torch.equal(out, want[i // 8][0]) and torch.equal(lse, want[i // 8][1])
    rows.release_workspaces()
    assert torch.cuda.memory_allocated() - before <= used - size
    again = layers[0][1].attend(cases[0].q, cases[0].dev_table, cases[0].T, cases[0].scale)
    assert torch.equal(again[0], want[0][0])
    del got, again
    del layers
    gc.collect()
    assert torch.cuda.memory_allocated() < before + size     # it goes with the last cache


def test_threads_with_a_cache_each():
    """Threads on one stream, each with a cache of its own, share that stream's
    workspace and not one another's partials."""
    import threading
    cases = [Case(70 + i, [5000 - 1000 * i, 900], 1, 128) for i in range(3)]
    want = [c.attend() for c in cases]
    got = [[] for _ in cases]

    def run(i):
        for _ in range(30):
            got[i].append(cases[i].attend())
    threads = [threading.Thread(target=run, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    torch.cuda.synchronize()
    for g, w in zip(got, want):
        assert len(g) == 30
        for out, lse in g:
            assert torch.equal(out, w[0]) and torch.equal(lse, w[1])


def test_workspaces_are_refused():
    c = Case(25, [50], 1, 4)
    ws = c.cache.workspace(1, 1, 4)
    for bad in (ws.cpu(), ws.numel(), ws[: 1 << 20].view(torch.float32), ws.view(1, -1),
                torch.empty(2 * ws.numel(), dtype=torch.uint8, device="cuda")[::2]):
        with pytest.raises(ValueError):
            c.attend(workspace=bad)
    with pytest.raises(ess.EssError):
        c.attend(workspace=ws[16:])                  # not 256-byte aligned
    c.check(*c.attend(workspace=ws))


def test_written_rows_are_attended_and_read():
    """Prompt rows and then a decode step's rows into the cache, attention over
    all of them, and the rows read back: as a server runs them."""
    from host_latent_cache_gb300.rows import RowCache
    g = torch.Generator(device="cuda").manual_seed(17)
    page, lens = 64, [130, 257]
    table = torch.tensor([[4, 0, 7, 9, 11], [1, 8, 2, 3, 5]], dtype=torch.int32, device="cuda")
    cache = RowCache(torch.zeros(12 * page, 400, dtype=torch.uint8, device="cuda"), "q4", page=page)
    gamma = torch.ones(512, dtype=torch.bfloat16, device="cuda")
    freq = [10000.0 ** (-i / 32.0) for i in range(32)]

    def put(b, t0, n):
        t = torch.arange(t0, t0 + n, device="cuda")
        slots = table[b, t // page].long() * page + t % page
        kv = torch.randn(n, 576, generator=g, device="cuda").to(torch.bfloat16)
        cache.write(kv, slots, gamma=gamma, pos=t.int(), inv_freq=freq)
        return slots
    slots = [put(b, 0, n) for b, n in enumerate(lens)]
    for step in range(3):
        for b in range(2):
            slots[b] = torch.cat([slots[b], put(b, lens[b] + step, 1)])
        T = torch.tensor([n + step + 1 for n in lens], dtype=torch.int32, device="cuda")
        q = torch.randn(2, 1, 32, 576, generator=g, device="cuda").to(torch.bfloat16)
        out, lse = cache.attend(q, table, T, 1 / 24.0)
        for b in range(2):
            k = cache.read(slots[b]).double()
            z = q[b, 0].double() @ k.T / 24.0
            want = torch.softmax(z, 1) @ k[:, :512]
            size = torch.softmax(z, 1) @ k[:, :512].abs()
            dz = 576 * 2.0 ** -24 * (q[b, 0].double().abs() @ k.abs().T).amax(1, keepdim=True) / 24
            tol = (2 * dz + 2.0 ** -11 + 2.0 ** -18) * size + 2.0 ** -8 * want.abs()
            assert ((out[b, 0].double() - want).abs() <= tol).all()
            assert ((lse[b, 0].double() - torch.logsumexp(z, 1)).abs() <= dz[:, 0] + 2.0 ** -16).all()
    assert cache.poll() == ess.ESS_OK


@pytest.mark.parametrize("mtp,lens", [(1, [3000, 130, 2048]), (2, [700, 2, 2900])])
def test_attention_over_the_indexers_list(mtp, lens):
    """The indexer's selection straight into the attention over a 4-bit copy of the
    same context, as a layer runs them, step after step on one stream."""
    from host_latent_cache_gb300 import workloads as W
    from host_latent_cache_gb300.rows import RowCache
    from host_latent_cache_gb300.session import Session
    cfg = W.v32_32k().replace(batch=3, T=3200, k=512, C=2048, mtp=mtp, mla_heads=32, layers=1,
                              T_per_req=lens)
    ld = W.gen_layer(cfg)
    sess = Session(cfg, [ld])
    n, page = ld.latent.shape[1], cfg.page
    per = n // page
    table = ld.page_table + per * np.arange(3, dtype=np.int32)[:, None]
    t = np.arange(n)
    slots = table[:, t // page].astype(np.int64) * page + t % page
    cache = RowCache(torch.zeros(3 * n, 400, dtype=torch.uint8, device="cuda"), "q4", page=page)
    kv = torch.from_numpy(ld.latent.view(np.int16)).cuda().view(torch.bfloat16)
    for b in range(3):
        cache.write(kv[b], torch.from_numpy(slots[b]).cuda())
    raw = cache.rows.cpu().numpy()
    T = torch.tensor(lens, dtype=torch.int32, device="cuda")
    dev_table = torch.from_numpy(table).cuda()
    qs = W.QueryStream(cfg)
    for _ in range(3):
        _, enc, qm = qs.next()
        qd, wd, qmd = sess.device_inputs(enc, W.head_weights(cfg, ld.w), qm)
        q = qmd.view(torch.bfloat16).view(3, mtp, 32, 576)
        sess.indexer_topk(0, qd, wd)
        out, lse = cache.attend(q, dev_table, T, cfg.sm_scale, tokens=sess.topk_idx)
        torch.cuda.synchronize()
        assert sess.poll() == ess.ESS_OK and cache.poll() == ess.ESS_OK
        top = sess.topk_idx.cpu().numpy()
        qf = q.double().cpu().numpy()
        for b in range(3):
            for m in range(mtp):
                at = top[b, m, :min(512, lens[b])].astype(np.int64)
                assert len(set(at.tolist())) == len(at) and at.max() < lens[b]
                k = R.row_values(raw[slots[b, at]], "q4")
                want, wl, size = R.attention(qf[b, m], k, cfg.sm_scale, np.ones((32, len(at)), bool))
                dz = 576 * 2.0 ** -24 * (np.abs(qf[b, m]) @ np.abs(k).T).max(axis=1) * cfg.sm_scale
                tol = (2 * dz[:, None] + 2.0 ** -11 + 2.0 ** -18) * size + 2.0 ** -8 * np.abs(want) \
                    + 2.0 ** -32 * np.abs(k[:, :512]).sum(axis=0)
                assert (np.abs(out[b, m].double().cpu().numpy() - want) <= tol).all()
                gl = lse[b, m].double().cpu().numpy()
                assert (np.abs(gl - wl) <= dz + 2.0 ** -20 * (1 + np.abs(wl))).all()
    sess.close()
