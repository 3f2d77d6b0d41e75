"""A prompt chunk's path as a layer runs it: norm, 8-bit projections, rotation on three
axes, cache rows, attention of the chunk, 8-bit output projection; and an indexer right
behind the kernels that may write its keys."""
import math

import numpy as np
import pytest
import torch

from host_latent_cache_gb300 import ess
from host_latent_cache_gb300 import workloads as W
from oracle import row_cache as R

pytestmark = pytest.mark.gpu
HEADS, DIM, PAGE = 16, 1024, 64
FREQ = [10000.0 ** (-i / 32.0) for i in range(32)]
AXES = [0] * 16 + [1, 2] * 8


@pytest.fixture(scope="module", autouse=True)
def _lib():
    from host_latent_cache_gb300 import build as B
    B.build()
    assert torch.cuda.is_available()
    ess.load()


class Layer:
    """Weights and a cache of two requests, and one pass of a chunk through them."""

    def __init__(self):
        from host_latent_cache_gb300.products import Weight8
        from host_latent_cache_gb300.rows import RowCache
        g = torch.Generator(device="cuda").manual_seed(7)
        rand = lambda *s: torch.randn(*s, generator=g, device="cuda")
        self.rand = rand
        self.gamma = (0.5 + torch.rand(DIM, generator=g, device="cuda")).to(torch.bfloat16)
        self.kv_gamma = (0.5 + torch.rand(512, generator=g, device="cuda")).to(torch.bfloat16)
        self.w_kv = Weight8.of((rand(576, DIM) / math.sqrt(DIM)).to(torch.bfloat16))
        self.w_q = Weight8.of((rand(HEADS * 576, DIM) / math.sqrt(DIM)).to(torch.bfloat16))
        self.w_o = Weight8.of((rand(DIM, HEADS * 512) / math.sqrt(HEADS * 512)).to(torch.bfloat16))
        self.cache = RowCache(torch.zeros(40 * PAGE, 400, dtype=torch.uint8, device="cuda"), "q4", page=PAGE)
        self.table = torch.randperm(40, generator=g, device="cuda").view(2, 20).to(torch.int32)

    def run(self, h, res, cu, T, pos, slots):
        """h, res bf16 [n][DIM]: what a user's program does with a chunk."""
        from host_latent_cache_gb300.products import quant_q8
        from host_latent_cache_gb300.rows import norm_q8, rotate
        n = h.shape[0]
        codes, scales, res = norm_q8(h, self.gamma, residual=res)
        kv = self.w_kv.product(codes, scales)
        q = self.w_q.product(codes, scales).view(n, HEADS, 576)
        self.cache.write(kv, slots, gamma=self.kv_gamma, pos=pos, inv_freq=FREQ, axes=AXES)
        rotate(q[:, :, 512:], pos, FREQ, axes=AXES, out=q[:, :, 512:])
        out, lse = self.cache.attend_chunk(q, cu, self.table, T, 1.0 / 24.0)
        oc, os_ = quant_q8(out.view(n, HEADS * 512))
        y = self.w_o.product(oc, os_, dtype=torch.float32)
        return {"res": res, "kv": kv, "q": q, "out": out, "lse": lse, "y": y}

    def chunk(self, news, before):
        """Inputs of a chunk with news[b] new tokens after before[b]."""
        n = sum(news)
        T = [a + b for a, b in zip(news, before)]
        t = np.concatenate([np.arange(b, b + a) for a, b in zip(news, before)])
        b = np.repeat([0, 1], news)
        slots = self.table.cpu().numpy()[b, t // PAGE].astype(np.int64) * PAGE + t % PAGE
        dev = lambda a, d: torch.from_numpy(np.ascontiguousarray(a)).to(d).cuda()
        return dict(h=self.rand(n, DIM).to(torch.bfloat16), res=self.rand(n, DIM).to(torch.bfloat16),
                    cu=dev(np.array([0, news[0], n]), torch.int32), T=dev(np.array(T), torch.int32),
                    pos=dev(np.stack([t, t // 24, t % 24]), torch.int32), slots=dev(slots, torch.int64))


def test_chunks_one_after_another():
    layer = Layer()
    before = [0, 0]
    for news in ([70, 130], [1, 64], [0, 5], [200, 1]):
        x = layer.chunk(news, before)
        got = layer.run(**x)
        torch.cuda.synchronize()
        assert torch.equal(got["res"], (x["h"].float() + x["res"].float()).to(torch.bfloat16))
        # the cache's rows of this chunk, read back, are the projection's normed and turned
        kv = got["kv"].double().cpu().numpy()
        pos = x["pos"].cpu().numpy()
        per = [R.rotate(kv[:, 512:], p, FREQ, False) for p in pos]
        turned = np.empty_like(per[0])
        for i, a in enumerate(AXES):
            turned[:, 2 * i:2 * i + 2] = per[a][:, 2 * i:2 * i + 2]
        rows = layer.cache.read(x["slots"]).double().cpu().numpy()
        tol = 2.0 ** -19 * np.abs(kv[:, 512:]).max(axis=1, keepdims=True) + 2.0 ** -8 * np.abs(turned) + 2.0 ** -134
        assert (np.abs(rows[:, 512:] - turned) <= tol).all()
        y = R.rms_norm(kv[:, :512], layer.kv_gamma.double().cpu().numpy(), 1e-6)
        packed, exps = R.q4_encode(y)
        want = R.q4_decode(packed, exps)
        # a value next to a border between codes may take either neighbour
        assert (rows[:, :512] != want).mean() < 1e-3
        # attention over what the cache holds
        q = got["q"].double().cpu().numpy()
        table, at = layer.table.cpu().numpy(), 0
        for b in range(2):
            T = before[b] + news[b]
            t = np.arange(T)
            k = R.row_values(layer.cache.rows.cpu().numpy()[table[b, t // PAGE].astype(np.int64) * PAGE + t % PAGE], "q4")
            for i in range(news[b]):
                sees = before[b] + i + 1
                o, l, size = R.attention(q[at], k[:sees], 1.0 / 24.0, np.ones((HEADS, sees), bool))
                dz = (576 * 2.0 ** -24) * (np.abs(q[at]) @ np.abs(k[:sees]).T).max(axis=1) / 24.0
                err = np.abs(got["out"][at].double().cpu().numpy() - o)
                assert (err <= (2 * dz[:, None] + 2.0 ** -11 + 2.0 ** -18) * size + 2.0 ** -8 * np.abs(o)
                        + 2.0 ** -32 * np.abs(k[:sees, :512]).sum(axis=0)).all()
                assert (np.abs(got["lse"][at].double().cpu().numpy() - l) <= dz + 2.0 ** -20 * (1 + np.abs(l))).all()
                at += 1
        before = [a + b for a, b in zip(before, news)]
    assert layer.cache.poll() == ess.ESS_OK
    assert all(w.poll() == ess.ESS_OK for w in (layer.w_kv, layer.w_q, layer.w_o))


def test_a_captured_chunk_on_another_stream():
    """A pass captured on a side stream, replayed on other inputs and lengths, leaves what
    eager passes leave, bit for bit."""
    eager, caught = Layer(), Layer()
    xs = [eager.chunk([70, 130], [0, 0]), eager.chunk([100, 100], [70, 130]), eager.chunk([5, 195], [170, 230])]
    bufs = {k: v.clone() for k, v in xs[0].items()}
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        caught.run(**bufs)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=side):
            got = caught.run(**bufs)
    torch.cuda.synchronize()
    for x in xs:
        want = eager.run(**x)
        for k, v in bufs.items():
            v.copy_(x[k])
        torch.cuda.synchronize()
        with torch.cuda.stream(side):
            graph.replay()
        torch.cuda.synchronize()
        for k in want:
            assert torch.equal(got[k], want[k]), k
        assert torch.equal(eager.cache.rows, caught.cache.rows)
    assert caught.cache.poll() == ess.ESS_OK


@pytest.mark.parametrize("how", ["eager", "graph"])
@pytest.mark.parametrize("writer", ["quant", "rotate", "product"])
def test_an_indexer_right_behind_what_writes_its_keys(writer, how):
    """Keys written by the kernel next ahead on the stream are the ones that are scored."""
    from host_latent_cache_gb300 import products, rows
    from host_latent_cache_gb300.session import Session
    if writer == "quant":
        cfg = W.v32_32k().replace(batch=2, T=32768, k=512, C=2048, mtp=1, mla_heads=16, layers=1)
    else:
        cfg = W.tiny().replace(T=32768, C=2048)
    ld = W.gen_layer(cfg)
    sess = Session(cfg, [ld])
    raw_keys = sess.keys[0].view(torch.uint8)
    g = torch.Generator(device="cuda").manual_seed(3)
    if writer == "quant":
        keys, scale = raw_keys.view(torch.float8_e4m3fn).view(-1, 128), sess.scale[0].view(-1, 1)
        raws = [torch.randn(keys.shape, generator=g, device="cuda").to(torch.bfloat16) for _ in range(3)]
        raw = torch.empty_like(raws[0])
        write = lambda: products.quant_q8(raw, codes=keys, scales=scale)
    elif writer == "rotate":
        keys = raw_keys.view(torch.bfloat16).view(-1, 1, 64)
        pos = torch.arange(keys.shape[0], device="cuda", dtype=torch.int32)
        raws = [torch.randn(keys.shape, generator=g, device="cuda").to(torch.bfloat16) for _ in range(3)]
        raw = torch.empty_like(raws[0])
        write = lambda: rows.rotate(raw, pos, FREQ, out=keys)
    else:
        keys = raw_keys.view(torch.bfloat16).view(-1, 64)
        weight = products.Weight8.of(torch.randn(64, 256, generator=g, device="cuda").to(torch.bfloat16))
        raws = [products.quant_q8(torch.randn(keys.shape[0], 256, generator=g, device="cuda").to(torch.bfloat16))[0]
                for _ in range(3)]
        raw, ones = torch.empty_like(raws[0]), torch.ones(keys.shape[0], 2, device="cuda")
        write = lambda: weight.product(raw, ones, out=keys)
    q, enc, qm = W.QueryStream(cfg).next()
    qd, wd, _ = sess.device_inputs(enc, W.head_weights(cfg, ld.w), qm)
    want = []
    for r in raws:
        raw.copy_(r)
        write()
        torch.cuda.synchronize()
        sess.scores_only(0, qd, wd)
        torch.cuda.synchronize()
        want.append(sess.scores.clone())
    assert not torch.equal(want[0], want[1])
    if how == "graph":
        sess.scores_only(0, qd, wd)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            write()
            sess.scores_only(0, qd, wd, torch.cuda.current_stream())
    for i in range(24):
        raw.copy_(raws[i % 3])
        torch.cuda.synchronize()
        if how == "graph":
            graph.replay()
        else:
            write()
            sess.scores_only(0, qd, wd)
        torch.cuda.synchronize()
        assert torch.equal(sess.scores, want[i % 3]), i
    assert sess.poll() == ess.ESS_OK
    sess.close()
