"""The row cache's oracle is pinned to the formats' definitions, and the C ABI
refuses what its kernels do not take, all without a GPU."""
import ctypes
import os
import re

import numpy as np
import pytest

from host_latent_cache_gb300 import build as B
from host_latent_cache_gb300 import ess
from oracle import compact_row as X
from oracle import row_cache as R


@pytest.fixture(scope="module")
def lib():
    B.build()
    return ess.load()


# ------------------------------------------------------------------ the oracle

def test_e2m1_codes_are_the_nearest_levels():
    rng = np.random.default_rng(1)
    a = np.concatenate([rng.uniform(0, 8, 4000), R.E2M1, (R.E2M1[1:] + R.E2M1[:-1]) / 2])
    code = R.nearest_code(a, R.E2M1)
    for x, c in zip(a, code):
        d = np.abs(R.E2M1 - x)
        best = np.flatnonzero(d == d.min())
        assert c in best and (len(best) == 1 or c % 2 == 0), (x, c)


def test_e4m3_codes_agree_with_the_compact_rows_encoder():
    rng = np.random.default_rng(2)
    a = np.concatenate([rng.uniform(0, 500, 500), 2.0 ** rng.uniform(-12, 9, 500), R.E4M3[::7]])
    code = R.nearest_code(a, R.E4M3)
    assert [int(c) for c in code] == [X.e4m3_encode(float(x)) for x in a]


@pytest.mark.parametrize("amax,exp", [(6.0, 0), (6.0001, 1), (3.0, -1), (0.0, 0), (1e-30, -23),
                                      (1e9, 13), (5.0, 0)])
def test_q4_scales(amax, exp):
    y = np.zeros((1, 512))
    y[0, 40] = -amax
    packed, exps = R.q4_encode(y)
    assert exps[0, 1] == exp + 127 and exps[0, 0] == 127
    v = R.q4_decode(packed, exps)
    assert np.all(v[0, :32] == 0) and np.all(v[0, 64:] == 0)
    if amax in (6.0, 3.0):
        assert v[0, 40] == -amax


def test_q4_rows_keep_their_values_when_encoded_again():
    rng = np.random.default_rng(3)
    y = rng.normal(size=(50, 512)) * 2.0 ** rng.integers(-20, 10, size=(50, 1))
    p, e = R.q4_encode(y)
    v = R.q4_decode(p, e)
    # a block whose largest code is below 6 may take a smaller scale, with the same values
    p2, e2 = R.q4_encode(v)
    assert np.array_equal(R.q4_decode(p2, e2), v)
    assert np.array_equal(v.astype(np.float16).astype(np.float64), v)   # exact in fp16


def test_attention_oracle_is_a_softmax():
    rng = np.random.default_rng(4)
    q, k = rng.normal(size=(3, 576)), rng.normal(size=(7, 576))
    keep = np.ones((3, 7), bool)
    keep[1, 3:] = False
    keep[2, :] = False
    out, lse, _ = R.attention(q, k, 0.05, keep)
    s = float(np.float32(0.05))
    for i, n in ((0, 7), (1, 3)):
        w = np.exp(k[:n] @ q[i] * s)
        assert np.allclose(out[i], (w[:, None] * k[:n, :512]).sum(0) / w.sum(), rtol=1e-12)
        assert np.isclose(lse[i], np.log(w.sum()), rtol=1e-12)
    assert np.all(out[2] == 0) and lse[2] == -np.inf


def test_rotation_oracle_at_far_positions():
    k = np.zeros((2, 64))
    k[:, 0] = 1.0
    f = [1.0] + [0.5] * 31
    out = R.rotate(k, np.array([1, 1000003]), f, False)
    assert np.allclose(out[:, 0], [np.cos(1.0), np.cos(1000003.0)], atol=1e-9)
    assert np.allclose(out[:, 1], [np.sin(1.0), np.sin(1000003.0)], atol=1e-9)


# ------------------------------------------------------------------ the sources

def test_kernels_that_start_early_take_no_read_only_pointers():
    """The row cache's kernels start while the kernel before them may still write
    what they read; a load through a __restrict__ const pointer (or __ldg) may be
    moved ahead of the wait for it."""
    for name in ("ess_rows.cu", "ess_rows.cuh", "ess_mla.cu"):
        with open(os.path.join(B.CSRC, name)) as f:
            code = re.sub(r"//[^\n]*", "", f.read())
        assert not re.search(r"__restrict__|__ldg|ld\.global\.nc", code), name


# ------------------------------------------------------------------ refusals

P = ctypes.c_void_p
A16, A256, BAD = P(1 << 20), P(1 << 20), P((1 << 20) + 8)   # never dereferenced: refused first
FREQ = (ctypes.c_double * 32)(*[1.0] * 32)


def test_row_bytes(lib):
    assert [ess.ess_row_bytes(f) for f in range(3)] == [1152, 656, 400]
    n = ctypes.c_int32(0)
    assert lib.ess_row_bytes(3, ctypes.byref(n)) == ess.ESS_ERR_INVALID_ARG
    assert lib.ess_row_bytes(0, None) == ess.ESS_ERR_INVALID_ARG


@pytest.mark.parametrize("status,taken", [(None, A16), (A16, None), (P((1 << 20) + 2), A16),
                                          (A16, P((1 << 20) + 2))])
def test_status_take_refusals(lib, status, taken):
    assert lib.ess_status_take(status, taken, None) == ess.ESS_ERR_INVALID_ARG


@pytest.mark.parametrize("page", [0, -1, 1 << 31, (1 << 32) + 64])
def test_pages_past_32_bits_are_refused(page):
    from host_latent_cache_gb300 import rows
    with pytest.raises(ValueError, match="a page has"):
        rows.RowCache(None, "q4", page=page)


WRITE = dict(kv=A16, stride=576, n=4, gamma=A16, eps=1e-6, freq=FREQ, pos=A16, pairs=0, slots=A16,
             rows=A16, n_rows=64, fmt=2)


@pytest.mark.parametrize("change", [
    dict(kv=None), dict(kv=BAD), dict(stride=568), dict(stride=577), dict(n=-1), dict(gamma=BAD),
    dict(eps=-1.0), dict(eps=float("nan")), dict(pos=None), dict(pairs=2), dict(slots=None),
    dict(rows=None), dict(rows=BAD), dict(n_rows=-1), dict(fmt=3), dict(fmt=-1),
    dict(freq=(ctypes.c_double * 32)(*[float("inf")] * 32)),
], ids=lambda c: "-".join(f"{k}" for k in c))
def test_write_refusals(lib, change):
    a = {**WRITE, **change}
    got = lib.ess_cache_write(a["kv"], a["stride"], a["n"], a["gamma"], a["eps"], a["freq"],
                              a["pos"], a["pairs"], a["slots"], a["rows"], a["n_rows"], a["fmt"],
                              None, None)
    assert got == ess.ESS_ERR_INVALID_ARG


def test_nothing_to_do_needs_no_buffers(lib):
    assert lib.ess_cache_write(None, 576, 0, None, 1e-6, None, None, 0, None, None, 0, 2, None,
                               None) == ess.ESS_OK
    assert lib.ess_cache_read(None, 0, 1, None, 0, None, None, None) == ess.ESS_OK
    assert lib.ess_norm_quant(None, 128, None, 0, None, 1e-6, 0, 128, None, None, None,
                              None) == ess.ESS_OK


READ = dict(rows=A16, n_rows=64, fmt=2, slots=A16, n=4, out=A16)


@pytest.mark.parametrize("change", [dict(rows=None), dict(rows=BAD), dict(n_rows=-1), dict(fmt=3),
                                    dict(slots=None), dict(n=-1), dict(out=None), dict(out=BAD)],
                         ids=lambda c: "-".join(c))
def test_read_refusals(lib, change):
    a = {**READ, **change}
    assert lib.ess_cache_read(a["rows"], a["n_rows"], a["fmt"], a["slots"], a["n"], a["out"], None,
                              None) == ess.ESS_ERR_INVALID_ARG


MLA = dict(q=A16, rows=A16, n_rows=640, fmt=2, table=A16, max_pages=10, page=64, T=A16, batch=1,
           ways=1, heads=16, tokens=None, k=0, scale=0.04, out=A16, ws=A256, ws_bytes=1 << 40)


@pytest.mark.parametrize("change,code", [
    (dict(q=None), 1), (dict(q=BAD), 1), (dict(rows=None), 1), (dict(rows=BAD), 1),
    (dict(n_rows=0), 1), (dict(fmt=3), 1), (dict(fmt=0), 3), (dict(fmt=1), 3),
    (dict(n_rows=1 << 31), 3), (dict(table=None), 1), (dict(max_pages=0), 1), (dict(page=0), 1),
    (dict(max_pages=1 << 26, page=64), 3), (dict(T=None), 1), (dict(batch=0), 1), (dict(ways=0), 1),
    (dict(ways=5), 3), (dict(heads=0), 1), (dict(heads=129), 3), (dict(tokens=A16, k=0), 1),
    (dict(scale=0.0), 1), (dict(scale=float("nan")), 1), (dict(scale=float("inf")), 1),
    (dict(out=None), 1), (dict(out=BAD), 1), (dict(ws=None), 1), (dict(ws=BAD), 1),
    (dict(ws_bytes=0), 4),
], ids=lambda c: "-".join(c) if isinstance(c, dict) else str(c))
def test_attention_refusals(lib, change, code):
    a = {**MLA, **change}
    got = lib.ess_cache_mla(a["q"], a["rows"], a["n_rows"], a["fmt"], a["table"], a["max_pages"],
                            a["page"], a["T"], a["batch"], a["ways"], a["heads"], a["tokens"],
                            a["k"], a["scale"], a["out"], None, a["ws"], a["ws_bytes"], None, None)
    assert got == code


def test_attention_workspace_sizes(lib):
    n = ctypes.c_size_t(0)
    assert lib.ess_cache_mla_bytes(8, 1, 128, ctypes.byref(n)) == ess.ESS_OK and n.value > 0
    assert lib.ess_cache_mla_bytes(8, 1, 128, None) == ess.ESS_ERR_INVALID_ARG
    assert lib.ess_cache_mla_bytes(0, 1, 128, ctypes.byref(n)) == ess.ESS_ERR_INVALID_ARG
    assert lib.ess_cache_mla_bytes(1, 5, 128, ctypes.byref(n)) == ess.ESS_ERR_UNSUPPORTED
    assert lib.ess_cache_mla_bytes(1, 1, 129, ctypes.byref(n)) == ess.ESS_ERR_UNSUPPORTED


@pytest.mark.parametrize("name", ["table", "T", "tokens", "lse", "status"])
def test_attention_refuses_odd_addresses(lib, name):
    odd = P((1 << 20) + 2)
    a = {**MLA, "k": 4, "lse": None, "status": None, name: odd}
    got = lib.ess_cache_mla(a["q"], a["rows"], a["n_rows"], a["fmt"], a["table"], a["max_pages"],
                            a["page"], a["T"], a["batch"], a["ways"], a["heads"], a["tokens"],
                            a["k"], a["scale"], a["out"], a["lse"], a["ws"], a["ws_bytes"],
                            a["status"], None)
    assert got == ess.ESS_ERR_INVALID_ARG


@pytest.mark.parametrize("name,at", [("slots", 4), ("pos", 2), ("status", 2)])
def test_row_calls_refuse_odd_addresses(lib, name, at):
    a = {**WRITE, "status": None, name: P((1 << 20) + at)}
    got = lib.ess_cache_write(a["kv"], a["stride"], a["n"], a["gamma"], a["eps"], a["freq"],
                              a["pos"], a["pairs"], a["slots"], a["rows"], a["n_rows"], a["fmt"],
                              a["status"], None)
    assert got == ess.ESS_ERR_INVALID_ARG
    if name != "pos":
        a = {**READ, "status": None, name: P((1 << 20) + at)}
        got = lib.ess_cache_read(a["rows"], a["n_rows"], a["fmt"], a["slots"], a["n"], a["out"],
                                 a["status"], None)
        assert got == ess.ESS_ERR_INVALID_ARG


NORM = dict(x=A16, xs=128, res=A16, rs=128, gamma=A16, eps=1e-6, n=4, dim=128, out=A16, codes=A16,
            scales=A16)


def test_norm_output_over_x_needs_one_stride(lib):
    """Over x the sums may go only where x's own rows lie."""
    a = {**NORM, "xs": 256, "out": A16, "res": P(1 << 24)}
    got = lib.ess_norm_quant(a["x"], a["xs"], a["res"], a["rs"], a["gamma"], a["eps"], a["n"],
                             a["dim"], a["out"], a["codes"], a["scales"], None)
    assert got == ess.ESS_ERR_INVALID_ARG


@pytest.mark.parametrize("change,code", [
    (dict(x=None), 1), (dict(x=BAD), 1), (dict(xs=120), 1), (dict(xs=129), 1), (dict(rs=120), 1),
    (dict(rs=130), 1), (dict(res=BAD), 1), (dict(gamma=None), 1), (dict(gamma=BAD), 1),
    (dict(eps=-1e-6), 1), (dict(n=-1), 1), (dict(dim=0), 1), (dict(dim=100), 3),
    (dict(dim=16392, xs=16392, rs=16392), 3), (dict(out=BAD), 1), (dict(res=None), 1),
    (dict(codes=None), 1), (dict(codes=BAD), 1), (dict(scales=None), 1),
], ids=lambda c: "-".join(c) if isinstance(c, dict) else str(c))
def test_norm_refusals(lib, change, code):
    a = {**NORM, **change}
    got = lib.ess_norm_quant(a["x"], a["xs"], a["res"], a["rs"], a["gamma"], a["eps"], a["n"],
                             a["dim"], a["out"], a["codes"], a["scales"], None)
    assert got == code
