"""The C ABI of the prompt chunk's path (8-bit products, rotation on several axes, chunk
attention) refuses what its kernels do not take, without a GPU."""
import ctypes
import os
import re

import pytest

from host_latent_cache_gb300 import build as B
from host_latent_cache_gb300 import ess

P = ctypes.c_void_p
A16, A256, BAD = P(1 << 20), P(1 << 20), P((1 << 20) + 8)   # never dereferenced: refused first
ODD = P((1 << 20) + 2)
FREQ = (ctypes.c_double * 32)(*[1.0] * 32)


def axis(*changes):
    a = [0] * 32
    for i, v in changes:
        a[i] = v
    return (ctypes.c_int32 * 32)(*a)


@pytest.fixture(scope="module")
def lib():
    B.build()
    return ess.load()


def ids(c):
    return "-".join(c) if isinstance(c, dict) else str(c)


def test_kernels_that_start_early_take_no_read_only_pointers():
    with open(os.path.join(B.CSRC, "ess_product.cu")) as f:
        code = re.sub(r"//[^\n]*", "", f.read())
    assert not re.search(r"__restrict__|__ldg|ld\.global\.nc", code)


QUANT = dict(x=A16, stride=256, n=4, dim=256, square=0, codes=A16, scales=A16)


@pytest.mark.parametrize("change,code", [
    (dict(x=None), 1), (dict(x=BAD), 1), (dict(stride=248), 1), (dict(stride=257), 1), (dict(n=-1), 1),
    (dict(dim=0), 1), (dict(dim=-8), 1), (dict(square=2), 1), (dict(codes=None), 1), (dict(codes=BAD), 1),
    (dict(scales=None), 1), (dict(scales=ODD), 1), (dict(dim=100), 3), (dict(n=1 << 31), 1),
    (dict(square=1, n=128 * 65535 + 1), 3),
], ids=ids)
def test_quant_refusals(lib, change, code):
    a = {**QUANT, **change}
    assert lib.ess_quant(a["x"], a["stride"], a["n"], a["dim"], a["square"], a["codes"], a["scales"], None) == code


PRODUCT = dict(x=A16, xs=A16, n=4, w=A16, ws=A16, outs=128, ins=256, out=A16, stride=128, fp32=0, status=None)


@pytest.mark.parametrize("change,code", [
    (dict(x=None), 1), (dict(x=BAD), 1), (dict(xs=None), 1), (dict(xs=ODD), 1), (dict(n=-1), 1),
    (dict(w=None), 1), (dict(w=BAD), 1), (dict(ws=None), 1), (dict(ws=ODD), 1), (dict(outs=0), 1),
    (dict(ins=0), 1), (dict(ins=24), 3), (dict(out=None), 1), (dict(out=P((1 << 20) + 1)), 1),
    (dict(out=ODD, fp32=1), 1), (dict(stride=127), 1), (dict(fp32=2), 1), (dict(status=ODD), 1),
    (dict(n=1 << 31), 3), (dict(ins=(1 << 26) + 16), 3),
], ids=ids)
def test_product_refusals(lib, change, code):
    a = {**PRODUCT, **change}
    assert lib.ess_product(a["x"], a["xs"], a["n"], a["w"], a["ws"], a["outs"], a["ins"], a["out"], a["stride"],
                           a["fp32"], a["status"], None) == code


WRITE = dict(kv=A16, freq=FREQ, pos=A16, axes=3, axis=axis(), status=None)


@pytest.mark.parametrize("change", [dict(axes=0), dict(axes=-1), dict(axis=axis((3, 3))), dict(axis=axis((31, -1))),
                                    dict(pos=None), dict(pos=ODD), dict(kv=None)], ids=ids)
def test_write_with_axes_refusals(lib, change):
    a = {**WRITE, **change}
    assert lib.ess_cache_write_axes(a["kv"], 576, 4, A16, 1e-6, a["freq"], a["pos"], a["axes"], a["axis"], 0, A16,
                                    A16, 64, 0, a["status"], None) == ess.ESS_ERR_INVALID_ARG


ROTATE = dict(x=A16, row=128, head=64, n=4, heads=2, freq=FREQ, pos=A16, axes=1, axis=None, pairs=0,
              out=P(1 << 21), orow=128, ohead=64)


@pytest.mark.parametrize("change,code", [
    (dict(x=None), 1), (dict(x=BAD), 1), (dict(row=132), 1), (dict(row=-128), 1), (dict(head=66), 1), (dict(head=-64), 1),
    (dict(n=-1), 1), (dict(heads=0), 1), (dict(freq=None), 1), (dict(freq=(ctypes.c_double * 32)(*[float("nan")] * 32)), 1),
    (dict(pos=None), 1), (dict(pos=ODD), 1), (dict(axes=0), 1), (dict(axis=axis((0, 1))), 1), (dict(pairs=2), 1),
    (dict(out=None), 1), (dict(out=BAD), 1), (dict(orow=130), 1), (dict(ohead=56), 1), (dict(orow=0), 1),
    (dict(out=A16, orow=256), 1), (dict(out=A16, ohead=72), 1), (dict(n=1 << 31), 3),
], ids=ids)
def test_rotate_refusals(lib, change, code):
    a = {**ROTATE, **change}
    assert lib.ess_rotate(a["x"], a["row"], a["head"], a["n"], a["heads"], a["freq"], a["pos"], a["axes"], a["axis"],
                          a["pairs"], a["out"], a["orow"], a["ohead"], None) == code


CHUNK = dict(q=A16, total=8, cu=A16, rows=A16, n_rows=640, fmt=2, table=A16, max_pages=10, page=64, T=A16, batch=1,
             heads=16, tokens=None, k=0, scale=0.04, out=A16, lse=None, ws=A256, ws_bytes=1 << 40, status=None)


@pytest.mark.parametrize("change,code", [
    (dict(q=None), 1), (dict(q=BAD), 1), (dict(total=-1), 1), (dict(cu=None), 1), (dict(cu=ODD), 1), (dict(rows=None), 1),
    (dict(rows=BAD), 1), (dict(n_rows=0), 1), (dict(fmt=3), 1), (dict(fmt=0), 3), (dict(fmt=1), 3),
    (dict(n_rows=1 << 31), 3), (dict(table=None), 1), (dict(table=ODD), 1), (dict(max_pages=0), 1), (dict(page=0), 1),
    (dict(max_pages=1 << 26, page=64), 3), (dict(T=None), 1), (dict(T=ODD), 1), (dict(batch=0), 1),
    (dict(batch=32769), 3), (dict(heads=0), 1), (dict(heads=129), 3), (dict(total=(1 << 31) // 16), 3),
    (dict(tokens=A16, k=0), 1), (dict(tokens=ODD, k=4), 1), (dict(scale=0.0), 1), (dict(scale=float("nan")), 1),
    (dict(scale=float("inf")), 1), (dict(out=None), 1), (dict(out=BAD), 1), (dict(lse=ODD), 1), (dict(ws=None), 1),
    (dict(ws=BAD), 1), (dict(ws_bytes=0), 4), (dict(status=ODD), 1),
], ids=ids)
def test_chunk_refusals(lib, change, code):
    a = {**CHUNK, **change}
    assert lib.ess_cache_chunk(a["q"], a["total"], a["cu"], a["rows"], a["n_rows"], a["fmt"], a["table"],
                               a["max_pages"], a["page"], a["T"], a["batch"], a["heads"], a["tokens"], a["k"],
                               a["scale"], a["out"], a["lse"], a["ws"], a["ws_bytes"], a["status"], None) == code


def test_chunk_workspace_size(lib):
    n = ctypes.c_size_t(0)
    assert lib.ess_cache_chunk_bytes(ctypes.byref(n)) == ess.ESS_OK and n.value > 0
    assert lib.ess_cache_chunk_bytes(None) == ess.ESS_ERR_INVALID_ARG


def test_nothing_to_do_needs_no_buffers(lib):
    assert lib.ess_quant(None, 128, 0, 128, 1, None, None, None) == ess.ESS_OK
    assert lib.ess_product(None, None, 0, None, None, 128, 256, None, 128, 0, None, None) == ess.ESS_OK
    assert lib.ess_rotate(None, 64, 64, 0, 1, FREQ, None, 1, None, 0, None, 64, 64, None) == ess.ESS_OK
    assert lib.ess_cache_chunk(None, 0, None, None, 1, 2, None, 1, 64, None, 1, 16, None, 0, 0.04, None, None, None, 0,
                               None, None) == ess.ESS_OK
