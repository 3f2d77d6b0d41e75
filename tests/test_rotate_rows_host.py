"""A rotation whose result rows would meet is refused, without a GPU."""
import ctypes

import pytest

from host_latent_cache_gb300 import build as B
from host_latent_cache_gb300 import ess

P = ctypes.c_void_p
FREQ = (ctypes.c_double * 32)(*[1.0] * 32)


def rotate(n, heads, row, head):
    return ess.load().ess_rotate(P(1 << 20), 64 * heads, 64, n, heads, FREQ, P(1 << 20), 1, None, 0, P(1 << 40), row, head,
                                 None)


def meet(n, heads, row, head):
    at = sorted(i * row + j * head for i in range(n) for j in range(heads))
    return any(b - a < 64 for a, b in zip(at, at[1:]))


@pytest.mark.parametrize("n,heads,row,head", [
    (2, 2, 64, 64), (3, 5, 64, 64), (2, 3, 128, 64), (4, 2, 64, 192), (2, 4, 192, 64), (2, 2, 64, 72), (2, 2, 120, 64),
    (2, 2, 64, 0), (2, 1, 0, 64), (1, 2, 64, 56), (2, 1, 56, 64), (2, 2, 0, 128), (2, 2, -128, 64), (2, 2, 128, -64),
    (1 << 20, 1 << 10, 64, 64), (1 << 30, 4, 1 << 40, 1 << 39), (1 << 20, 1 << 10, 1 << 62, 1 << 62),
])
def test_rows_that_meet_are_refused(n, heads, row, head):
    B.build()
    assert n * heads > 100 or min(row, head) < 0 or meet(n, heads, row, head)
    assert rotate(n, heads, row, head) == ess.ESS_ERR_INVALID_ARG


@pytest.mark.parametrize("heads,row,head", [(3, 192, 64), (1, 64, 0), (8, 8 * 576, 576), (2, 200, 64), (3, 72 * 3, 72)])
def test_rows_that_keep_apart_pass_that_check(heads, row, head):
    """More tokens than the kernel takes are unsupported, which is seen behind it."""
    B.build()
    assert not meet(7, heads, row, head)
    assert rotate((1 << 31) // -(-heads // 4) + 1, heads, row, head) == ess.ESS_ERR_UNSUPPORTED
