"""Lists whose tokens do not stand at their front: a query token that sees s tokens attends to
the first s entries, and nothing is said of those behind."""
import numpy as np
import pytest

from host_latent_cache_gb300 import ess
from test_gpu_chunk import Chunks, _lib   # noqa: F401  (the fixture builds the library)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("heads", [16, 128])
@pytest.mark.parametrize("where", ["end", "between", "far"])
def test_tokens_behind_the_ones_seen_are_not_read(where, heads):
    k = 300
    c = Chunks(heads, [(90, 90), (5, 700), (40, 200)], heads)
    tokens = np.full((c.total, k), -1, dtype=np.int32)
    for b, (n, T) in enumerate(c.requests):
        for i in range(n):
            sees = T - n + i + 1
            some = c.rng.permutation(sees)[:k]
            at = {"end": np.arange(k - some.size, k), "between": np.arange(some.size) * (k // some.size),
                  "far": np.arange(some.size)}[where]
            row = tokens[c.cu[b] + i]
            row[at] = some
            if where == "far" and sees < k:
                row[sees:] = 1 << 30      # no token at all, where nothing is read
    out, lse = c.attend(tokens)
    assert c.cache.poll() == ess.ESS_OK
    c.check(out, lse, tokens, some=0.4)   # of the first min(k, s) entries
    if where == "end":                    # 90 new tokens without a prefix: none of the 300 entries is among the first 90
        assert (out[:90] == 0).all() and (lse[:90] == -float("inf")).all()
