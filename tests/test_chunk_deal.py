"""How the chunk attention deals its units to pairs of CTAs, restated in 64-bit integers that
wrap as the kernel's do: every tile belongs to one pair, for any number of units that the
call takes.  More are refused.  No GPU.
"""
import os
import re

import ctypes
import numpy as np
import pytest

from host_latent_cache_gb300 import build as B
from host_latent_cache_gb300 import ess

P = ctypes.c_void_p
A16 = P(1 << 20)
THREADS = 26 * 32


def constant(name):
    with open(os.path.join(B.CSRC, "ess_mla.cu")) as f:
        m = re.search(rf"\b{name} = (\d+);", f.read())
    assert m, name
    return int(m.group(1))


def deal(units, nt, pairs, shift, cost):
    """(first tile, end tile) of each pair, tiles numbered through all units of nt tiles each;
    None where no thread of a pair's CTAs finds its first or last one."""
    i64 = np.int64
    per = -(-units // THREADS)
    v0 = np.minimum(units, np.arange(THREADS, dtype=i64) * per)
    count = np.minimum(units, v0 + per) - v0
    with np.errstate(over="ignore"):
        mine = (count * i64(nt)) + (count << i64(shift))
        total = np.add.accumulate(mine)[-1]
        before = np.add.accumulate(mine) - mine
        mask = i64((1 << shift) - 1)
        tiles = int(total & mask)
        cost = cost if tiles >= (cost + 1) * pairs else 0
        tiles_before = before & mask
        pos0 = tiles_before + i64(cost) * (before >> i64(shift))
        pos1 = pos0 + (mine & mask) + i64(cost) * (mine >> i64(shift))
        everything = tiles + cost * int(total >> i64(shift))
    busy = max(tiles, 1) if tiles < pairs else pairs
    # (as the kernel: a sum below 2^31 is divided as 32 bits without a sign)
    share = ((everything & 0xFFFFFFFF) // busy if everything < 0x7FFFFFFF else everything // busy)
    extra = everything - share * busy

    def find(at, end):
        found = [tiles] if end and at == everything else []
        for j in np.nonzero((pos0 <= at) & (at < pos1))[0]:
            off = at - int(pos0[j])
            found.append(int(tiles_before[j]) + off // (nt + cost) * nt + max(off % (nt + cost) - cost, 0))
        return found[0] if len(found) == 1 else None

    return [(find(share * p + min(p, extra), 0), find(share * (p + 1) + min(p + 1, extra), 1))
            for p in range(min(pairs, tiles) if tiles > 0 else pairs)]


def covers(units, nt, pairs, shift, cost):
    got = deal(units, nt, pairs, shift, cost)
    at = 0
    for first, end in got:
        if first != at or end is None or not first < end < first + (1 << 31):
            return False
        at = end
    return at == units * nt


UNITS = [1, 2, 75, 76, 77, 831, 832, 833, 10007, (1 << 20) - 1, 1 << 20, (1 << 20) + 1, 1 << 21, (1 << 25) + 5,
         (1 << 26) - 1]


@pytest.mark.parametrize("nt", [1, 2, 3, 16, 257])
@pytest.mark.parametrize("units", UNITS)
def test_every_tile_has_one_pair(units, nt):
    shift, cost = constant("kChunkSegShift"), constant("kChunkSegmentCost")
    assert units < 1 << (63 - shift) and units * nt < 1 << shift
    assert covers(units, nt, min(76, units * nt), shift, cost)


def test_most_tiles_of_a_call():
    shift, cost = constant("kChunkSegShift"), constant("kChunkSegmentCost")
    for units in (8193, 1 << 20, (1 << 26) - 1):
        nt = min(((1 << shift) - 1) // units, (1 << 24) - 2)
        assert covers(units, nt, 76, shift, cost)


def test_a_bit_too_high_is_found():
    """The restatement sees what it is for: 20 bits for segments, one of them the sign."""
    assert covers((1 << 20) - 1, 1, 76, 43, 3)
    assert not covers(1 << 20, 1, 76, 43, 3) and not covers(1 << 21, 16, 76, 43, 3)


def test_requests_of_a_few_query_tokens_stay_below_theirs():
    shift, cost = constant("kSegShift"), constant("kSegmentCost")
    assert covers(65535 * 4, 1, 76, shift, cost) and covers(65535 * 4, 8192, 76, shift, cost)
    assert 65535 * 4 < 1 << (63 - shift) and 65535 * 4 * ((1 << 24) - 2) < 1 << shift


@pytest.mark.parametrize("change", [
    dict(total=1 << 26, heads=1, tokens=A16, k=1), dict(total=1 << 27, heads=8, tokens=A16, k=64),
    dict(total=1 << 25, heads=2, tokens=A16, k=4097 * 128, max_pages=1 << 14),
    dict(total=8193, heads=128, max_pages=(1 << 25) - 4),
], ids=lambda c: "-".join(f"{k}{v}" for k, v in c.items() if k != "tokens"))
def test_more_units_or_tiles_are_refused(change):
    B.build()
    a = dict(total=8, heads=16, tokens=None, k=0, max_pages=10)
    a.update(change)
    code = ess.load().ess_cache_chunk(A16, a["total"], A16, A16, 640, ess.ESS_ROW_Q4, A16, a["max_pages"], 64, A16, 1,
                                      a["heads"], a["tokens"], a["k"], 0.04, A16, None, A16, 1 << 40, None, None)
    assert code == ess.ESS_ERR_UNSUPPORTED
