"""Paged attention at the edges of what it promises: tokens that see nothing beside numbers that are not finite."""
import math

import pytest
import torch

from test_paged_gpu import BF16, F32, Cache, draw, oracle, tolerance

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def oal():
    from grouped_quadratic_gb300 import build, oal
    build.build()
    oal.load_library()
    return oal


def put(c, j, value, b=0):
    """Key and value j of a sequence."""
    for pool in (c.Kp, c.Vp):
        pool[c.table[b, j // c.page].item(), :, j % c.page] = value


@pytest.mark.parametrize("dtype", [F32, BF16])
@pytest.mark.parametrize("bad", [math.nan, math.inf])
@pytest.mark.parametrize("T,past", [(3, 30), (8, 40), (60, 30), (3, 2000), (8, 2000), (90, 2000), (300, 900)])
def test_tokens_that_see_nothing_beside_bad_numbers(oal, dtype, bad, T, past):
    """Of three tokens one sees nothing and gets zeros, one does not see the key that is bad, one does (and is not
    looked at); the keys in one piece and in several."""
    c = Cache(1, 2, [past], [T], 16, dtype, seed=101, fill=bad)
    Q = draw((1, 6, T, 64), dtype, 102, 1.5)
    first = torch.zeros(1, T, dtype=torch.int32)
    first[:, ::3], first[:, 1::3] = 1 << 28, past - 4
    put(c, past - 5, bad)
    Y = oal.oal_paged_attention(Q, c.Kp, c.Vp, c.table, c.past, first=first.cuda())
    oal.oal_sync_status()
    assert (Y[:, :, ::3] == 0).all()
    put(c, past - 5, 0.0)
    want, size = oracle(c, Q, [T], first=first.cuda())
    off = (Y.double() - want).abs() - tolerance(dtype, want, size)
    assert (off[:, :, 1::3] <= 0).all()
