"""Paged attention and its cache: arguments at the edges of what is taken (no GPU needed)."""
import pytest
import torch

from test_paged import lib   # noqa: F401 (a fixture)


@pytest.mark.parametrize("window", [-1, 1 << 31, 1 << 32, (1 << 32) + 5, -(1 << 32)])
def test_windows_that_no_int_holds_are_refused(lib, window):
    from grouped_quadratic_gb300 import oal
    q, pool = torch.zeros(1, 4, 3, 64), torch.zeros(4, 2, 16, 64)
    table, past = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(oal.OALError, match="window"):
        oal.oal_paged_attention(q, pool, pool, table, past, window=window)
