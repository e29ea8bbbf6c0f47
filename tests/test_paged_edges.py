"""Paged attention and its cache: arguments at the edges of what is taken (no GPU needed)."""
import pytest
import torch

from test_paged import append, attend, lib   # noqa: F401 (lib: a fixture)


@pytest.mark.parametrize("window", [-1, 1 << 31, 1 << 32, (1 << 32) + 5, -(1 << 32)])
def test_windows_that_no_int_holds_are_refused(lib, window):
    from grouped_quadratic_gb300 import oal
    q, pool = torch.zeros(1, 4, 3, 64), torch.zeros(4, 2, 16, 64)
    table, past = torch.zeros(1, 4, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(oal.OALError, match="window"):
        oal.oal_paged_attention(q, pool, pool, table, past, window=window)


@pytest.mark.parametrize("call", [append, attend])
def test_pages_apart_by_multiples_of_16_bytes(lib, call):
    """8 elements of bf16, 4 of fp32."""
    least = 2 * 16 * 64
    for dtype, off, status in ((1, 8, 0), (1, 4, 1), (1, 2, 1), (0, 8, 0), (0, 4, 0), (0, 2, 1), (0, -4, 1), (1, -8, 1)):
        assert call(lib, B=0, dtype=dtype, page_stride=least + off) == status
