"""Calls of the paged-cache operations at the edges of what is documented, on a
machine without a GPU: refused with a reason before any CUDA call."""
import ctypes

import pytest

from test_paged_host import INVALID, UNSUPPORTED, _append, _pages, lib  # noqa: F401 (lib is a fixture)


@pytest.mark.parametrize("rows", [(1 << 30) + 1, (1 << 31) - 4, (1 << 31) - 1])
def test_append_row_numbers_stay_within_32_bits(lib, rows):
    """Rows are taken four at a time, in blocks of rows / (8 SMs): near 2^31 rows a number could pass it."""
    a = _append(n_rows=rows)
    assert lib.attn_append_paged(ctypes.byref(a), None) == UNSUPPORTED
    assert b"too many rows" in lib.attn_last_error()
