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


@pytest.mark.parametrize("out,other,off", [
    ("slot", "new_len", 0), ("slot", "seq_len", 3), ("row_seq", "n_keep", 0), ("row_end", "slot", 31),
    ("seq_row", "seq_len_out", 0), ("seq_len_out", "seq_len", 1), ("seq_len_out", "new_len", 0),
    ("free_state_out", "free_state", 1), ("slot", "page_table", 31), ("row_end", "free_ring", 63),
    ("page_table", "free_ring", 5)])
def test_page_tables_arrays_that_overlap(lib, out, other, off):
    """Every CTA reads the inputs while others write: an output inside another array is refused, by one entry too."""
    at = dict(row_seq=0x100000, row_end=0x110000, seq_row=0x120000, n_keep=0x130000)
    a = _pages(**at)
    setattr(a, out, getattr(a, other) + 4 * off)
    assert lib.attn_page_tables(ctypes.byref(a), None) == INVALID
    assert b"overlap" in lib.attn_last_error()


def test_page_tables_arrays_that_touch(lib):
    """Neighbours in one buffer are no overlap: the call gets as far as CUDA."""
    a = _pages(seq_len=0x1000, new_len=0x1010, seq_len_out=0x1020, free_state=0x1030, free_state_out=0x1038,
               slot=0x1040, row_end=0x1040 + 4 * 32)
    lib.attn_page_tables(ctypes.byref(a), None)
    assert b"overlap" not in lib.attn_last_error()
