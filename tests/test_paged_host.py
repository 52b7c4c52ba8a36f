"""The paged-cache operations on a machine without a GPU: their argument blocks
have the header's layout, and calls that the kernels do not cover are refused
before any CUDA call, with their reason."""
import ctypes
import os
import subprocess

import pytest

import attention_split_attn_b200 as A

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "attn.h")
INVALID, UNSUPPORTED = -1, -2


@pytest.fixture(scope="module")
def lib():
    from attention_split_attn_b200 import build
    build.build()
    return A.load_library()


@pytest.mark.parametrize("name,mirror", [("attn_page_args", A.AttnPageArgs), ("attn_append_args", A.AttnAppendArgs),
                                         ("attn_paged_args", A.AttnPagedArgs)])
def test_struct_layout_matches_header(tmp_path, name, mirror):
    fields = [f[0] for f in mirror._fields_]
    src = tmp_path / "layout.c"
    lines = ["#include <stdio.h>", "#include <stddef.h>", '#include "attn.h"', "int main(void){",
             f'printf("size %zu\\n", sizeof({name}));']
    lines += [f'printf("{f} %zu\\n", offsetof({name}, {f}));' for f in fields]
    src.write_text("\n".join(lines + ["return 0;}"]))
    exe = tmp_path / "layout"
    subprocess.check_call(["gcc", "-std=c11", "-I", os.path.dirname(HEADER), str(src), "-o", str(exe)])
    got = dict(l.split() for l in subprocess.check_output([str(exe)], text=True).splitlines())
    assert int(got["size"]) == ctypes.sizeof(mirror)
    for f in fields:
        assert int(got[f]) == getattr(mirror, f).offset, f


def _paged(**over):
    a = A.AttnPagedArgs()
    a.n_rows, a.n_head_q, a.n_head_kv, a.head_dim, a.n_pages, a.page_size = 3, 8, 2, 128, 40, 32
    a.q, a.k, a.v, a.out, a.page_table, a.row_end = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000, 0x60000
    a.q_type = a.kv_type = a.out_type = A.ATTN_BF16
    a.q_stride_row, a.q_stride_head = 8 * 128, 128
    a.o_stride_row, a.o_stride_head = 8 * 128, 128
    a.kv_stride_page, a.kv_stride_cell, a.kv_stride_head = 32 * 256, 256, 128
    a.n_tables, a.table_width, a.table_stride = 3, 10, 10
    a.scale = 0.1
    for k, v in over.items():
        setattr(a, k, v)
    return a


E4 = dict(kv_type=A.ATTN_FP8_E4M3, k_scale=0x70000, v_scale=0x80000, scale_stride_cell=2)


@pytest.mark.parametrize("over", [{}, dict(page_size=48, kv_stride_page=48 * 256), dict(row_begin=0x70000),
                                  dict(n_tables=1, row_table=0x70000), dict(out_type=A.ATTN_F32), E4,
                                  dict(n_rows=0, q=0), dict(n_pages=0, k=0, v=0)])
def test_paged_accepts(lib, over):
    for op in (A.OP_DECODE_PAGED, A.OP_DECODE_SHARED):
        assert A.paged_supports(_paged(**over), op) == 0, lib.attn_last_error()


@pytest.mark.parametrize("want,word,over", [
    (INVALID, b"negative size", dict(n_rows=-1)),
    (INVALID, b"multiple", dict(n_head_q=7)),
    (UNSUPPORTED, b"head_dim", dict(head_dim=96)),
    (UNSUPPORTED, b"cache dtype", dict(q_type=A.ATTN_F16)),
    (UNSUPPORTED, b"> 16", dict(n_head_q=34)),
    (UNSUPPORTED, b"F16, BF16, e4m3 or int8", dict(kv_type=A.ATTN_F32, q_type=A.ATTN_F32)),
    (UNSUPPORTED, b"head_dim 64", dict(head_dim=64, **E4)),
    (UNSUPPORTED, b"> 8", dict(n_head_q=18, **E4)),
    (INVALID, b"needs k_scale", dict(kv_type=A.ATTN_I8)),
    (INVALID, b"scale_stride_cell", dict(E4, scale_stride_cell=1)),
    (INVALID, b"only for", dict(k_scale=0x70000, v_scale=0x70000)),
    (UNSUPPORTED, b"out must be", dict(out_type=A.ATTN_I8)),
    (INVALID, b"page_size", dict(page_size=0)),
    (UNSUPPORTED, b"multiple of 16", dict(page_size=24)),
    (UNSUPPORTED, b"2^31", dict(n_pages=1 << 26)),
    (UNSUPPORTED, b"2^31", dict(table_width=1 << 26, table_stride=1 << 26)),
    (UNSUPPORTED, b"multiples of 16 bytes", dict(k=0x20008)),
    (UNSUPPORTED, b"multiples of 16 bytes", dict(kv_stride_cell=252)),
    (UNSUPPORTED, b"zero kv stride", dict(kv_stride_head=0)),
    (INVALID, b"negative kv stride", dict(kv_stride_page=-8)),
    (INVALID, b"scale is NaN", dict(scale=float("nan"))),
    (INVALID, b"NULL", dict(row_end=0)),
    (INVALID, b"page_table is NULL", dict(page_table=0)),
    (INVALID, b"table_stride", dict(table_stride=9)),
    (INVALID, b"no row_table", dict(n_tables=2)),
    (UNSUPPORTED, b"multiples of 8", dict(q_stride_head=132)),
    (INVALID, b"reserved", dict(reserved=(ctypes.c_int32 * 4)(0, 1, 0, 0))),
])
def test_paged_refuses(lib, want, word, over):
    for op in (A.OP_DECODE_PAGED, A.OP_DECODE_SHARED):
        a = _paged(**over)
        assert A.paged_supports(a, op) == want
        assert word in lib.attn_last_error()
        assert lib.attn_paged_workspace_size(ctypes.byref(a), op) == 0
        fn = lib.attn_decode_paged if op == A.OP_DECODE_PAGED else lib.attn_decode_shared
        assert fn(ctypes.byref(a), None, 0, None) == want


def test_groups_are_for_decode_shared(lib):
    a = _paged(n_groups=1, group_begin=0x70000, group_len=0x80000)
    assert A.paged_supports(a, A.OP_DECODE_SHARED) == 0
    assert A.paged_supports(a, A.OP_DECODE_PAGED) == INVALID
    assert A.paged_supports(_paged(n_groups=1), A.OP_DECODE_SHARED) == INVALID
    assert A.paged_supports(_paged(n_groups=-1), A.OP_DECODE_SHARED) == INVALID
    assert A.paged_supports(_paged(), 0) == INVALID


def _append(**over):
    a = A.AttnAppendArgs()
    a.n_rows, a.n_head_kv, a.head_dim, a.n_pages, a.page_size = 5, 2, 128, 40, 24
    a.k_new, a.v_new, a.slot, a.k, a.v = 0x10000, 0x20000, 0x30000, 0x40000, 0x50000
    a.new_type, a.kv_type = A.ATTN_F32, A.ATTN_BF16
    a.new_stride_row, a.new_stride_head = 256, 128
    a.kv_stride_page, a.kv_stride_cell, a.kv_stride_head = 24 * 256, 256, 128
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("want,word,over", [
    (INVALID, b"n_rows < 0", dict(n_rows=-1)),
    (INVALID, b"n_head_kv", dict(n_head_kv=0)),
    (UNSUPPORTED, b"head_dim", dict(head_dim=80)),
    (UNSUPPORTED, b"new rows must be F32", dict(new_type=A.ATTN_FP8_E4M3)),
    (UNSUPPORTED, b"the cache must be", dict(kv_type=A.ATTN_F32)),
    (INVALID, b"needs k_scale", dict(kv_type=A.ATTN_FP8_E4M3)),
    (INVALID, b"only for", dict(k_scale=0x10000)),
    (INVALID, b"page_size", dict(page_size=0)),
    (UNSUPPORTED, b"2^31", dict(n_pages=1 << 27)),
    (UNSUPPORTED, b"multiples of 16 bytes", dict(v=0x50004)),
    (UNSUPPORTED, b"zero kv stride", dict(kv_stride_cell=0)),
    (INVALID, b"NULL", dict(slot=0)),
    (INVALID, b"negative stride", dict(new_stride_row=-8)),
    (UNSUPPORTED, b"new rows and their strides", dict(new_stride_row=258)),
    (INVALID, b"reserved", dict(reserved=(ctypes.c_int32 * 4)(1, 0, 0, 0))),
])
def test_append_refuses(lib, want, word, over):
    assert lib.attn_append_paged(ctypes.byref(_append(**over)), None) == want
    assert word in lib.attn_last_error()


def test_append_of_nothing_is_ok(lib):
    assert lib.attn_append_paged(ctypes.byref(_append(n_rows=0, k_new=0)), None) == 0
    assert lib.attn_append_paged(ctypes.byref(_append(n_pages=0, k=0, v=0)), None) == 0


def _pages(**over):
    a = A.AttnPageArgs()
    a.n_seqs, a.page_size, a.n_pages, a.table_width, a.n_rows, a.table_stride = 4, 16, 64, 8, 32, 8
    for i, f in enumerate(("seq_len", "new_len", "page_table", "free_ring", "free_state", "free_state_out", "slot",
                           "seq_len_out")):
        setattr(a, f, 0x10000 * (i + 1))
    for k, v in over.items():
        setattr(a, k, v)
    return a


@pytest.mark.parametrize("want,word,over", [
    (INVALID, b"negative size", dict(n_seqs=-1)),
    (INVALID, b"negative size", dict(n_rows=-1)),
    (UNSUPPORTED, b"16385 sequences", dict(n_seqs=16385)),
    (INVALID, b"page_size", dict(page_size=0)),
    (UNSUPPORTED, b"2^31", dict(n_pages=1 << 28)),
    (UNSUPPORTED, b"2^31", dict(table_width=1 << 28, table_stride=1 << 28)),
    (INVALID, b"free_state is NULL", dict(free_state=0)),
    (INVALID, b"slot is NULL", dict(slot=0)),
    (INVALID, b"free_ring is NULL", dict(free_ring=0)),
    (INVALID, b"seq_len", dict(seq_len=0)),
    (INVALID, b"page_table is NULL", dict(page_table=0)),
    (INVALID, b"table_stride", dict(table_stride=7)),
    (INVALID, b"input array", dict(free_state_out=0x50000)),
    (INVALID, b"input array", dict(seq_len_out=0x10000)),
    (INVALID, b"reserved", dict(reserved=(ctypes.c_int32 * 4)(0, 0, 0, 7))),
])
def test_page_tables_refuses(lib, want, word, over):
    assert lib.attn_page_tables(ctypes.byref(_pages(**over)), None) == want
    assert word in lib.attn_last_error()


def test_null_blocks_are_refused(lib):
    assert lib.attn_page_tables(None, None) == INVALID
    assert lib.attn_append_paged(None, None) == INVALID
    assert lib.attn_decode_paged(None, None, 0, None) == INVALID
    assert lib.attn_decode_shared(None, None, 0, None) == INVALID
