"""A prepared argument block holds addresses, so it keeps the tensors behind
them: blocks made from temporaries, on a machine without a GPU."""
import gc
import weakref

import pytest
import torch

import attention_split_attn_b200 as A
from test_streams_host import OnGpu


def _blocks():
    i, f, h = torch.int32, torch.float32, torch.bfloat16

    def flat(t):
        return A.make_args(t(h, 2, 4, 64), t(h, 16, 2, 64), t(h, 16, 2, 64), t(h, 2, 4, 64), scale=1.0,
                           **{n: t(i, 16) for n in ("row_begin", "row_end", "cell_seq", "row_seq", "cell_pos", "row_pos")},
                           mask=t(f, 2, 16), alibi_slopes=t(f, 4), sinks=t(f, 4))

    def flat_codes(t):
        return A.make_args(t(h, 2, 4, 64), t(torch.int8, 16, 2, 64), t(torch.int8, 16, 2, 64), t(h, 2, 4, 64), scale=1.0,
                           k_scale=t(f, 16, 2), v_scale=t(f, 16, 2))

    def selected(t):
        return A.make_selected_args(t(h, 2, 4, 64), t(h, 16, 2, 64), t(h, 16, 2, 64), t(h, 2, 4, 64), t(i, 2, 8),
                                    scale=1.0, sorted_out=t(i, 2, 8), count_out=t(i, 2), sinks=t(f, 4))

    def pages(t):
        return A.make_page_args(t(i, 2), t(i, 2), t(i, 2, 3), t(i, 9), t(i, 2), page_size=16, n_rows=4, n_keep=t(i, 2),
                                outputs=A.PageTables(*(t(i, 9) for _ in A.PageTables._fields)))

    def append(t):
        return A.make_append_args(t(h, 3, 2, 64), t(h, 3, 2, 64), t(i, 3), t(torch.int8, 4, 16, 2, 64),
                                  t(torch.int8, 4, 16, 2, 64), k_scale=t(f, 64, 2), v_scale=t(f, 64, 2))

    def paged(t):
        return A.make_paged_args(t(h, 2, 4, 64), t(h, 4, 16, 2, 64), t(h, 4, 16, 2, 64), t(h, 2, 4, 64), t(i, 2, 3),
                                 t(i, 2), scale=1.0, row_begin=t(i, 2), row_table=t(i, 2), group_begin=t(i, 2),
                                 group_len=t(i, 1), alibi_slopes=t(f, 4), sinks=t(f, 4))
    return [flat, flat_codes, selected, pages, append, paged]


@pytest.mark.parametrize("make", _blocks(), ids=lambda f: f.__name__)
def test_blocks_keep_their_tensors(make):
    alive = []

    def t(dtype, *shape):
        x = torch.zeros(shape, dtype=dtype).as_subclass(OnGpu)
        alive.append(weakref.ref(x))
        return x

    block = make(t)
    gc.collect()
    assert all(r() is not None for r in alive)
    del block
    gc.collect()
    assert all(r() is None for r in alive)     # and no longer than that
