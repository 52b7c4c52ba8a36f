"""attn_decode_shared on its tensor-core form with what attn_page_tables leaves
when a step's rows do not all fit, and groups that name the shared cells
through other pages."""
import numpy as np
import pytest
import torch

import attention_split_attn_b200 as A
import paged_reference as ref
from parity import compare, poisoned_workspace
from test_parity_paged import Case, I32, i32

pytestmark = pytest.mark.gpu


def run_shared(args):
    """decode_shared in its shared form: its workspace holds more than the row form's."""
    need = A.paged_workspace_size(args, A.OP_DECODE_SHARED)
    assert need > A.paged_workspace_size(_without_groups(args), A.OP_DECODE_PAGED)
    A.attn_decode_shared_args(args, ws=poisoned_workspace(need))
    torch.cuda.synchronize()


def _without_groups(args):
    a = A.AttnPagedArgs.from_buffer_copy(args)
    a.n_groups, a.group_begin, a.group_len = 0, None, None
    return a


def _step(n_rows, new, P=16, width=40_000, Hq=8, Hkv=8, D=128):
    """A first step of len(new) sequences with room for n_rows rows: tables, append, and the shared decode's block."""
    n, pages = len(new), 64
    g = torch.Generator().manual_seed(n_rows)
    rnd = lambda h: torch.randn(n_rows, h, D, generator=g).to(torch.bfloat16)
    q, kn, vn = rnd(Hq), rnd(Hkv), rnd(Hkv)
    table = torch.full((n, width), -1, dtype=I32, device="cuda")
    o = A.page_tables(i32([0] * n).cuda(), i32(new).cuda(), table, torch.arange(pages, dtype=I32, device="cuda"),
                      i32([0, pages]).cuda(), page_size=P, n_rows=n_rows)
    k, v = (torch.zeros(pages, P, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    A.append_paged(kn.cuda(), vn.cuda(), o.slot, k, v)
    out = torch.full((n_rows, Hq, D), 7.0, dtype=torch.bfloat16, device="cuda")
    a = A.make_paged_args(q.cuda(), k, v, out, table, o.row_end, scale=0.09, row_table=o.row_seq,
                          group_begin=o.seq_row, group_len=o.seq_len)
    want = ref.attention(q, k.cpu(), v.cpu(), table[:, :8].cpu(), o.row_end.cpu(), scale=0.09,
                         row_table=np.maximum(o.row_seq.cpu().numpy(), 0))
    return a, o, out, want


@pytest.mark.parametrize("new", [[20, 40, 30], [20, 30, 0, 9, 50], [50, 3], [40, 1, 1]])
def test_sequences_whose_rows_do_not_fit(cuda_lib, new):
    """The sequence that does not fit sees nothing, and neither it nor those behind it disturb the others."""
    a, o, out, want = _step(48, new)
    run_shared(a)
    assert o.seq_row.tolist() == np.concatenate([[0], np.cumsum(new)]).tolist()
    fits = np.cumsum(new) <= 48
    assert o.seq_len.tolist() == np.where(fits, new, 0).tolist()
    compare(out, want, 1e-5, 2e-2)
    A.check_device_status()


def test_group_behind_the_rows_still_shares_the_others(cuda_lib):
    """Shared cells come through the first row's table; the second row names other pages there."""
    c = Case(42, [100, 120, 0, 0], P=16, Hq=4, Hkv=2, D=64, groups=[(2, 64), (2, 32)], garbage=False)
    want = c.expected()
    c.table[1, :4] = c.table[0, 4]
    c.groups["group_begin"] = i32([0, 2, 9])
    run_shared(c.args(A.OP_DECODE_SHARED))
    A.check_device_status()
    compare(c.dev["out"], want, 1e-5, 2e-2)


def test_group_behind_the_rows_with_a_row_that_sees_cells(cuda_lib):
    c = Case(43, [100, 120, 31, 0], P=16, Hq=4, Hkv=2, D=64, groups=[(2, 64), (2, 32)])
    c.groups["group_begin"] = i32([0, 2, 9])
    want = c.expected()
    run_shared(c.args(A.OP_DECODE_SHARED))
    with pytest.raises(A.AttnError, match="INVALID_ARG"):
        A.check_device_status()
    compare(c.dev["out"], want, 1e-5, 2e-2)
