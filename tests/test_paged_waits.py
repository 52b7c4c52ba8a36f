"""Bounded waits of the paged decode kernels: a wait that cannot complete gives
up, is reported once, and leaves NaN in every row that it kept from being
computed -- not what an earlier call left in the workspace or the output.

reserved[0] makes a kernel's warps first wait, for that many microseconds, on a
barrier that nothing arrives at (as in attn_prefill).  Nothing faults, traps or
hangs: each wait ends after 1 ms and the next call on the context is correct.
"""
import pytest
import torch

import attention_split_attn_b200 as A
from parity import compare, poisoned_workspace
from test_paged_host import INVALID, _paged, lib  # noqa: F401 (a fixture)
from test_parity_paged import Case

STALL_US = 1000


@pytest.mark.parametrize("over", [dict(v=-1), dict(v=1000001)])
def test_wait_limits_are_refused(lib, over):
    for op in (A.OP_DECODE_PAGED, A.OP_DECODE_SHARED):
        a = _paged()
        a.reserved[0] = over["v"]
        assert A.paged_supports(a, op) == INVALID
        assert b"bounded-wait" in lib.attn_last_error()


def _stalled(c, op):
    """A good call, the same call with a wait that runs out on the same workspace and output, and a good call again:
    the three outputs.  The timeout is reported once."""
    a = c.args(op)
    ws = poisoned_workspace(A.paged_workspace_size(a, op))
    fn = A.attn_decode_paged_args if op == A.OP_DECODE_PAGED else A.attn_decode_shared_args
    outs = []
    for stall in (0, STALL_US, 0):
        a.reserved[0] = stall
        fn(a, ws=ws)
        torch.cuda.synchronize()
        outs.append(c.dev["out"].clone())
        if stall:
            with pytest.raises(A.AttnError) as e:
                A.check_device_status()
            assert e.value.status == -5          # ATTN_ERR_DEVICE_TIMEOUT
        A.check_device_status()
    return outs


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 128, 256])
@pytest.mark.parametrize("rows,Hq,end", [(4, 8, 500), (90, 4, 300), (3, 4, 9000)])
def test_shared_rows_of_a_timed_out_run_are_nan(cuda_lib, rows, Hq, end, D):
    """Blocks of one and of two tiles of rows, pieces that finish their rows (the whole context is shared) and units
    cut over several runs.  The rows of no group do not pass that kernel."""
    ends = [end + (i % 3) for i in range(rows)] + [40, 30]
    ends[1] = end - 7                                   # a row whose cells are all shared
    c = Case(61, ends, P=16, Hq=Hq, Hkv=2, D=D, groups=[(rows, end)], sinks=True)
    want = c.expected()
    good, bad, again = _stalled(c, A.OP_DECODE_SHARED)
    compare(good, want, 1e-5, 2e-2)
    assert torch.isnan(bad[:rows]).all()
    assert torch.equal(bad[rows:], good[rows:])
    assert torch.equal(again, good)


@pytest.mark.gpu
@pytest.mark.parametrize("op", [A.OP_DECODE_PAGED, A.OP_DECODE_SHARED])
@pytest.mark.parametrize("rows,longest,over", [(1500, 40, dict(D=64, Hq=4, Hkv=4)), (7, 3000, {}),
                                               (700, 50, dict(cache="e4m3", Hq=8, Hkv=8)),
                                               (600, 60, dict(D=256, Hq=32, Hkv=2))])
def test_single_rows_of_a_timed_out_warp_are_nan(cuda_lib, rows, longest, over, op):
    """More (row, KV head) pairs than warps, so that a warp's run holds several, and rows over many warps."""
    ends = [(7 * i) % longest for i in range(rows)]
    c = Case(62, ends, P=16, **over)
    want = c.expected()
    good, bad, again = _stalled(c, op)
    compare(good, want, 1e-5, 2e-2)
    sees = torch.tensor(ends) > 0
    assert torch.isnan(bad[sees.cuda()]).all() and (bad[~sees.cuda()] == 0).all()
    assert torch.equal(again, good)
