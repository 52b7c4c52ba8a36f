"""Calls on another stream than the current one, with memory that the binding
allocates: work still queued on the current stream must not meet it."""
import pytest
import torch

import attention_split_attn_b200 as A
from parity import compare
from test_parity_paged import Case, I32, i32

pytestmark = pytest.mark.gpu

CYCLES = 100_000_000   # about 50 ms


def _queue_writes_to(nbytes):
    """A freed block of the current stream's pool that queued work has yet to overwrite."""
    junk = torch.empty(nbytes, dtype=torch.uint8, device="cuda")
    torch.cuda._sleep(CYCLES)
    junk.fill_(0xFF)
    return junk.data_ptr()


@pytest.mark.parametrize("op", [A.OP_DECODE_PAGED, A.OP_DECODE_SHARED])
def test_default_workspace(cuda_lib, op):
    c = Case(41, [900, 700, 800, 750], P=16, sinks=True, groups=[(4, 690)])
    want, a, side = c.expected(), c.args(op), torch.cuda.Stream()
    need = A.paged_workspace_size(a, op)
    torch.cuda.synchronize()
    at = _queue_writes_to(need)
    fn = A.attn_decode_paged_args if op == A.OP_DECODE_PAGED else A.attn_decode_shared_args
    ws = fn(a, stream=side)
    assert ws.data_ptr() != at
    side.synchronize()
    got = c.dev["out"].clone()
    torch.cuda.synchronize()
    compare(got, want, 1e-5, 2e-2)
    A.check_device_status()


def test_slot_map_dropped_while_the_append_waits(cuda_lib):
    P, pages, rows = 16, 64, 100
    k = torch.zeros(pages, P, 1, 64, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    new = torch.randn(rows, 1, 64, device="cuda").to(torch.bfloat16)
    table, ring = torch.zeros(1, 8, dtype=I32, device="cuda"), torch.arange(pages, device="cuda").to(I32)
    lens, grow, state = i32([0]).cuda(), i32([rows]).cuda(), i32([0, pages]).cuda()
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    _queue_writes_to(4 * rows)
    o = A.page_tables(lens, grow, table, ring, state, page_size=P, n_rows=rows, stream=side)
    with torch.cuda.stream(side):
        torch.cuda._sleep(CYCLES)
    A.append_paged(new, new, o.slot, k, v, stream=side)
    del o
    others = [torch.full((rows,), pages * P - 1, dtype=I32, device="cuda") for _ in range(8)]
    torch.cuda.synchronize()
    assert torch.equal(k.view(-1, 1, 64)[:rows], new) and torch.equal(v.view(-1, 1, 64)[:rows], new)
    assert (k.view(-1, 64)[rows:] == 0).all()
    A.check_device_status()
    del others
