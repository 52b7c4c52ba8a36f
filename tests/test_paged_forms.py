"""attn_decode_shared on its tensor-core form where small tables would run row
by row: a pool past 2^32 elements, rows without a table, and a serving loop,
eager and as a replayed graph, whose lengths and groups change every step."""
import numpy as np
import pytest
import torch

import attention_split_attn_b200 as A
import paged_reference as ref
from parity import compare, poisoned_workspace
from test_paged_groups import run_shared
from test_parity_paged import Case, I32, i32

pytestmark = pytest.mark.gpu


def _wide(table, cells, P):
    """The table with columns behind it that no range reaches."""
    t = torch.full((table.shape[0], max(table.shape[1], cells // P)), -9, dtype=I32)
    t[:, :table.shape[1]] = table
    return t.cuda()


def test_offsets_past_32_bits(cuda_lib):
    P, Hkv, D = 64, 8, 256
    pages = (1 << 32) // (P * Hkv * D) + 50
    k = torch.zeros(pages, P, Hkv, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    use = [pages - 1, 3, pages - 2, pages // 2]
    g = torch.Generator().manual_seed(1)
    ks, vs = (torch.randn(4 * P, Hkv, D, generator=g).to(torch.bfloat16) for _ in range(2))
    A.append_paged(ks.cuda(), vs.cuda(), i32(np.concatenate([np.arange(P) + u * P for u in use])).cuda(), k, v)
    q = torch.randn(3, 8, D, generator=g).to(torch.bfloat16)
    ends = i32([4 * P, 3 * P + 5, 2 * P])
    want = ref.attention(q, ks.reshape(4, P, Hkv, D), vs.reshape(4, P, Hkv, D), i32([[0, 1, 2, 3]] * 3), ends,
                         scale=0.06)
    out = torch.empty(3, 8, D, dtype=torch.bfloat16, device="cuda")
    a = A.make_paged_args(q.cuda(), k, v, out, _wide(i32([use] * 3), 4096, P), ends.cuda(), scale=0.06,
                          group_begin=i32([0, 3]).cuda(), group_len=i32([2 * P + 9]).cuda())
    run_shared(a)
    compare(out, want, 1e-5, 2e-2)
    A.check_device_status()


@pytest.mark.parametrize("row", [0, 1, 2])
def test_rows_of_a_group_without_a_table(cuda_lib, row):
    """The group's first row gives the shared cells: without its table nothing is shared, and the others read theirs."""
    c = Case(71, [64, 70, 80], P=16, D=64, row_table=[0, 1, 2], groups=[(3, 48)])
    want = c.expected()
    want[row] = 0
    c.row_table[row] = 3
    run_shared(c.args(A.OP_DECODE_SHARED))
    with pytest.raises(A.AttnError, match="INVALID_ARG"):
        A.check_device_status()
    compare(c.dev["out"], want, 1e-5, 2e-2)


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("G,D", [(2, 128), (7, 64)])
def test_serving_loop(cuda_lib, graph, G, D):
    """Chunks of prompts and single tokens; a step's rows pass the room for them now and then.  Every row is checked
    against the keys and values that its sequence was given, and against decode_paged's rows."""
    rng, gen = np.random.default_rng(72), torch.Generator().manual_seed(72)
    n, P, n_pages, T, Hkv = 5, 16, 80, 64, 2
    Hq, most = G * Hkv, 300
    width = (66 << 20) // (T * Hkv * D * 4) // P + 1
    k, v = (torch.zeros(n_pages, P, Hkv, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    z = lambda *s: torch.zeros(*s, dtype=I32, device="cuda")
    table, ring = z(n, width) - 1, torch.randperm(n_pages, generator=gen).to(I32).cuda()
    lens, new_len, state = z(n), z(n), i32([3, n_pages]).cuda()
    q, kn, vn = (torch.zeros(T, h, D, dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv))
    out, rows_out = (torch.zeros(T, Hq, D, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    pa = A.make_page_args(lens, new_len, table, ring, state, page_size=P, n_rows=T)
    o = pa.outputs
    aa = A.make_append_args(kn, vn, o.slot, k, v)
    kw = dict(scale=0.09, row_table=o.row_seq)
    sa = A.make_paged_args(q, k, v, out, table, o.row_end, group_begin=o.seq_row, group_len=o.seq_len, **kw)
    da = A.make_paged_args(q, k, v, rows_out, table, o.row_end, **kw)
    need = [A.paged_workspace_size(sa, A.OP_DECODE_SHARED), A.paged_workspace_size(da, A.OP_DECODE_PAGED)]
    assert need[0] > need[1]
    ws = poisoned_workspace(need[0])

    def step():
        A.attn_page_tables_args(pa)
        A.attn_append_paged_args(aa)
        A.attn_decode_shared_args(sa, ws=ws)
        A.attn_decode_paged_args(da, ws=ws)
        lens.copy_(o.seq_len)
        state.copy_(o.free_state)

    if graph:
        step()                    # no rows yet
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        g.replay()
    kept = [[torch.zeros(0, Hkv, D)] * 2 for _ in range(n)]
    shared = refused = 0
    for it in range(12):
        cur = lens.tolist()
        new = [int(rng.choice([0, 1, 1, 12, 40])) if c < most else -1 for c in cur]
        if it % 5 == 4:
            new[int(rng.integers(n))] = -1
        new_len.copy_(i32(new))
        rows = [torch.randn(T, h, D, generator=gen).to(torch.bfloat16) for h in (Hq, Hkv, Hkv)]
        for t, r in zip((q, kn, vn), rows):
            t.copy_(r)
        g.replay() if graph else step()
        torch.cuda.synchronize()
        A.check_device_status()
        got_len, t = lens.tolist(), 0
        want = np.zeros((T, Hq, D))
        for i in range(n):
            if new[i] < 0:
                kept[i] = [torch.zeros(0, Hkv, D)] * 2
                continue
            r0, t = t, t + new[i]
            if got_len[i] == cur[i]:
                refused += new[i] > 0
                continue
            shared += new[i] > 1
            kept[i] = [torch.cat([x, r[r0:t].float()]) for x, r in zip(kept[i], rows[1:])]
            m = len(kept[i][0])
            pad = lambda y: torch.cat([y, torch.zeros(-m % P, Hkv, D)]).reshape(-1, P, Hkv, D)
            want[r0:t] = ref.attention(rows[0][r0:t], pad(kept[i][0]), pad(kept[i][1]), i32([list(range(-(-m // P)))]),
                                       i32([cur[i] + 1 + j for j in range(new[i])]), scale=0.09,
                                       row_table=[0] * new[i])
        compare(out, want, 1e-5, 2e-2, f"step {it}, shared")
        compare(rows_out, want, 1e-5, 2e-2, f"step {it}, row by row")
    assert shared and refused
    del pa, aa, sa, da
