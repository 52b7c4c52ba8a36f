"""The paged-cache operations on a B200 against plain implementations: page
bookkeeping exactly, appended values and codes exactly, attention against 64
bits.

Attention tolerances are those of the other operations (parity.py): NMSE 1e-5
and 2e-2 absolute.  They hold the roundings with room to spare: a 16-bit
output is off by at most 2^-9 (bf16) relative to itself and the weights by
2^-9 each before they are averaged, so the relative error's square stays below
(2^-9)^2 (1 + 1) = 7.6e-6 in the worst case where every rounding is a half step
in one direction, a third of that for evenly spread ones.
"""
import math

import numpy as np
import pytest
import torch

import attention_split_attn_b200 as A
import paged_reference as ref
from parity import compare, poisoned_workspace

pytestmark = pytest.mark.gpu

I32 = torch.int32
DT = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}


def i32(x):
    return torch.tensor(np.asarray(x), dtype=I32)


# ---------------------------------------------------------------------------
# page tables
# ---------------------------------------------------------------------------

def _pool_state(rng, lens, P, width, spare, extra=0):
    """Tables that hold `lens`, a ring of `spare` free pages somewhere in it."""
    held = [-(-int(x) // P) for x in lens]
    n_pages = sum(held) + spare + extra
    ids = rng.permutation(n_pages)
    table = np.full((len(lens), width), -1, dtype=np.int64)
    at = 0
    for i, h in enumerate(held):
        table[i, :h] = ids[at:at + h]
        at += h
    ring = np.full(n_pages, -1, dtype=np.int64)
    head = int(rng.integers(0, max(n_pages, 1)))
    for k in range(spare):
        ring[(head + k) % n_pages] = ids[at + k]
    return table, ring, [head if n_pages else 0, spare]


def _run_tables(lens, new, table, ring, state, P, n_rows, keep=None):
    t, r = i32(table).cuda(), i32(ring).cuda()
    o = A.page_tables(i32(lens).cuda(), i32(new).cuda(), t, r, i32(state).cuda(), page_size=P, n_rows=n_rows,
                      n_keep=None if keep is None else i32(keep).cuda())
    torch.cuda.synchronize()
    return [x.cpu().numpy() for x in o] + [t.cpu().numpy(), r.cpu().numpy()]


NAMES = ("slot", "row_seq", "row_end", "seq_row", "seq_len", "state", "table", "ring")


def _check_tables(lens, new, table, ring, state, P, n_rows, keep=None):
    got = _run_tables(lens, new, table, ring, state, P, n_rows, keep)
    want = ref.page_tables(lens, new, table, ring, state, P, n_rows, keep)
    for name, g, w in zip(NAMES, got, want):
        assert np.array_equal(g, w), (name, np.argwhere(g != w)[:5], g[:8], w[:8])
    A.check_device_status()
    return got


@pytest.mark.parametrize("P", [1, 16, 24, 128])
@pytest.mark.parametrize("n", [1, 31, 513, 1500])
def test_page_tables(cuda_lib, n, P):
    rng = np.random.default_rng(n * 1000 + P)
    lens = rng.integers(0, 300, n)
    new = np.where(rng.random(n) < 0.6, rng.integers(0, 3, n), rng.integers(0, 200, n))
    new[rng.random(n) < 0.2] = -1
    width = 500 // P + 1
    table, ring, state = _pool_state(rng, lens, P, width, spare=n * (200 // P + 2))
    keep = np.minimum(rng.integers(0, 3, n), -(-lens // P))
    _check_tables(lens, new, table, ring, state, P, int(np.maximum(new, 0).sum()) + 7, keep)


def test_page_tables_of_the_most_sequences(cuda_lib):
    rng = np.random.default_rng(4)
    n = 16384
    lens, new = rng.integers(0, 40, n), rng.integers(-1, 3, n)
    table, ring, state = _pool_state(rng, lens, 16, 4, spare=n)
    _check_tables(lens, new, table, ring, state, 16, 2 * n)


def test_page_tables_then_flat_decode(cuda_lib):
    """attn_decode right behind attn_page_tables reads the row ends of that step, call after call."""
    k = torch.randn(64, 2, 64, device="cuda").to(torch.bfloat16)
    q = torch.randn(4, 4, 64, device="cuda").to(torch.bfloat16)
    out = torch.empty_like(q)
    new, table, ring = i32([1] * 4).cuda(), torch.zeros(4, 4, dtype=I32, device="cuda"), torch.arange(16).to(I32).cuda()
    lens = [i32([a, 3, 17, 40 - a]).cuda() for a in range(30)]
    pa = [A.make_page_args(x, new, table.clone(), ring.clone(), i32([0, 16]).cuda(), page_size=16, n_rows=4)
          for x in lens]
    da = [A.make_args(q, k, k, out, scale=0.1, row_begin=torch.zeros(4, dtype=I32, device="cuda"),
                      row_end=a.outputs.row_end) for a in pa]
    ws = torch.empty(A.workspace_size(da[0], A.OP_DECODE), dtype=torch.uint8, device="cuda")
    outs = []
    for a, d in zip(pa, da):
        A.attn_page_tables_args(a)
        A.attn_decode_args(d, ws=ws)
        outs.append(out.clone())
    torch.cuda.synchronize()
    pages = k.reshape(4, 16, 2, 64)
    for x, got in zip(lens, outs):
        compare(got, ref.attention(q.cpu(), pages.cpu(), pages.cpu(), i32([[0, 1, 2, 3]]), x.cpu() + 1, scale=0.1,
                                   row_table=[0] * 4), 1e-5, 2e-2)


@pytest.mark.parametrize("what", ["ring", "rows", "width"])
def test_page_tables_sequences_that_cannot_grow(cuda_lib, what):
    rng = np.random.default_rng(5)
    lens, new = np.array([10, 32, 0, 64, 31, 5]), np.array([30, 1, 70, 0, 1, -1])
    width = 3 if what == "width" else 10
    table, ring, state = _pool_state(rng, lens, 32, width, spare=2 if what == "ring" else 20, extra=6)
    n_rows = 90 if what == "rows" else 128
    got = _check_tables(lens, new, table, ring, state, 32, n_rows)
    assert (got[4] == lens).any()      # somebody was refused
    assert (got[4] != lens).any()      # and somebody was not


def test_page_tables_of_nothing(cuda_lib):
    rng = np.random.default_rng(6)
    _check_tables([], [], np.zeros((0, 4), dtype=np.int64), np.arange(5), [3, 5], 16, 9)
    table, ring, state = _pool_state(rng, [7, 0], 16, 2, spare=1)
    _check_tables([7, 0], [0, 0], table, ring, state, 16, 0)
    _check_tables([7, 0], [-1, -1], table, ring, state, 16, 4)


def test_page_tables_record_what_cannot_be(cuda_lib):
    ok = dict(P=16, n_rows=40)
    table, ring, state = _pool_state(np.random.default_rng(7), [20, 20], 16, 4, spare=4)
    for lens, new, t, r, st in (
            ([-1, 20], [1, 1], table, ring, state),                         # a length below 0
            ([65, 20], [1, 1], table, ring, state),                         # ... beyond its table row
            ([20, 20], [1, 1], np.where(table == table[0, 1], 99, table), ring, state),   # an id outside the pool
            ([20, 20], [16, 1], table, np.full_like(ring, -7), state),      # ... in the ring
            ([20, 20], [1, 1], table, ring, [len(ring), 1]),                # a ring that cannot be
            ([20, 20], [1, -1], table, ring, [0, len(ring)])):              # more pages than the ring holds
        got = _run_tables(lens, new, t, r, st, **ok)
        with pytest.raises(A.AttnError, match="INVALID_ARG"):
            A.check_device_status()
        slot = got[0]
        assert ((slot >= -1) & (slot < len(ring) * 16)).all()
    A.check_device_status()


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------

def _empty_pool(pages, P, Hkv, D, dtype, order, seed):
    g = torch.Generator(device="cuda").manual_seed(seed)
    shape = (pages, Hkv, P, D) if order == "hnd" else (pages, P, Hkv, D)
    mk = lambda: torch.randint(-100, 100, shape, generator=g, device="cuda", dtype=torch.int8).to(
        dtype if dtype != torch.int8 else torch.int8)
    k, v = mk(), mk()
    return (k.transpose(1, 2), v.transpose(1, 2)) if order == "hnd" else (k, v)


def _slots(rng, rows, pages, P):
    slot = rng.permutation(pages * P)[:rows]
    slot[::7] = -1
    if rows > 3:
        slot[3] = pages * P          # beyond the pool: skipped like padding
    return slot


@pytest.mark.parametrize("order", ["nhd", "hnd"])
@pytest.mark.parametrize("new,cache", [("bf16", "bf16"), ("f16", "f16"), ("f32", "bf16"), ("f32", "f16"),
                                       ("f16", "bf16"), ("bf16", "f16")])
@pytest.mark.parametrize("rows,Hkv,D,P", [(1, 1, 64, 16), (37, 3, 128, 24), (700, 8, 256, 16)])
def test_append_copies(cuda_lib, rows, Hkv, D, P, new, cache, order):
    rng = np.random.default_rng(rows + D)
    pages = rows // P + 3
    k, v = _empty_pool(pages, P, Hkv, D, DT[cache], order, 1)
    # new rows with a stride: the K and V halves of one projection's output
    kv = torch.randn(rows, 2 * Hkv + 1, D, device="cuda").to(DT[new])
    kn, vn = kv[:, :Hkv], kv[:, Hkv:2 * Hkv]
    slot = _slots(rng, rows, pages, P)
    wk, wv = k.clone(), v.clone()
    for t, s in enumerate(slot):
        if 0 <= s < pages * P:
            wk[s // P, s % P], wv[s // P, s % P] = kn[t].to(DT[cache]), vn[t].to(DT[cache])
    A.append_paged(kn, vn, i32(slot).cuda(), k, v)
    torch.cuda.synchronize()
    assert torch.equal(k, wk) and torch.equal(v, wv)


def _codes64(x, fmt):
    """Scale and values (as code values) of rows x [..., D] in 64 bits."""
    top = 448.0 if fmt == "e4m3" else 127.0
    s = (x.double().abs().amax(-1) / top).float()
    y = x.double() / torch.where(s == 0, 1.0, s).double()[..., None]
    if fmt == "i8":
        return s, y.round()
    vals = torch.arange(127, dtype=torch.uint8).view(torch.float8_e4m3fn).double()
    mids = (vals[1:] + vals[:-1]) / 2
    lo, hi = torch.searchsorted(mids, y.abs().contiguous()), torch.searchsorted(mids, y.abs().contiguous(), right=True)
    return s, torch.sign(y) * vals[torch.where(lo % 2 == 0, lo, hi)]


@pytest.mark.parametrize("order", ["nhd", "hnd"])
@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
@pytest.mark.parametrize("new", ["bf16", "f16", "f32"])
@pytest.mark.parametrize("rows,Hkv,D,P", [(1, 1, 64, 16), (300, 2, 128, 24), (65, 8, 256, 32)])
def test_append_quantizes_to_the_nearest_code(cuda_lib, rows, Hkv, D, P, new, fmt, order):
    rng = np.random.default_rng(rows + D)
    pages = rows // P + 2
    k, v = _empty_pool(pages, P, Hkv, D, torch.int8, order, 2)
    dt = torch.int8 if fmt == "i8" else torch.float8_e4m3fn
    k, v = k.view(dt), v.view(dt)
    ks = torch.full((pages * P, Hkv + 1), 7.0, device="cuda")[:, :Hkv]
    vs = torch.full((pages * P, Hkv + 1), 9.0, device="cuda")[:, :Hkv]
    g = torch.Generator().manual_seed(rows)
    kn, vn = (torch.randn(rows, Hkv, D, generator=g).to(DT[new]) for _ in range(2))
    # quotients on the border between codes: small whole numbers beside the amax
    kn[0, 0] = torch.arange(D).to(DT[new]) % 64 - 31
    kn[0, 0, 0] = 448.0 if fmt == "e4m3" else 127.0
    vn[0, 0] = (torch.arange(D) % 255 - 127).to(DT[new]) * 0.5
    vn[-1, -1] = 0
    slot = _slots(rng, rows, pages, P)
    slot[0] = pages * P - 1
    slot[1:] = np.where(slot[1:] == pages * P - 1, -1, slot[1:])
    wk, wv, wks, wvs = k.cpu().float(), v.cpu().float(), ks.cpu().clone(), vs.cpu().clone()
    for new_rows, w, ws in ((kn, wk, wks), (vn, wv, wvs)):
        s, y = _codes64(new_rows, fmt)
        for t, sl in enumerate(slot):
            if 0 <= sl < pages * P:
                w[sl // P, sl % P], ws[sl] = y[t].float(), s[t]
    A.append_paged(kn.cuda(), vn.cuda(), i32(slot).cuda(), k, v, k_scale=ks, v_scale=vs)
    torch.cuda.synchronize()
    assert torch.equal(ks.cpu(), wks) and torch.equal(vs.cpu(), wvs)
    for got, want in ((k.cpu().float(), wk), (v.cpu().float(), wv)):   # (cells that are not written may hold NaN codes)
        off = (got != want) & ~(got.isnan() & want.isnan())
        assert not off.any(), (off.nonzero()[:5], got[off][:5], want[off][:5])


@pytest.mark.parametrize("fmt", ["e4m3", "i8"])
def test_append_of_non_finite_rows_gives_non_finite_values(cuda_lib, fmt):
    dt = torch.int8 if fmt == "i8" else torch.float8_e4m3fn
    k = torch.zeros(1, 16, 1, 128, dtype=torch.int8, device="cuda").view(dt)
    v = k.clone()
    ks, vs = torch.zeros(16, 1, device="cuda"), torch.zeros(16, 1, device="cuda")
    kn = torch.randn(4, 1, 128, device="cuda")
    vn = torch.full((4, 1, 128), 1e-45, device="cuda")      # a scale that rounds to 0
    kn[0, 0, 3], kn[1, 0, 4], kn[2, 0, 5] = math.nan, math.inf, -math.inf
    A.append_paged(kn, vn, i32([2, 3, 4, 5]).cuda(), k, v, k_scale=ks, v_scale=vs)
    got = (k.float()[0, :, 0] * ks)
    assert torch.isnan(got[2:5]).any(-1).all() and torch.isfinite(got[5]).all()
    assert (v.float()[0, :, 0] * vs == 0).all()


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------

class Case:
    """A pool, tables and rows; `groups` (rows per group, shared cells) makes tables that begin alike."""

    def __init__(self, seed, ends, *, Hq=8, Hkv=2, D=128, P=16, cache="bf16", q="bf16", out=None, order="nhd",
                 begins=None, row_table=None, groups=None, sinks=False, alibi=False, softcap=0.0, garbage=True,
                 scale=None):
        rng, g = np.random.default_rng(seed), torch.Generator().manual_seed(seed)
        R = len(ends)
        n_tab = R if row_table is None else max(row_table) + 1
        lens = [0] * n_tab
        for r, e in enumerate(ends):
            t = r if row_table is None else row_table[r]
            lens[t] = max(lens[t], e)
        held = [-(-x // P) for x in lens]
        width = max(held) + 2
        pages = sum(held) + 3
        ids = rng.permutation(pages)
        table = np.full((n_tab, width), -1, dtype=np.int64)
        at = 0
        for t in range(n_tab):
            table[t, :held[t]] = ids[at:at + held[t]]
            at += held[t]
        self.kw = dict(scale=scale if scale is not None else 1 / math.sqrt(D), softcap=softcap)
        self.groups = None
        if groups is not None:
            begin = np.concatenate([[0], np.cumsum([n for n, _ in groups])])
            for (n, L), r0 in zip(groups, begin):
                first = r0 if row_table is None else row_table[r0] if n else 0
                for r in range(r0, r0 + n):
                    t = r if row_table is None else row_table[r]
                    table[t, :L // P] = table[first, :L // P]
            self.groups = dict(group_begin=i32(begin), group_len=i32([L for _, L in groups]))
        shape = (pages, Hkv, P, D) if order == "hnd" else (pages, P, Hkv, D)
        mk = lambda: (torch.randn(shape, generator=g).transpose(1, 2) if order == "hnd" else
                      torch.randn(shape, generator=g))
        k, v = mk(), mk()
        if groups is not None:    # a partly shared page: copies of the first row's cells
            for (n, L), r0 in zip(groups, begin):
                part = L % P
                for r in range(r0 + 1, r0 + n):
                    t, f = (r, r0) if row_table is None else (row_table[r], row_table[r0])
                    if part and t != f:
                        for x in (k, v):
                            x[table[t, L // P], :part] = x[table[f, L // P], :part]
        self.scales = {}
        if cache in ("e4m3", "i8"):
            ks, kc = _codes64(k, cache)
            vs, vc = _codes64(v, cache)
            dt = torch.int8 if cache == "i8" else torch.float8_e4m3fn
            k, v = kc.to(dt), vc.to(dt)
            self.scales = dict(k_scale=ks.reshape(pages * P, Hkv).contiguous(),
                               v_scale=vs.reshape(pages * P, Hkv).contiguous())
        else:
            k, v = k.to(DT[cache]), v.to(DT[cache])
        if garbage and cache in DT:   # cells that no row sees hold what they like
            seen = torch.zeros(pages * P, dtype=torch.bool)
            for r in range(R):
                t = r if row_table is None else row_table[r]
                c = np.arange(max(0, begins[r]) if begins is not None else 0, min(ends[r], width * P))
                seen[table[t][c // P] * P + c % P] = True
            hidden = (~seen).reshape(pages, P)
            k[hidden], v[hidden] = math.nan, math.inf
        self.k, self.v, self.table = k, v, i32(table)
        self.q = torch.randn(R, Hq, D, generator=g).to(DT[q if cache in ("e4m3", "i8") else cache])
        self.ends, self.begins = i32(ends), None if begins is None else i32(begins)
        self.row_table = None if row_table is None else i32(row_table)
        self.sinks = torch.randn(Hq, generator=g) if sinks else None
        self.slopes = torch.tensor([2.0 ** (-8 * (h + 1) / Hq) for h in range(Hq)]) if alibi else None
        self.out_dtype = DT[out] if out else self.q.dtype

    def expected(self):
        return ref.attention(self.q, self.k, self.v, self.table, self.ends, row_begin=self.begins,
                             row_table=self.row_table, slopes=self.slopes, sinks=self.sinks, **self.kw, **self.scales)

    def args(self, op, narrow=False):
        # decode_shared runs row by row where the tables cannot hold much: tables wide enough that it does not (the
        # entries behind a row's pages are never read), unless narrow
        cell = len(self.ends) * self.k.shape[2] * self.k.shape[3] * 4
        cols = self.table.shape[1] if narrow or op != A.OP_DECODE_SHARED else (65 << 20) // (cell * self.k.shape[1]) + 1
        table = torch.full((self.table.shape[0], max(cols, self.table.shape[1])), -7, dtype=I32)
        table[:, :self.table.shape[1]] = self.table
        up = lambda t: None if t is None else t.cuda()
        like = lambda t: torch.empty_strided(t.shape, t.stride(), dtype=t.dtype, device="cuda").copy_(t)
        self.dev = dict(q=up(self.q), k=like(self.k), v=like(self.v), table=up(table), ends=up(self.ends),
                        out=torch.full(self.q.shape, math.nan, dtype=self.out_dtype, device="cuda"))
        self.opt = dict(row_begin=up(self.begins), row_table=up(self.row_table), alibi_slopes=up(self.slopes),
                        sinks=up(self.sinks), **{n: up(t) for n, t in self.scales.items()})
        if op == A.OP_DECODE_SHARED and self.groups is not None:
            self.opt.update({n: up(t) for n, t in self.groups.items()})
        d = self.dev
        return A.make_paged_args(d["q"], d["k"], d["v"], d["out"], d["table"], d["ends"], **self.kw, **self.opt)

    def run(self, op, narrow=False):
        a = self.args(op, narrow)
        ws = poisoned_workspace(A.paged_workspace_size(a, op))
        fn = A.attn_decode_paged_args if op == A.OP_DECODE_PAGED else A.attn_decode_shared_args
        fn(a, ws=ws)
        torch.cuda.synchronize()
        return self.dev["out"]


def check(case, op=A.OP_DECODE_PAGED, want=None, narrow=False):
    got = case.run(op, narrow)
    A.check_device_status()
    want = case.expected() if want is None else want
    compare(got, want, 1e-5, 2e-2)
    return got, want


@pytest.mark.parametrize("order", ["nhd", "hnd"])
@pytest.mark.parametrize("P", [16, 48, 128])
@pytest.mark.parametrize("D,Hq,Hkv,cache", [(64, 4, 4, "bf16"), (128, 8, 2, "bf16"), (256, 6, 2, "f16"),
                                            (128, 16, 1, "f16"), (64, 7, 1, "f16"), (256, 24, 2, "bf16")])
def test_paged_16_bit(cuda_lib, D, Hq, Hkv, cache, P, order):
    check(Case(D + P, [1, 15, 16, 17, 700, 0, 333], D=D, Hq=Hq, Hkv=Hkv, cache=cache, P=P, order=order))


@pytest.mark.parametrize("P", [16, 32, 80])
@pytest.mark.parametrize("D,Hq,Hkv,q", [(128, 8, 2, "bf16"), (128, 8, 1, "f16"), (256, 3, 3, "bf16")])
@pytest.mark.parametrize("cache", ["e4m3", "i8"])
def test_paged_one_byte(cuda_lib, cache, D, Hq, Hkv, q, P):
    check(Case(D + P, [1, 16, 31, 500, 0, 129], D=D, Hq=Hq, Hkv=Hkv, cache=cache, q=q, P=P))


@pytest.mark.parametrize("over", [dict(sinks=True), dict(alibi=True), dict(softcap=20.0),
                                  dict(sinks=True, alibi=True, softcap=5.0), dict(out="f32"),
                                  dict(scale=0.0), dict(cache="f16", out="bf16")])
def test_paged_features(cuda_lib, over):
    check(Case(11, [900, 64, 0, 3], P=32, **over))


@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_paged_windows(cuda_lib, cache):
    ends = [900, 900, 900, 40, 40, 40, 17]
    begins = [0, 123, 899, 40, 41, -5, 16]
    check(Case(12, ends, begins=begins, cache=cache, alibi=True, sinks=False))


def test_paged_rows_of_one_table(cuda_lib):
    """Rows that read one table, more rows than are planned in the kernel (64)."""
    ends = list(range(1, 131))
    check(Case(13, ends, row_table=[0] * 130, P=48, Hq=4, Hkv=2, D=64))


def test_paged_many_rows(cuda_lib):
    rng = np.random.default_rng(14)
    check(Case(14, rng.integers(0, 90, 200).tolist(), Hq=4, Hkv=1, D=64, P=16, sinks=True))


def test_paged_range_past_the_table(cuda_lib):
    """A range that ends past the table is clipped; distances keep row_end as given."""
    c = Case(15, [100, 64], P=16, alibi=True)
    c.table = c.table[:, :4].contiguous()
    check(c)


def test_paged_strided_q_and_out(cuda_lib):
    c = Case(16, [100, 64, 7], Hq=4, Hkv=2, D=64)
    want = c.expected()
    a = c.args(A.OP_DECODE_PAGED)
    big = torch.zeros(3, 9, 64, dtype=c.q.dtype, device="cuda")
    big[:, 2:6] = c.dev["q"]
    out = torch.full((3, 11, 64), 5.0, dtype=torch.float32, device="cuda")
    d = c.dev
    A.decode_paged(big[:, 2:6], d["k"], d["v"], out[:, 3:7], d["table"], d["ends"], **c.kw)
    torch.cuda.synchronize()
    compare(out[:, 3:7], want, 1e-5, 2e-2)
    assert (out[:, :3] == 5).all() and (out[:, 7:] == 5).all()
    del a


@pytest.mark.parametrize("op", [A.OP_DECODE_PAGED, A.OP_DECODE_SHARED])
def test_nan_and_infinities_in_seen_cells(cuda_lib, op):
    """NaN in a visible V stays in its element, NaN in a visible K takes the row, nothing else is touched."""
    c = Case(17, [300, 300, 200], Hq=4, Hkv=2, D=64, P=16, groups=[(2, 192), (1, 100)])
    slot = lambda r, cell: (int(c.table[r, cell // 16]), cell % 16)
    p, o = slot(1, 250)
    c.v[p, o, 0, 5] = math.nan
    p, o = slot(2, 150)
    c.k[p, o, 1, 7] = math.nan
    got, want = check(c, op)
    assert np.isnan(want[1, :2, 5]).all() and np.isnan(want).sum() == 2 + 2 * 64


@pytest.mark.parametrize("op", [A.OP_DECODE_PAGED, A.OP_DECODE_SHARED])
def test_bad_ids_read_as_zeros_and_are_recorded(cuda_lib, op):
    c = Case(18, [64, 64, 40], P=16, D=64, garbage=False, groups=[(2, 48)])
    good = c.table.clone()
    c.table[1, 3] = c.k.shape[0]       # an id outside the pool, in a range
    c.table[2, 2] = -1
    c.table[0, 4] = 1 << 30            # and one that no range reaches
    got = c.run(op)
    with pytest.raises(A.AttnError, match="INVALID_ARG"):
        A.check_device_status()
    zero = c.k.shape[0]
    c.k = torch.cat([c.k, torch.zeros_like(c.k[:1])])
    c.v = torch.cat([c.v, torch.zeros_like(c.v[:1])])
    c.table = good
    c.table[1, 3] = c.table[2, 2] = zero
    compare(got, c.expected(), 1e-5, 2e-2)


@pytest.mark.parametrize("op", [A.OP_DECODE_PAGED, A.OP_DECODE_SHARED])
def test_row_table_outside_the_tables(cuda_lib, op):
    c = Case(19, [64, 64], P=16, D=64, row_table=[0, 1])
    want = c.expected()
    want[1] = 0
    c.row_table[1] = 2
    got = c.run(op)
    with pytest.raises(A.AttnError, match="INVALID_ARG"):
        A.check_device_status()
    compare(got, want, 1e-5, 2e-2)


def test_no_pages_and_no_rows(cuda_lib):
    k = torch.zeros(0, 16, 2, 64, dtype=torch.bfloat16, device="cuda")
    q = torch.randn(2, 4, 64, device="cuda").to(torch.bfloat16)
    out = torch.full_like(q, 3.0)
    table = torch.zeros(2, 4, dtype=I32, device="cuda")
    A.decode_paged(q, k, k, out, table, i32([9, 0]).cuda(), scale=1.0)
    torch.cuda.synchronize()
    assert (out == 0).all()
    A.decode_paged(q[:0], k, k, out[:0], table, i32([]).cuda(), scale=1.0)
    A.check_device_status()


def test_offsets_past_32_bits(cuda_lib):
    """A pool of more than 2^32 elements: pages at its end and scattered rows."""
    P, Hkv, D = 64, 8, 256
    pages = (1 << 32) // (P * Hkv * D) + 50
    k = torch.zeros(pages, P, Hkv, D, dtype=torch.bfloat16, device="cuda")
    v = torch.zeros_like(k)
    use = [pages - 1, 3, pages - 2, pages // 2]
    g = torch.Generator().manual_seed(1)
    ks, vs = (torch.randn(4 * P, Hkv, D, generator=g).to(torch.bfloat16) for _ in range(2))
    slot = i32(np.concatenate([np.arange(P) + u * P for u in use])).cuda()
    A.append_paged(ks.cuda(), vs.cuda(), slot, k, v)
    q = torch.randn(2, 8, D, generator=g).to(torch.bfloat16)
    table = i32([use, use])
    ends = i32([4 * P, 3 * P + 5])
    want = ref.attention(q, ks.reshape(4, P, Hkv, D), vs.reshape(4, P, Hkv, D), i32([[0, 1, 2, 3]] * 2), ends,
                         scale=0.06)
    for groups in ({}, dict(group_begin=i32([0, 2]).cuda(), group_len=i32([2 * P + 9]).cuda())):
        out = torch.empty(2, 8, D, dtype=torch.bfloat16, device="cuda")
        (A.decode_shared if groups else A.decode_paged)(q.cuda(), k, v, out, table.cuda(), ends.cuda(), scale=0.06,
                                                        **groups)
        compare(out, want, 1e-5, 2e-2)
    A.check_device_status()


# ---------------------------------------------------------------------------
# shared prefixes
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("order", ["nhd", "hnd"])
@pytest.mark.parametrize("P", [16, 48, 128, 256])
@pytest.mark.parametrize("D,Hq,Hkv,cache", [(64, 4, 4, "bf16"), (128, 8, 2, "bf16"), (256, 6, 2, "f16"),
                                            (128, 16, 1, "f16"), (64, 7, 1, "f16"), (256, 24, 2, "bf16")])
def test_shared(cuda_lib, D, Hq, Hkv, cache, P, order):
    ends = [300, 301, 450, 299, 70, 64, 64, 700, 20]
    check(Case(D + P, ends, D=D, Hq=Hq, Hkv=Hkv, cache=cache, P=P, order=order,
               groups=[(4, 299), (3, 64), (1, 600)]), A.OP_DECODE_SHARED)


@pytest.mark.parametrize("over", [dict(sinks=True), dict(alibi=True), dict(softcap=20.0), dict(softcap=0.5),
                                  dict(sinks=True, alibi=True, softcap=5.0), dict(out="f32"), dict(scale=0.0),
                                  dict(scale=-0.3), dict(cache="f16", out="bf16"), dict(cache="f16", softcap=30.0)])
def test_shared_features(cuda_lib, over):
    check(Case(21, [500, 520, 640, 500, 90], P=32, groups=[(4, 500)], **over), A.OP_DECODE_SHARED)


@pytest.mark.parametrize("n,G", [(1, 1), (31, 4), (33, 4), (65, 4), (130, 1), (257, 1), (19, 7), (40, 12)])
def test_shared_group_sizes(cuda_lib, n, G):
    """Rows that fill their tiles partly, exactly, and over several tiles."""
    rng = np.random.default_rng(n)
    ends = (200 + rng.integers(0, 40, n)).tolist()
    check(Case(22 + n, ends, P=16, Hq=2 * G, Hkv=2, D=64, groups=[(n, 200)]), A.OP_DECODE_SHARED)


@pytest.mark.parametrize("tokens,start", [(1, 0), (5, 0), (130, 0), (200, 77), (300, 1000)])
@pytest.mark.parametrize("alibi", [False, True])
def test_shared_prompt(cuda_lib, tokens, start, alibi):
    """A prompt's rows: one table, every row one cell more, the whole context shared."""
    ends = [start + 1 + i for i in range(tokens)]
    check(Case(23 + tokens, ends, P=16, Hq=4, Hkv=2, D=128, row_table=[0] * tokens, alibi=alibi,
               groups=[(tokens, start + tokens)]), A.OP_DECODE_SHARED)


def test_shared_prompt_with_nan_in_a_later_token(cuda_lib):
    """A token whose V is NaN reaches the rows that see it and no earlier one."""
    n = 200
    c = Case(24, [i + 1 for i in range(n)], P=16, Hq=2, Hkv=1, D=64, row_table=[0] * n, groups=[(n, n)])
    c.v[int(c.table[0, 150 // 16]), 150 % 16, 0, 3] = math.nan
    c.v[int(c.table[0, 160 // 16]), 160 % 16, 0, 9] = math.inf
    got, want = check(c, A.OP_DECODE_SHARED)
    assert np.isnan(want[:, 0, 3]).sum() == 50


def test_shared_edges(cuda_lib):
    """Groups of no rows, prefixes of no cells, rows that end inside the prefix or see nothing, rows of no group,
    a prefix past the table, windows that begin inside the prefix or behind it."""
    ends = [100, 40, 0, 130, 64, 64, 90, 200, 210]
    begins = [0, 0, 0, 70, 10, 60, 0, 0, 205]
    for grp in ([(4, 96), (0, 50), (2, 64), (1, 0)], [(0, 0)], [(4, 97), (2, -3), (3, 10_000)], [(9, 33)]):
        c = Case(25, ends, P=16, Hq=4, Hkv=2, D=64, begins=begins, row_table=[0, 0, 0, 0, 1, 1, 2, 2, 2], groups=grp,
                 garbage=False)
        check(c, A.OP_DECODE_SHARED)
    check(Case(26, ends, P=16, Hq=4, Hkv=2, D=64, begins=begins), A.OP_DECODE_SHARED)   # no groups given


@pytest.mark.parametrize("begin", [[0, 5, 3], [0, 2, 9], [-1, 2, 4]])
def test_shared_groups_that_cannot_be(cuda_lib, begin):
    c = Case(27, [100, 120, 90, 99], P=16, Hq=4, Hkv=2, D=64, groups=[(2, 64), (2, 32)])
    c.groups["group_begin"] = i32(begin)
    got = c.run(A.OP_DECODE_SHARED)
    with pytest.raises(A.AttnError, match="INVALID_ARG"):
        A.check_device_status()
    compare(got, c.expected(), 1e-5, 2e-2)


@pytest.mark.parametrize("cache", ["e4m3", "i8"])
def test_shared_one_byte(cuda_lib, cache):
    check(Case(28, [300, 301, 450, 299], D=128, P=16, cache=cache, groups=[(4, 299)]), A.OP_DECODE_SHARED)


def test_shared_over_narrow_tables(cuda_lib):
    """Tables that hold little are read row by row: the same result, and group arrays that cannot be do not matter."""
    c = Case(34, [300, 301, 450, 299], D=64, P=16, groups=[(4, 299)], sinks=True)
    check(c, A.OP_DECODE_SHARED, narrow=True)


def test_shared_many_blocks(cuda_lib):
    """More blocks than the planner keeps in shared memory, and more units than runs."""
    n = 2500
    rng = np.random.default_rng(35)
    table_of = (np.arange(n) // 2).tolist()
    ends = (20 + rng.integers(0, 30, n)).tolist()
    check(Case(35, ends, D=64, P=16, Hq=2, Hkv=1, row_table=table_of, groups=[(2, 25)] * (n // 2)), A.OP_DECODE_SHARED)


def test_shared_is_deterministic(cuda_lib):
    c = Case(29, [2000 + i for i in range(70)], P=16, Hq=8, Hkv=2, D=64, groups=[(40, 1990), (30, 1500)])
    first = c.run(A.OP_DECODE_SHARED).clone()
    for _ in range(3):
        assert torch.equal(first, c.run(A.OP_DECODE_SHARED))


# ---------------------------------------------------------------------------
# a serving loop
# ---------------------------------------------------------------------------

def _serve(graph, cache="bf16"):
    """Sequences that start, grow, end and start again; every step's rows are checked against the keys and values
    that their sequence was given."""
    rng, gen = np.random.default_rng(30), torch.Generator().manual_seed(30)
    n, P, width, n_pages, T, Hq, Hkv, D = 6, 16, 12, 40, 48, 4, 2, 128
    dt = {"bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn}[cache]
    k, v = (torch.zeros(n_pages, P, Hkv, D, device="cuda").to(dt) for _ in range(2))
    sc = {} if cache == "bf16" else dict(k_scale=torch.zeros(n_pages * P, Hkv, device="cuda"),
                                         v_scale=torch.zeros(n_pages * P, Hkv, device="cuda"))
    z = lambda *s: torch.zeros(*s, dtype=I32, device="cuda")
    table, ring = z(n, width) - 1, torch.randperm(n_pages, generator=gen).to(I32).cuda()
    new_len = z(n)
    q, kn, vn = (torch.zeros(T, h, D, dtype=torch.bfloat16, device="cuda") for h in (Hq, Hkv, Hkv))
    out = torch.zeros(T, Hq, D, dtype=torch.bfloat16, device="cuda")
    lens, state = z(n), i32([7, n_pages]).cuda()
    pa = A.make_page_args(lens, new_len, table, ring, state, page_size=P, n_rows=T)
    o = pa.outputs
    aa = A.make_append_args(kn, vn, o.slot, k, v, **sc)
    row_table = z(T)
    da = A.make_paged_args(q, k, v, out, table, o.row_end, scale=0.09, row_table=row_table, **sc)
    sa = A.make_paged_args(q, k, v, out, table, o.row_end, scale=0.09, row_table=row_table, group_begin=o.seq_row,
                           group_len=o.seq_len, **sc)
    ws = poisoned_workspace(max(A.paged_workspace_size(da, A.OP_DECODE_PAGED),
                                A.paged_workspace_size(sa, A.OP_DECODE_SHARED)))
    out2 = torch.zeros_like(out)

    def step():
        A.attn_page_tables_args(pa)
        A.attn_append_paged_args(aa)
        row_table.copy_(o.row_seq)
        A.attn_decode_shared_args(sa, ws=ws)
        out2.copy_(out)
        A.attn_decode_paged_args(da, ws=ws)
        lens.copy_(o.seq_len)
        state.copy_(o.free_state)

    g = None
    if graph:
        keep = [t.clone() for t in (ring, state)]
        step()                    # with no rows; warm-up before the capture
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step()
        ring.copy_(keep[0])
        state.copy_(keep[1])
        lens.zero_()
    kept = [[torch.zeros(0, Hkv, D), torch.zeros(0, Hkv, D)] for _ in range(n)]
    for it in range(14):
        cur = lens.tolist()
        new = [int(rng.choice([0, 1, 1, 1, 9, 20])) if c < width * P - 20 else -1 for c in cur]
        if it % 4 == 3:
            new[int(rng.integers(n))] = -1
        while sum(max(x, 0) for x in new) > T:
            new[int(np.argmax(new))] = 1
        new_len.copy_(i32(new))
        rows = [torch.randn(T, h, D, generator=gen).to(torch.bfloat16) for h in (Hq, Hkv, Hkv)]
        for t, r in zip((q, kn, vn), rows):
            t.copy_(r)
        g.replay() if g else step()
        torch.cuda.synchronize()
        A.check_device_status()
        got_len, t = lens.tolist(), 0
        want = np.zeros((T, Hq, D))
        for i in range(n):
            if new[i] < 0:
                assert got_len[i] == 0
                kept[i] = [torch.zeros(0, Hkv, D)] * 2
                continue
            r0, t = t, t + new[i]
            if got_len[i] == cur[i]:
                continue               # nothing new, or no page was left for it
            assert got_len[i] == cur[i] + new[i]
            for x, r in ((0, rows[1]), (1, rows[2])):
                y = r[r0:t].float()
                if cache == "e4m3":
                    s, c = _codes64(y, "e4m3")
                    y = (c * s.double()[..., None]).float()
                kept[i][x] = torch.cat([kept[i][x], y])
            m = len(kept[i][0])
            pad = lambda y: torch.cat([y, torch.zeros(-m % 16, Hkv, D)]).reshape(-1, 16, Hkv, D)
            ends = i32([cur[i] + 1 + j for j in range(new[i])])
            tab = i32([list(range(-(-m // 16)))])
            want[r0:t] = ref.attention(rows[0][r0:t], pad(kept[i][0]), pad(kept[i][1]), tab, ends, scale=0.09,
                                       row_table=[0] * new[i])
        compare(out, want, 1e-5, 2e-2, f"step {it}")
        compare(out2, want, 1e-5, 2e-2, f"step {it}, shared")
        free = state.tolist()[1]
        assert free + sum(-(-x // P) for x in got_len) == n_pages      # no page is lost


@pytest.mark.parametrize("graph", [False, True])
@pytest.mark.parametrize("cache", ["bf16", "e4m3"])
def test_serving_loop(cuda_lib, graph, cache):
    _serve(graph, cache)


def test_two_streams_with_workspaces_of_their_own(cuda_lib):
    cases = [Case(31, [900, 700], P=16, sinks=True), Case(32, [400, 1300], P=16, groups=[(2, 390)])]
    want = [c.expected() for c in cases]
    ops = [A.OP_DECODE_PAGED, A.OP_DECODE_SHARED]
    args = [c.args(op) for c, op in zip(cases, ops)]
    ws = [poisoned_workspace(A.paged_workspace_size(a, op)) for a, op in zip(args, ops)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in cases]
    for _ in range(5):
        A.attn_decode_paged_args(args[0], ws=ws[0], stream=streams[0])
        A.attn_decode_shared_args(args[1], ws=ws[1], stream=streams[1])
    torch.cuda.synchronize()
    for c, w in zip(cases, want):
        compare(c.dev["out"], w, 1e-5, 2e-2)


def test_python_refusals(cuda_lib):
    c = Case(33, [40, 50], P=16)
    a = c.args(A.OP_DECODE_PAGED)
    d = c.dev
    with pytest.raises(ValueError, match="share shape"):
        A.make_paged_args(d["q"], d["k"], d["v"][:2], d["out"], d["table"], d["ends"], scale=1.0)
    with pytest.raises(ValueError, match="row_end"):
        A.make_paged_args(d["q"], d["k"], d["v"], d["out"], d["table"], d["ends"].long(), scale=1.0)
    with pytest.raises(ValueError, match="one CUDA device"):
        A.make_paged_args(d["q"], d["k"], d["v"], d["out"], d["table"], d["ends"], scale=1.0, sinks=torch.zeros(8))
    with pytest.raises(ValueError, match="group_begin"):
        A.make_paged_args(d["q"], d["k"], d["v"], d["out"], d["table"], d["ends"], scale=1.0,
                          group_len=d["ends"])
    with pytest.raises(A.AttnError, match="workspace"):
        A.attn_decode_paged_args(a, ws=torch.empty(256, dtype=torch.uint8, device="cuda"))
    with pytest.raises(ValueError, match="heads and dim"):
        A.make_append_args(d["q"], d["q"], d["ends"], d["k"], d["v"])
    with pytest.raises(ValueError, match="seq_len"):
        A.make_page_args(d["ends"].float(), d["ends"], d["table"], d["ends"], d["ends"], page_size=16, n_rows=4)
