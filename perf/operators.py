"""The paged-cache operators as they are measured: their cases, inputs, plain
forms and 64-bit values.

Four operators that a serving step runs one after the other:
  tables  block tables and slot maps built from the sequences' lengths;
  append  the step's K/V rows written through the slot map;
  paged   decode attention of single rows over a paged cache;
  shared  the same for groups of rows whose tables begin with the same cells
          (a common prompt; a prompt's own rows, which share their context).
With ``own`` false every operator is computed by elementary torch operations
in 32 bits, with ``own`` true by the library's calls.
"""
from __future__ import annotations

import math
import random

import numpy as np
import torch

own = False

_TYPES = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16, "e4m3": torch.float8_e4m3fn,
          "i8": torch.int8}
_BYTES = {"f32": 4, "f16": 2, "bf16": 2, "e4m3": 1, "i8": 1}


# ---------------------------------------------------------------------------
# cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # One decode step's bookkeeping of a 16-sequence batch: the smallest call, all latency.
        dict(name="tables-step", op="tables", seqs=16, page=16, len_lo=1024, len_hi=8192, new_lo=1, new_hi=1,
             release=0.0),
        # A busy server's step: prompts of up to a few hundred tokens beside single tokens, and finished sequences.
        dict(name="tables-mixed", op="tables", seqs=509, page=64, len_lo=1, len_hi=16384, new_lo=1, new_hi=400,
             release=0.1),
        # The same 16 sequences' new rows.
        dict(name="append-step", op="append", rows=16, pad=0, hkv=8, dim=128, page=16, pages=64, new="bf16",
             cache="bf16", order="nhd"),
        # A prompt chunk's rows, into pages that keep each head's cells together; some rows are padding.
        dict(name="append-prompt", op="append", rows=14001, pad=47, hkv=4, dim=256, page=64, pages=256, new="f16",
             cache="f16", order="hnd"),
        # A chunk quantized on its way into a one-byte cache.
        dict(name="append-e4m3", op="append", rows=2048, pad=0, hkv=8, dim=128, page=32, pages=80, new="bf16",
             cache="e4m3", order="nhd"),
        # The GQA decode batch (16 sequences of 1024 to 8192 cells) over 16-cell pages.
        dict(name="paged-batch", op="paged", rows=16, len_lo=1024, len_hi=8192, hq=32, hkv=8, dim=128, page=16,
             cache="bf16", q="bf16", order="nhd", softcap=0.0, sinks=True, alibi=False, window=0),
        # One long sequence (latency of a single token at depth).
        dict(name="paged-long-row", op="paged", rows=1, len_lo=130857, len_hi=130857, hq=32, hkv=8, dim=128, page=64,
             cache="bf16", q="bf16", order="hnd", softcap=0.0, sinks=False, alibi=False, window=0),
        # A larger batch over a one-byte cache.
        dict(name="paged-e4m3", op="paged", rows=61, len_lo=1, len_hi=8192, hq=32, hkv=8, dim=128, page=32,
             cache="e4m3", q="bf16", order="nhd", softcap=0.0, sinks=False, alibi=False, window=0),
        # Few rows behind a short common prompt: latency of the two-part form.
        dict(name="shared-few", op="shared", groups=1, rows_lo=8, rows_hi=8, pre_lo=1024, pre_hi=1024, own_lo=1,
             own_hi=128, hq=32, hkv=8, dim=128, page=16, cache="bf16", order="nhd", softcap=0.0, sinks=False,
             alibi=False),
        # A batch behind one long system prompt.
        dict(name="shared-batch", op="shared", groups=1, rows_lo=64, rows_hi=64, pre_lo=8192, pre_hi=8192, own_lo=1,
             own_hi=1024, hq=32, hkv=8, dim=128, page=16, cache="bf16", order="nhd", softcap=0.0, sinks=True,
             alibi=False),
        # Several prompts at once, ragged in every direction, capped scores.
        dict(name="shared-groups", op="shared", groups=5, rows_lo=3, rows_hi=90, pre_lo=700, pre_hi=20000, own_lo=0,
             own_hi=700, hq=40, hkv=4, dim=64, page=48, cache="f16", order="hnd", softcap=50.0, sinks=False,
             alibi=True),
        # A prompt chunk at depth: 2048 rows of one sequence, row by row one cell more.
        dict(name="shared-prompt", op="prompt", tokens=2048, start=12000, hq=64, hkv=8, dim=128, page=64,
             cache="bf16", order="nhd", softcap=0.0, sinks=True, alibi=False),
    ]


def _log(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["tables", "append", "paged", "paged", "shared", "shared", "prompt"])
    if op == "tables":
        hi = _log(rng, 1, 400)
        return dict(op=op, seqs=_log(rng, 1, 600), page=rng.choice([1, 16, 24, 32, 64, 128]), len_lo=1,
                    len_hi=_log(rng, 16, 16384), new_lo=1, new_hi=hi, release=rng.choice([0.0, 0.05, 0.3]))
    if op == "append":
        cache, new = rng.choice([("bf16", "bf16"), ("f16", "f16"), ("e4m3", "bf16"), ("i8", "f16"), ("bf16", "f32")])
        dim, hkv, page = rng.choice([64, 128, 256]), rng.choice([1, 2, 4, 8]), rng.choice([8, 16, 48, 64])
        rows = _log(rng, 1, 12000 * 1024 // (dim * hkv)) if cache in ("bf16", "f16") else _log(rng, 1, 2048)
        rows = min(rows, 14000)
        pad = rng.choice([0, 5])
        return dict(op=op, rows=rows, pad=pad, hkv=hkv, dim=dim, page=page,
                    pages=(rows + page - 1) // page + 1 + rng.randrange(16), new=new, cache=cache,
                    order=rng.choice(["nhd", "hnd"]))
    dim = rng.choice([64, 128, 128, 256])
    hkv = rng.choice([1, 2, 4, 8])
    page = rng.choice([16, 32, 48, 64, 128])
    order = rng.choice(["nhd", "hnd"])
    softcap = rng.choice([0.0, 0.0, 30.0])
    sinks, alibi = rng.random() < 0.4, rng.random() < 0.25
    if op == "paged":
        cache = rng.choice(["bf16", "bf16", "f16", "e4m3", "i8"])
        g = rng.choice([1, 2, 4, 7, 8] if cache in ("e4m3", "i8") else [1, 2, 4, 5, 8, 12, 16])
        if cache in ("e4m3", "i8") and dim == 64:
            dim = 128
        rows = _log(rng, 1, 200)
        most = max(64, min(131072, 120_000_000 // (rows * hkv * dim)))
        return dict(op=op, rows=rows, len_lo=1, len_hi=_log(rng, 16, most), hq=hkv * g, hkv=hkv, dim=dim, page=page,
                    cache=cache, q=rng.choice(["bf16", "f16"]) if cache in ("e4m3", "i8") else cache, order=order,
                    softcap=softcap, sinks=sinks, alibi=alibi, window=rng.choice([0, 0, 777]))
    g = rng.choice([1, 2, 4, 7, 8, 12])
    cache = rng.choice(["bf16", "f16"])
    if op == "shared":
        groups = rng.randint(1, 5)
        hi = _log(rng, 1, 96)
        pre = _log(rng, 16, 20000)
        return dict(op=op, groups=groups, rows_lo=1, rows_hi=hi, pre_lo=min(16, pre), pre_hi=pre, own_lo=0,
                    own_hi=_log(rng, 1, 1000), hq=hkv * g, hkv=hkv, dim=dim, page=page, cache=cache, order=order,
                    softcap=softcap, sinks=sinks, alibi=alibi)
    return dict(op=op, tokens=_log(rng, 1, 1500), start=rng.choice([0, _log(rng, 1, 8000)]), hq=hkv * g, hkv=hkv,
                dim=dim, page=page, cache=cache, order=order, softcap=softcap, sinks=sinks, alibi=alibi)


# ---------------------------------------------------------------------------
# inputs
# ---------------------------------------------------------------------------

def _lens(rng, lo, hi, n):
    return rng.integers(lo, hi + 1, size=n)


def _sizes(case, lo, hi, n):
    """n whole numbers that the case alone settles (sizes of inputs and outputs; a seed only changes their order)."""
    r = random.Random(repr(sorted((k, v) for k, v in case.items() if k != "name")))
    return np.array([r.randint(lo, hi) for _ in range(n)], dtype=np.int64)


def _dev(a):
    return torch.from_numpy(np.ascontiguousarray(np.asarray(a, dtype=np.int32))).cuda()


def _normal(seed, shape, dtype):
    g = torch.Generator(device="cuda").manual_seed(seed)
    return torch.randn(shape, generator=g, device="cuda", dtype=torch.float32).to(dtype)


def _cache(seed, pages, page, hkv, dim, cache, order):
    """K, V [pages, page, hkv, dim] (order "hnd": the cells of a head lie together) and their scales or None."""
    def one(s):
        x = _normal(s, (pages, hkv, page, dim) if order == "hnd" else (pages, page, hkv, dim), torch.float32)
        x = x.transpose(1, 2) if order == "hnd" else x
        if cache in ("bf16", "f16"):
            return x.to(_TYPES[cache]), None
        scale = x.abs().amax(-1) / (448.0 if cache == "e4m3" else 127.0)
        y = x / scale[..., None]
        y = y.round().clamp(-127, 127).to(torch.int8) if cache == "i8" else y.to(torch.float8_e4m3fn)
        return y, scale.reshape(pages * page, hkv).contiguous()
    k, ks = one(seed)
    v, vs = one(seed + 1)
    return k, v, ks, vs


def _head_extras(case, seed):
    hq = case["hq"]
    sinks = _normal(seed + 7, (hq,), torch.float32) if case["sinks"] else None
    slopes = (torch.tensor([2.0 ** (-8.0 * (h + 1) / hq) for h in range(hq)], dtype=torch.float32, device="cuda")
              if case["alibi"] else None)
    return sinks, slopes


def _attention_state(case, seed):
    """Rows, tables and groups of an attention case, all lengths also on the host (as a scheduler has them)."""
    rng = np.random.default_rng(seed)
    op, P = case["op"], case["page"]
    if op == "paged":
        R = case["rows"]
        end = _lens(rng, case["len_lo"], case["len_hi"], R)
        begin = np.maximum(end - case["window"], 0) if case["window"] else np.zeros(R, dtype=np.int64)
        row_table, table_len, groups, pre = np.arange(R), end.copy(), None, None
        group_of = None
    elif op == "shared":
        n = rng.permutation(_sizes(case, case["rows_lo"], case["rows_hi"], case["groups"]))
        pre = _lens(rng, case["pre_lo"], case["pre_hi"], case["groups"])
        R = int(n.sum())
        groups = np.concatenate([[0], np.cumsum(n)])
        group_of = np.repeat(np.arange(case["groups"]), n)
        end = pre[group_of] + _lens(rng, case["own_lo"], case["own_hi"], R)
        begin = np.zeros(R, dtype=np.int64)
        row_table, table_len = np.arange(R), end.copy()
    else:   # prompt: one sequence, every row one cell more
        R = case["tokens"]
        end = case["start"] + 1 + np.arange(R)
        begin = np.zeros(R, dtype=np.int64)
        row_table, table_len = np.zeros(R, dtype=np.int64), np.array([case["start"] + R])
        groups, group_of, pre = np.array([0, R]), np.zeros(R, dtype=np.int64), np.array([case["start"] + R])
    # pages: a group's whole prefix pages are one set of pages named by all its tables
    n_tab = len(table_len)
    held = (table_len + P - 1) // P
    width = int(held.max()) + 1
    table = np.full((n_tab, width), -1, dtype=np.int64)
    total = int(held.sum())
    order = rng.permutation(total + 3)
    used = 0
    shared_pages = {}
    for i in range(n_tab):
        k0 = 0
        if op == "shared":
            g = int(group_of[i])
            k0 = int(pre[g]) // P
            if g not in shared_pages:
                shared_pages[g] = order[used:used + k0].copy()
                used += k0
            table[i, :k0] = shared_pages[g]
        k = int(held[i])
        table[i, k0:k] = order[used:used + max(k - k0, 0)]
        used += max(k - k0, 0)
    live = table[table >= 0]
    uniq, inv = np.unique(live, return_inverse=True)       # close the gaps: the pool holds what is used
    perm = rng.permutation(len(uniq) + 3)[:len(uniq)]
    table[table >= 0] = perm[inv]
    pages = len(uniq) + 3
    s = dict(case=case, end=end, begin=begin, row_table=row_table, table=table, groups=groups, pre=pre,
             group_of=group_of, pages=pages, R=R)
    s["k"], s["v"], s["ks"], s["vs"] = _cache(seed * 13 + 1, pages, P, case["hkv"], case["dim"], case["cache"],
                                              case["order"])
    qt = _TYPES[case.get("q", case["cache"])]
    s["q"] = _normal(seed * 13 + 5, (R, case["hq"], case["dim"]), qt)
    s["out"] = torch.empty((R, case["hq"], case["dim"]), dtype=qt, device="cuda")
    s["sinks"], s["slopes"] = _head_extras(case, seed * 13)
    s["scale"] = 1.0 / math.sqrt(case["dim"])
    s["d_table"], s["d_end"], s["d_begin"] = _dev(table), _dev(end), _dev(begin)
    s["d_row_table"] = None if op != "prompt" else _dev(row_table)
    if groups is not None:
        s["d_groups"], s["d_pre"] = _dev(groups), _dev(pre)
        # two rows of a group may both write a partly shared page: copies of the first row's cells
        if op == "shared":
            for g in range(len(pre)):
                part = int(pre[g]) % P
                rows = np.arange(groups[g], groups[g + 1])
                if part and len(rows) > 1:
                    pg = torch.from_numpy(table[rows, int(pre[g]) // P]).cuda()
                    for t in (s["k"], s["v"]):
                        t[pg[1:], :part] = t[pg[0], :part]
    return s


def _tables_state(case, seed):
    rng = np.random.default_rng(seed)
    n, P = case["seqs"], case["page"]
    ln = _lens(rng, case["len_lo"], case["len_hi"], n)
    # half of the sequences add the fewest tokens, the others a chunk of any size; some are finished
    new = _sizes(case, case["new_lo"], case["new_hi"], n)
    new[::2] = case["new_lo"]
    new[:int(case["release"] * n)] = -1
    new = rng.permutation(new)
    width = int((case["len_hi"] + case["new_hi"] + P - 1) // P)
    held = (ln + P - 1) // P
    spare = int(np.maximum((ln + np.maximum(new, 0) + P - 1) // P - held, 0).sum()) + 5
    pages = n * width + 5                       # a pool that holds every sequence at its longest
    ids = rng.permutation(pages)[:int(held.sum()) + spare]
    table = np.full((n, width), -1, dtype=np.int64)
    at = 0
    for i in range(n):
        table[i, :held[i]] = ids[at:at + held[i]]
        at += int(held[i])
    ring = np.full(pages, -1, dtype=np.int64)
    head = int(rng.integers(0, pages))
    ring[(head + np.arange(spare)) % pages] = ids[at:]
    rows = int(np.maximum(new, 0).sum())
    rows = max(1, (rows + 15) // 16 * 16)     # the step's padded row count
    keep = np.minimum(rng.integers(0, 3, size=n), held)
    s = dict(case=case, n=n, P=P, width=width, pages=pages, rows=rows, ln=ln, new=new, table=table, ring=ring,
             head=head, count=spare, keep=keep)
    s["d_len"], s["d_new"], s["d_table"], s["d_ring"] = _dev(ln), _dev(new), _dev(table), _dev(ring)
    s["d_state"], s["d_keep"] = _dev([head, spare]), _dev(keep)
    return s


def _append_state(case, seed):
    rng = np.random.default_rng(seed)
    P, pages, rows = case["page"], case["pages"], case["rows"]
    # consecutive positions of a few sequences: runs of cells inside random pages
    need = (rows + P - 1) // P
    pg = rng.permutation(pages)[:need]
    slot = (pg[:, None] * P + np.arange(P)[None, :]).reshape(-1)[:rows]
    slot = np.concatenate([slot, np.full(case["pad"], -1)])
    T = rows + case["pad"]
    s = dict(case=case, rows=rows, slot=slot)
    nt = _TYPES[case["new"]]
    s["k_new"] = _normal(seed * 7 + 1, (T, case["hkv"], case["dim"]), nt)
    s["v_new"] = _normal(seed * 7 + 2, (T, case["hkv"], case["dim"]), nt)
    s["k"], s["v"], s["ks"], s["vs"] = _cache(seed * 7 + 3, pages, P, case["hkv"], case["dim"], case["cache"],
                                              case["order"])
    s["d_slot"] = _dev(slot)
    s["d_slot64"] = s["d_slot"][:rows].long()
    return s


def prepare(case, seed):
    op = case["op"]
    if op == "tables":
        s = _tables_state(case, seed)
    elif op == "append":
        s = _append_state(case, seed)
    else:
        s = _attention_state(case, seed)
    if own:
        import attention_split_attn_b200 as A
        s["A"] = A
        if op == "tables":
            s["handle"] = A.make_page_args(s["d_len"], s["d_new"], s["d_table"], s["d_ring"], s["d_state"],
                                           page_size=s["P"], n_rows=s["rows"], n_keep=s["d_keep"])
        elif op == "append":
            s["handle"] = A.make_append_args(s["k_new"], s["v_new"], s["d_slot"], s["k"], s["v"], k_scale=s["ks"],
                                             v_scale=s["vs"])
        else:
            kw = dict(scale=s["scale"], softcap=case["softcap"], sinks=s["sinks"], alibi_slopes=s["slopes"],
                      row_table=s["d_row_table"], k_scale=s["ks"], v_scale=s["vs"],
                      row_begin=s["d_begin"] if case.get("window") else None)
            if s["groups"] is not None:
                kw.update(group_begin=s["d_groups"], group_len=s["d_pre"])
            s["handle"] = A.make_paged_args(s["q"], s["k"], s["v"], s["out"], s["d_table"], s["d_end"], **kw)
            op_id = A.OP_DECODE_SHARED if s["groups"] is not None else A.OP_DECODE_PAGED
            s["ws"] = torch.empty(max(1, A.paged_workspace_size(s["handle"], op_id)), dtype=torch.uint8,
                                  device="cuda")
    return s


# ---------------------------------------------------------------------------
# one pass
# ---------------------------------------------------------------------------

def run(s):
    op = s["case"]["op"]
    if not own:
        return {"tables": _plain_tables, "append": _plain_append, "paged": _plain_paged, "shared": _plain_shared,
                "prompt": _plain_shared}[op](s)
    A = s["A"]
    if op == "tables":
        o = A.attn_page_tables_args(s["handle"])
        return [s["d_table"], o.slot, o.row_seq, o.row_end, o.seq_row, o.seq_len, s["d_ring"], o.free_state]
    if op == "append":
        A.attn_append_paged_args(s["handle"])
        return _cache_values(s)
    if op == "paged":
        A.attn_decode_paged_args(s["handle"], ws=s["ws"])
    else:
        A.attn_decode_shared_args(s["handle"], ws=s["ws"])
    return s["out"]


def _cache_values(s):
    if s["ks"] is None:
        return [s["k"], s["v"]]
    sh = s["k"].shape
    return [s["k"].float() * s["ks"].view(sh[0], sh[1], sh[2], 1), s["v"].float() * s["vs"].view(sh[0], sh[1], sh[2], 1),
            s["ks"], s["vs"]]


def _plain_tables(s):
    P, W, NP, n, T = s["P"], s["width"], s["pages"], s["n"], s["rows"]
    ln, nn, table, ring = s["d_len"].long(), s["d_new"].long(), s["d_table"], s["d_ring"]
    head, count = s["d_state"][0].long(), s["d_state"][1].long()
    grow = nn.clamp(min=0)
    held = (ln + P - 1) // P
    fits = (ln + grow) <= W * P
    need = torch.where(fits, (ln + grow + P - 1) // P - held, 0)
    inc, rinc = need.cumsum(0), grow.cumsum(0)
    ok = (nn >= 0) & fits & ((need == 0) | (inc <= count)) & (rinc <= T)
    used = torch.where(ok & (need > 0), inc, 0).max()
    seq_len = torch.where(nn < 0, 0, torch.where(ok, ln + grow, ln))
    t = torch.arange(T, device="cuda")
    i = torch.searchsorted(rinc, t, right=True)
    valid = i < n
    i = i.clamp(max=n - 1)
    pos = ln[i] + t - (rinc - grow)[i]
    pi = pos // P
    fresh = ring[(head + (inc - need)[i] + pi - held[i]).clamp(min=0) % NP]
    old = table[i, pi.clamp(max=W - 1)]
    phys = torch.where(pi < held[i], old, fresh).long()
    good = valid & ok[i]
    slot = torch.where(good, phys * P + pos % P, -1)
    wide = torch.cat([table, torch.zeros_like(table[:, :1])], 1)
    wide[i, torch.where(good & (pos % P == 0), pi, W)] = phys.int()
    keep = s["d_keep"].long()
    rel = torch.where(nn < 0, (held - keep).clamp(min=0), 0)
    col = torch.arange(W, device="cuda")[None, :]
    mine = (nn < 0)[:, None] & (col >= keep[:, None]) & (col < held[:, None])
    dest = (head + count + (rel.cumsum(0) - rel)[:, None] + col - keep[:, None]) % NP
    more = torch.cat([ring, torch.zeros_like(ring[:1])])
    more[torch.where(mine, dest, NP)] = table
    state = torch.stack([(head + used) % NP, count - used + rel.sum()])
    zero = torch.zeros_like(rinc[:1])
    return [wide[:, :W], slot.int(), torch.where(valid, i, -1).int(), torch.where(good, pos + 1, 0).int(),
            torch.cat([zero, rinc]).int(), seq_len.int(), more[:NP], state.int()]


def _plain_append(s):
    P, n = s["case"]["page"], s["rows"]
    page, off = s["d_slot64"] // P, s["d_slot64"] % P
    for new, cache, scales in ((s["k_new"], s["k"], s["ks"]), (s["v_new"], s["v"], s["vs"])):
        x = new[:n]
        if scales is not None:
            e4 = s["case"]["cache"] == "e4m3"
            scale = (x.double().abs().amax(-1) / (448.0 if e4 else 127.0)).float()
            scales[s["d_slot64"]] = scale
            # 64 bits: a quotient next to the border between two codes has to fall on its own side of it
            x = x.double() / torch.where(scale == 0, 1.0, scale)[..., None].double()
            if e4:
                step = (((torch.frexp(x)[1].long() - 4).clamp(min=-9) + 1023) << 52).view(torch.float64)   # a power of 2
                x = (x / step).round() * step
            else:
                x = x.round()
        cache[page, off] = x.to(cache.dtype)
    return _cache_values(s)


def _cells(s, t, scales, pages):
    """Cells of the pages named by `pages` [...], in 32 bits: [..., len(pages) * P, hkv, dim]."""
    x = t[pages.long()].float()                                  # [..., n, P, hkv, dim]
    if scales is not None:
        sh = t.shape
        x = x * scales.view(sh[0], sh[1], sh[2], 1)[pages.long()]
    return x.flatten(-4, -3)


def _transform(s, x, dist):
    """Scores [..., hq-like, rows..., cells] after the cap and the distance bias."""
    if s["case"]["softcap"] > 0:
        x = s["case"]["softcap"] * torch.tanh(x / s["case"]["softcap"])
    if s["slopes"] is not None:
        x = x - dist
    return x


def _finish(s, x, sink):
    """exp(x - max) and the sums, with the sink as one more logit; rows that see nothing give weights of 0."""
    m = x.amax(-1, keepdim=True)
    if sink is not None:
        m = torch.maximum(m, sink)
    m = torch.where(m == -math.inf, 0.0, m)
    p = torch.exp(x - m)
    z = p.sum(-1, keepdim=True)
    if sink is not None:
        z = z + torch.exp(sink - m)
    return p / torch.where(z == 0, 1.0, z)


def _plain_paged(s):
    c = s["case"]
    P, hkv, G, D = c["page"], c["hkv"], c["hq"] // c["hkv"], c["dim"]
    n_pages = (int(s["end"].max()) + P - 1) // P
    step = max(1, int(2e9 // max(1, n_pages * P * hkv * D * 4)))     # rows at a time: 2 GB of cells
    cell = torch.arange(n_pages * P, device="cuda")
    for r0 in range(0, s["R"], step):
        r1 = min(s["R"], r0 + step)
        tab = s["d_table"][r0:r1, :n_pages].clamp(min=0)
        k, v = _cells(s, s["k"], s["ks"], tab), _cells(s, s["v"], s["vs"], tab)     # [r, N, hkv, D]
        q = s["q"][r0:r1].float().view(r1 - r0, hkv, G, D)
        x = torch.matmul(q, k.permute(0, 2, 3, 1)) * s["scale"]                      # [r, hkv, G, N]
        end, begin = s["d_end"][r0:r1, None, None, None], s["d_begin"][r0:r1, None, None, None]
        slopes = None if s["slopes"] is None else s["slopes"].view(1, hkv, G, 1)
        x = _transform(s, x, None if slopes is None else slopes * (end - 1 - cell))
        x = torch.where((cell < end) & (cell >= begin), x, -math.inf)
        p = _finish(s, x, None if s["sinks"] is None else s["sinks"].view(1, hkv, G, 1))
        s["out"][r0:r1] = torch.matmul(p, v.permute(0, 2, 1, 3)).reshape(r1 - r0, hkv * G, D)
    return s["out"]


def _plain_shared(s):
    """Per group: the scores of all its rows over the shared cells in one product per KV head, each row's own cells
    beside them, one softmax over both."""
    c = s["case"]
    P, hkv, G, D = c["page"], c["hkv"], c["hq"] // c["hkv"], c["dim"]
    for g in range(len(s["pre"])):
        r0, r1, L = int(s["groups"][g]), int(s["groups"][g + 1]), int(s["pre"][g])
        if r1 == r0:
            continue
        n = r1 - r0
        first = int(s["row_table"][r0])
        np_ = (L + P - 1) // P
        k = _cells(s, s["k"], None, s["d_table"][first, :np_].clamp(min=0))[:L]       # [L, hkv, D]
        v = _cells(s, s["v"], None, s["d_table"][first, :np_].clamp(min=0))[:L]
        far = int(s["end"][r0:r1].max())
        own_cells = far > L
        if own_cells:
            lo = L // P
            tab = s["d_table"][r0:r1, lo:(far + P - 1) // P].clamp(min=0)
            ko, vo = _cells(s, s["k"], None, tab), _cells(s, s["v"], None, tab)       # [n, M, hkv, D]
            at = lo * P + torch.arange(ko.shape[1], device="cuda")
        cell = torch.arange(L, device="cuda")
        end = s["d_end"][r0:r1, None, None]
        for h in range(hkv):
            q = s["q"][r0:r1, h * G:(h + 1) * G].float()                              # [n, G, D]
            sl = None if s["slopes"] is None else s["slopes"][h * G:(h + 1) * G].view(1, G, 1)
            sink = None if s["sinks"] is None else s["sinks"][h * G:(h + 1) * G].view(1, G, 1)
            x = torch.matmul(q.reshape(n * G, D), k[:, h].t()).view(n, G, L) * s["scale"]
            x = _transform(s, x, None if sl is None else sl * (end - 1 - cell))
            x = torch.where(cell < end, x, -math.inf)
            if own_cells:
                y = torch.matmul(q, ko[:, :, h].transpose(1, 2)) * s["scale"]         # [n, G, M]
                y = _transform(s, y, None if sl is None else sl * (end - 1 - at))
                y = torch.where((at >= L) & (at < end), y, -math.inf)
                x = torch.cat([x, y], -1)
            p = _finish(s, x, sink)
            o = torch.matmul(p[..., :L].reshape(n * G, L), v[:, h]).view(n, G, D)
            if own_cells:
                o = o + torch.matmul(p[..., L:], vo[:, :, h])
            s["out"][r0:r1, h * G:(h + 1) * G] = o
    return s["out"]


# ---------------------------------------------------------------------------
# work
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "tables":
        new = case["seqs"] * (1 + case["new_hi"]) / 2
        held = case["seqs"] * (case["len_lo"] + case["len_hi"]) / 2 / case["page"]
        # lengths, counts and first rows per sequence; three values per row; taken and released pages
        return {"bytes": int(20 * case["seqs"] + 12 * new + 8 * new / case["page"] + 8 * case["release"] * held),
                "flops": 0}
    if op == "append":
        n = case["rows"] * case["hkv"] * case["dim"] * 2
        b = n * (_BYTES[case["new"]] + _BYTES[case["cache"]]) + 4 * (case["rows"] + case["pad"])
        if case["cache"] in ("e4m3", "i8"):
            b += case["rows"] * case["hkv"] * 8
        return {"bytes": b, "flops": 3 * n if case["cache"] in ("e4m3", "i8") else 0}
    s = _shape(case)
    es, qs = _BYTES[case["cache"]], _BYTES[case.get("q", case["cache"])]
    cell = 2 * case["dim"] * es + (8 if es == 1 else 0)
    io = 2 * s["R"] * case["hq"] * case["dim"] * qs
    return {"bytes": int(s["cells"] * case["hkv"] * cell + io), "flops": int(4 * case["dim"] * case["hq"] * s["seen"])}


def _shape(case):
    """Expected rows, distinct cells read and (row, cell) pairs seen."""
    if case["op"] == "paged":
        mean = (case["len_lo"] + case["len_hi"]) / 2
        mean = min(mean, case["window"]) if case["window"] else mean
        return dict(R=case["rows"], cells=case["rows"] * mean, seen=case["rows"] * mean)
    if case["op"] == "shared":
        R = case["groups"] * (case["rows_lo"] + case["rows_hi"]) / 2
        pre, mine = (case["pre_lo"] + case["pre_hi"]) / 2, (case["own_lo"] + case["own_hi"]) / 2
        return dict(R=R, cells=case["groups"] * pre + R * mine, seen=R * (pre + mine))
    n = case["tokens"]
    return dict(R=n, cells=case["start"] + n, seen=n * case["start"] + n * (n + 1) / 2)


# ---------------------------------------------------------------------------
# 64-bit values, from the definitions
# ---------------------------------------------------------------------------

def exact(case, seed):
    op = case["op"]
    if op == "tables":
        return _exact_tables(_tables_state(case, seed))
    if op == "append":
        return _exact_append(_append_state(case, seed))
    s = _attention_state(case, seed)
    if s["R"] * case["hq"] * float(s["end"].max()) * case["dim"] > 3e12:
        return None
    return _exact_rows(s)


def _exact_tables(s):
    """A page at a time, sequence by sequence."""
    P, W, NP, T = s["P"], s["width"], s["pages"], s["rows"]
    table, ring = s["table"].copy(), s["ring"].copy()
    slot, row_seq, row_end = np.full(T, -1), np.full(T, -1), np.zeros(T, dtype=np.int64)
    seq_row, seq_len = [0], []
    asked = taken = pushed = 0
    before = s["ring"]
    for i in range(s["n"]):
        ln, new = int(s["ln"][i]), int(s["new"][i])
        held = -(-ln // P)
        if new < 0:
            for j in range(int(s["keep"][i]), held):
                ring[(s["head"] + s["count"] + pushed) % NP] = s["table"][i, j]
                pushed += 1
            seq_row.append(seq_row[-1])
            seq_len.append(0)
            continue
        t0 = seq_row[-1]
        seq_row.append(t0 + new)
        fits = ln + new <= W * P
        want = -(-(ln + new) // P) - held if fits else 0
        first = asked
        asked += want
        ok = fits and (want == 0 or asked <= s["count"]) and t0 + new <= T
        for t in range(t0, min(t0 + new, T)):
            row_seq[t] = i
        if not ok:
            seq_len.append(ln)
            continue
        for j in range(want):
            table[i, held + j] = before[(s["head"] + first + j) % NP]
            taken = asked
        for t in range(t0, t0 + new):
            p = ln + t - t0
            slot[t] = table[i, p // P] * P + p % P
            row_end[t] = p + 1
        seq_len.append(ln + new)
    state = np.array([(s["head"] + taken) % NP, s["count"] - taken + pushed])
    return [torch.from_numpy(np.asarray(a, dtype=np.int32))
            for a in (table, slot, row_seq, row_end, np.array(seq_row), np.array(seq_len), ring, state)]


def _exact_append(s):
    c = s["case"]
    P, out, outs = c["page"], [], []
    for new, cache, scales in ((s["k_new"], s["k"], s["ks"]), (s["v_new"], s["v"], s["vs"])):
        x = new[:s["rows"]].double()
        page, off = torch.div(s["d_slot64"], P, rounding_mode="floor"), s["d_slot64"] % P
        val = cache.double()
        if scales is None:
            val[page, off] = x.to(cache.dtype).double()
            out.append(val)
            continue
        val = val * scales.double().view(*val.shape[:3], 1)
        top = 448.0 if c["cache"] == "e4m3" else 127.0
        scale = (x.abs().amax(-1) / top).float().double()     # the scale as it is stored
        y = x / scale[..., None]
        if c["cache"] == "e4m3":     # the nearest of the format's 127 magnitudes, ties to the even code
            codes = [m / 512.0 for m in range(8)] + [(8 + m) / 512.0 * 2 ** e for e in range(15) for m in range(8)][:119]
            codes = torch.tensor(codes, dtype=torch.float64, device=y.device)
            mids = (codes[1:] + codes[:-1]) / 2
            lo = torch.searchsorted(mids, y.abs().contiguous())
            hi = torch.searchsorted(mids, y.abs().contiguous(), right=True)
            y = torch.sign(y) * codes[torch.where(lo % 2 == 0, lo, hi)]
        else:
            y = torch.round(y)
        val[page, off] = y * scale[..., None]
        out.append(val)
        sc = scales.double()
        sc[s["d_slot64"]] = scale
        outs.append(sc)
    return out + outs


def _exact_rows(s):
    """Row by row for single rows, head by head for a prompt's: the definition over the cells of the row's table."""
    c = s["case"]
    P, hkv, G = c["page"], c["hkv"], c["hq"] // c["hkv"]
    res = torch.zeros(s["out"].shape, dtype=torch.float64, device="cuda")
    pos = torch.arange(int(s["end"].max()), device="cuda", dtype=torch.float64)
    one_table = c["op"] == "prompt"
    block = 256 if one_table else 1
    for r0 in range(0, s["R"], block):
        r1 = min(s["R"], r0 + block)
        n = int(s["end"][r0:r1].max())
        if n == 0:
            continue
        ids = torch.arange(n, device="cuda")
        pg = s["d_table"][int(s["row_table"][r0])].long()[ids // P]
        k, v = s["k"][pg, ids % P].double(), s["v"][pg, ids % P].double()             # [n, hkv, D]
        if s["ks"] is not None:
            k = k * s["ks"][pg * P + ids % P].double()[..., None]
            v = v * s["vs"][pg * P + ids % P].double()[..., None]
        e, b = s["d_end"][r0:r1].double()[:, None], s["d_begin"][r0:r1].double()[:, None]
        hidden = (pos[:n] >= e) | (pos[:n] < b)                                       # [rows, n]
        for h in range(c["hq"]):
            x = (s["q"][r0:r1, h].double() @ k[:, h // G].T) * s["scale"]
            if c["softcap"] > 0:
                x = c["softcap"] * torch.tanh(x / c["softcap"])
            if s["slopes"] is not None:
                x = x - float(s["slopes"][h]) * (e - 1 - pos[:n]).abs()
            x = x.masked_fill(hidden, -math.inf)
            if s["sinks"] is not None:
                x = torch.cat([x, s["sinks"][h].double().expand(r1 - r0, 1)], 1)
            w = torch.softmax(x, 1)[:, :n].nan_to_num(0.0)
            res[r0:r1, h] = w @ v[:, h // G]
    return res
