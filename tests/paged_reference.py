"""Plain implementations of the paged-cache operations, for their tests: page
bookkeeping one page at a time, attention row by row in 64 bits."""
from __future__ import annotations

import math

import numpy as np
import torch


def page_tables(seq_len, new_len, table, ring, state, P, n_rows, n_keep=None):
    """The outputs of attn_page_tables, and the updated table and ring, as int64 arrays."""
    table, ring, before = table.copy(), ring.copy(), ring.copy()
    n, width = table.shape
    n_pages = len(ring)
    head, count = int(state[0]), int(state[1])
    slot, row_seq, row_end = np.full(n_rows, -1), np.full(n_rows, -1), np.zeros(n_rows, dtype=np.int64)
    seq_row, seq_len_out, asked, taken, pushed = [0], [], 0, 0, 0
    for i in range(n):
        ln, new = int(seq_len[i]), int(new_len[i])
        held = -(-ln // P)
        t0 = seq_row[-1]
        if new < 0:
            for j in range(int(n_keep[i]) if n_keep is not None else 0, held):
                ring[(head + count + pushed) % n_pages] = table[i, j]
                pushed += 1
            seq_row.append(t0)
            seq_len_out.append(0)
            continue
        seq_row.append(t0 + new)
        row_seq[t0:min(t0 + new, n_rows)] = i
        fits = ln + new <= width * P
        need = -(-(ln + new) // P) - held if fits else 0
        first = asked
        asked += need
        if not fits or (need > 0 and asked > count) or t0 + new > n_rows:
            seq_len_out.append(ln)
            continue
        for j in range(need):
            table[i, held + j] = before[(head + first + j) % n_pages]
            taken = asked
        for t in range(t0, t0 + new):
            pos = ln + t - t0
            slot[t] = table[i, pos // P] * P + pos % P
            row_end[t] = pos + 1
        seq_len_out.append(ln + new)
    state_out = [(head + taken) % n_pages if n_pages else 0, count - taken + pushed]
    return [np.asarray(x, dtype=np.int64)
            for x in (slot, row_seq, row_end, seq_row, seq_len_out, state_out, table, ring)]


def attention(q, k, v, table, row_end, *, scale, softcap=0.0, row_begin=None, row_table=None, slopes=None,
              sinks=None, k_scale=None, v_scale=None):
    """softmax(transformed logits) V of each row over its visible cells, in 64
    bits, as a numpy array [rows, heads, dim] (CPU tensors in)."""
    n_pages, P, Hkv, D = k.shape
    R, Hq, _ = q.shape
    G = Hq // Hkv
    kf = k.to(torch.float64).reshape(n_pages * P, Hkv, D)
    vf = v.to(torch.float64).reshape(n_pages * P, Hkv, D)
    if k_scale is not None:
        kf = kf * k_scale.to(torch.float64)[:, :, None]
        vf = vf * v_scale.to(torch.float64)[:, :, None]
    out = torch.zeros(R, Hq, D, dtype=torch.float64)
    for r in range(R):
        end = int(row_end[r])
        lo = max(0, int(row_begin[r]) if row_begin is not None else 0)
        hi = min(end, table.shape[1] * P)
        c = torch.arange(lo, max(hi, lo))
        t = int(row_table[r]) if row_table is not None else r
        slot = table[t].long()[c // P] * P + c % P
        for h in range(Hq):
            x = kf[slot, h // G] @ q[r, h].to(torch.float64) * scale
            if softcap > 0:
                x = softcap * torch.tanh(x / softcap)
            if slopes is not None:
                x = x - float(slopes[h]) * (end - 1 - c).abs().to(torch.float64)
            s = torch.tensor([float(sinks[h])] if sinks is not None else [], dtype=torch.float64)
            y = torch.cat([x, s])
            m = y.max() if len(y) else torch.tensor(-math.inf)
            if torch.isnan(y).any() or m == math.inf:
                out[r, h] = math.nan
                continue
            if m == -math.inf:
                continue
            p = torch.exp(x - m)
            out[r, h] = (p / (p.sum() + torch.exp(s - m).sum())) @ vf[slot, h // G]
    return out.numpy()
