"""The paged serving step (oracle side): block tables and slot maps from
request lengths, the append of a ragged batch's new tokens, and attention of
drafted token trees ([P1] hybrid KV cache manager paragraph: blocks of a
shared pool; "compressor-state blocks").

Test infrastructure: only the tests use this module.

Readings adopted (the pages give none of these):
* pages are taken from and given back to a stack of free page numbers, one
  sequence after the other; everything given back is pushed before anything
  is taken; an entry that got no page (-1) gives none back;
* a drafted node at position p attends as the token at p would with its
  ancestors appended to the caches: entries [0, N(p)), window positions
  [p - W, t), its strict ancestors;
* with a lookahead L an entry is written L positions before its block leaves
  the window.
"""
from __future__ import annotations

import numpy as np

from .attention import shared_kv_decode
from .compress import n_entries, tap_positions
from .rope import rope


def cache_rows(t: int, window: int, stride: int, lookahead: int = 0) -> int:
    """Rows of a cache of a sequence of t tokens (stride 0: its window cache)."""
    return min(t, window) if stride == 0 else n_entries(t + lookahead, window, stride)


def block_table_update(t_old, t_new, table, free, page_rows: int, window: int, stride: int, lookahead: int = 0):
    """table: list of lists of page numbers, free: list (a stack).  Returns the new (table, free)."""
    table, free = [list(r) for r in table], list(free)
    pages = [[-(-cache_rows(t, window, stride, lookahead) // page_rows) for t in ts] for ts in (t_old, t_new)]
    for b, (o, n) in enumerate(zip(*pages)):
        for j in range(n, o):
            if table[b][j] >= 0:
                free.append(table[b][j])
    for b, (o, n) in enumerate(zip(*pages)):
        for j in range(o, n):
            table[b][j] = free.pop() if free else -1
    return table, free


def slot_map(t_old, t_new, comp_table, win_table, page_rows: int, win_page_rows: int, window: int, stride: int,
             lookahead: int = 0):
    """(cu, seq, pos, win_slot, comp_slot) as lists, one token after the other."""
    cu, seq, pos, win, comp = [0], [], [], [], []

    def slot(row, pages, page):
        pg = pages[row // page]
        return -1 if pg < 0 else pg * page + row % page

    for b, (o, n) in enumerate(zip(t_old, t_new)):
        for p in range(o, n):
            seq.append(b)
            pos.append(p)
            win.append(slot(p % window, win_table[b], win_page_rows) if window and p + window >= n else -1)
            e = n_entries(p + lookahead, window, stride)
            due = n_entries(p + 1 + lookahead, window, stride) > e
            comp.append(slot(e, comp_table[b], page_rows) if due else -1)
        cu.append(len(seq))
    return cu, seq, pos, win, comp


def append_rows(hist, t_old: int, t_new: int, w, window: int, stride: int, lookahead: int = 0, rope_dim: int = 64,
                base: float = 10000.0):
    """What appending positions t_old .. t_new - 1 of one sequence writes, from its whole history hist [t_new][D]
    (float64, unrotated): ({window row: values}, {entry: values}, {raw ring row: values})."""
    w = np.asarray(w, dtype=np.float64)
    ring = window + w.shape[0]
    win = {p % window: rope(hist[p], p, rope_dim, base) for p in range(max(t_old, t_new - window), t_new)} if window else {}
    ents = {}
    for e in range(n_entries(t_old + lookahead, window, stride), n_entries(t_new + lookahead, window, stride)):
        taps = tap_positions(e, stride, w.shape[0])
        acc = np.zeros(hist.shape[1])
        for j, p in enumerate(taps):
            if p >= 0:
                acc += w[j] * hist[p]
        ents[e] = rope(acc, stride * e, rope_dim, base)
    raw = {p % ring: hist[p] for p in range(max(t_old, t_new - ring), t_new)}
    return win, ents, raw


def ancestors(parent) -> list[list[int]]:
    """The strict ancestors of every node of one sequence's drafted tree(s)."""
    out: list[list[int]] = []
    for j, p in enumerate(parent):
        assert -1 <= p < j
        out.append([] if p < 0 else out[p] + [int(p)])
    return out


def window_positions(t: int, window: int) -> np.ndarray:
    """Position held by every window row r < min(t, window): the last one congruent to r."""
    r = np.arange(min(t, window))
    return r + (t - 1 - r) // window * window if len(r) else r


def tree_decode(q, comp, win, draft, parent, t: int, window: int, stride: int, idx=None, scale: float = 512 ** -0.5,
                rope_dim: int = 64, base: float = 10000.0) -> np.ndarray:
    """One sequence: q [m][H][D], comp [>= entries][D], win [min(t, W)][D] (row r: window_positions), draft [m][D],
    idx: per node a list of entries, None: all.  Returns [m][H][D]; zeros for a node that sees no row."""
    held = window_positions(t, window)
    out = []
    for j, path in enumerate(ancestors(parent)):
        p = t + len(path)
        n = n_entries(p, window, stride)
        rows = [comp[:n] if idx is None else comp[[e for e in idx[j][:min(n, len(idx[j]))] if 0 <= e < n]],
                win[held >= p - window], draft[path]]
        rows = np.concatenate([np.asarray(x, dtype=np.float64).reshape(-1, q.shape[-1]) for x in rows])
        out.append(shared_kv_decode(q[j], rows, scale, p, rope_dim, base) if len(rows) else np.zeros(q[j].shape))
    return np.stack(out)
