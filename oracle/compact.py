"""Eviction by accumulated attention weight, on the host: which tokens a
sequence keeps, and the pool, tables, counts and free stack behind it.  Written
from the rules of the interface alone; nothing here is shared with the CUDA
path."""
from __future__ import annotations

import numpy as np


def keep_heavy(mass, seq_len, budget, n_first: int, n_recent: int):
    """(kept indices of all sequences one after the other, int64 offsets)."""
    out, off = [], [0]
    for a, n in enumerate(int(x) for x in seq_len):
        must = np.zeros(n, bool)
        must[:n_first] = True
        if n_recent:
            must[max(0, n - n_recent):] = True
        m = np.asarray(mass[a][:n], np.float64) + 0.0
        m = np.where(np.isnan(m), -np.inf, m)
        # NaN is below every number, -inf among them
        order = sorted(np.nonzero(~must)[0], key=lambda t: (-m[t], np.isnan(mass[a][t]), t))
        more = max(0, min(int(budget[a]), n) - int(must.sum()))
        idx = np.sort(np.concatenate([np.nonzero(must)[0], np.asarray(order[:more], np.int64)])).astype(np.int64)
        out.append(idx)
        off.append(off[-1] + len(idx))
    return np.concatenate(out) if out else np.zeros(0, np.int64), np.asarray(off, np.int64)


def compact(slabs, table, seq_len, idx, idx_off, mass, refcount, free, block: int):
    """The state after a compaction: (slabs, table, seq_len, mass, refcount,
    free, sequences that were left alone).  slabs: arrays [capacity][heads]
    [block][row]; free: the stack as a list, its top last."""
    slabs = [np.array(s) for s in slabs]
    before = [s.copy() for s in slabs]
    table, seq_len, refcount, free = np.array(table), np.array(seq_len), np.array(refcount), list(free)
    mass = None if mass is None else np.array(mass)
    start, cap, gone, left_alone = refcount.copy(), len(refcount), [], []
    for a in range(len(seq_len)):
        n, keep = int(seq_len[a]), np.asarray(idx[idx_off[a]:idx_off[a + 1]], np.int64)
        nb_old, nb_new = -(-n // block), -(-len(keep) // block)
        was = table[a].copy()
        bad = (np.diff(keep) <= 0).any() or (len(keep) > 0 and (keep[0] < 0 or keep[-1] >= n))
        bad = bad or ((was[:nb_old] < 0) | (was[:nb_old] >= cap)).any()
        moved = np.nonzero(keep != np.arange(len(keep)))[0]
        first = moved[0] // block if len(moved) and not bad else nb_new
        fresh = [] if bad else [b for b in range(first, nb_new) if start[was[b]] > 1]
        if bad or len(fresh) > len(free):
            left_alone.append(a)
            continue
        for b in fresh:
            table[a, b] = free.pop()
            refcount[table[a, b]] = 1
            gone.append(was[b])
        gone += list(was[nb_new:nb_old])
        table[a, nb_new:nb_old] = -1
        for i, t in enumerate(keep):
            if i // block < first:
                continue
            for s, x in zip(slabs, before):
                s[table[a, i // block], :, i % block] = x[was[t // block], :, t % block]
        if mass is not None:
            mass[a, :len(keep)] = mass[a, keep]
            mass[a, len(keep):n] = 0
        seq_len[a] = len(keep)
    for id_ in gone:
        refcount[id_] -= 1
    free += sorted({int(x) for x in gone if refcount[x] == 0}, reverse=True)
    return slabs, table, seq_len, mass, refcount, free, left_alone
