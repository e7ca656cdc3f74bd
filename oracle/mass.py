"""Attention weights of query rows over a paged pool, in fp64, added up by token.

Rows are packed as in oracle.extend: row j of the n rows of sequence a is its
token seq_len[a] - n + j; decode steps have one row each and see everything."""
from __future__ import annotations

import numpy as np


def attend(q, k_pool, v_pool, block_table, tok_off, seq_len, block_tokens: int, scale: float, causal: bool):
    """(out [T][Hq][d], sum_p p |V| of it, weights by token: a list of [seq_len[a]]
    arrays, the largest sum of |q_i k_i| * scale); v_pool None: no out.  Blocks
    whose id lies outside the pool take their tokens out."""
    q = np.asarray(q, np.float64)
    T, hq, d = q.shape
    cap, hkv = k_pool.shape[:2]
    g = hq // hkv
    out, mag, big, mass = np.zeros((T, hq, d)), np.zeros((T, hq, d)), 0.0, []
    for a in range(len(seq_len)):
        t0, t1, n = int(tok_off[a]), int(tok_off[a + 1]), int(seq_len[a])
        ids = np.asarray(block_table[a][: -(-n // block_tokens)])
        there = np.repeat((ids >= 0) & (ids < cap), block_tokens)[:n]
        ids = np.where((ids >= 0) & (ids < cap), ids, 0)
        m = np.zeros(n)
        lim = np.arange(t1 - t0) + n - (t1 - t0) + 1 if causal else np.full(t1 - t0, n)
        seen = (np.arange(n) < lim[:, None]) & there
        for h in range(hkv if n else 0):
            K = k_pool[ids, h].reshape(-1, d)[:n].astype(np.float64)
            K = np.where(there[:, None], K, 0.0)
            for e in range(h * g, h * g + g):
                S = q[t0:t1, e] @ K.T * scale
                big = max(big, float(np.where(seen, np.abs(q[t0:t1, e]) @ np.abs(K).T * scale, 0.0).max(initial=0.0)))
                S = np.where(seen, S, -np.inf)
                top = S.max(-1, keepdims=True)
                P = np.exp(S - np.where(np.isfinite(top), top, 0.0))
                P /= np.maximum(P.sum(-1, keepdims=True), 1e-300)
                m += P.sum(0)
                if v_pool is not None:
                    V = v_pool[ids, h].reshape(-1, d)[:n].astype(np.float64)
                    V = np.where(there[:, None], V, 0.0)
                    out[t0:t1, e], mag[t0:t1, e] = P @ V, P @ np.abs(V)
        mass.append(m)
    return out, mag, mass, big
