"""New tokens in a shared paged KV pool, in fp64: rotary positions on one to
three axes, the rotated append, the read-back, and attention of query chunks.

Packed rows of sequence a are tok_off[a] .. tok_off[a + 1); row j of its n
rows is token seq_len[a] - n + j.  Rotation pairs dimension i with i + d/2 (as
oracle.rope); the first section[0] pairs turn with axis 0, and so on.  Nothing
here is shared with the CUDA path."""
from __future__ import annotations

import numpy as np


def axes_frequencies(head_dim: int, theta: float, sections, own_spectrum: bool = False):
    """(angular frequency, axis) of every pair."""
    w, axis = [], []
    for a, s in enumerate(sections):
        for j in range(s):
            i = len(w)
            e = -j / s if own_spectrum else -2.0 * i / head_dim
            w.append(float(np.float32(theta)) ** e)
            axis.append(a)
    assert len(w) == head_dim // 2
    return np.array(w), np.array(axis)


def rotate_axes(x, pos, theta: float, sections, own_spectrum=False, inverse=False):
    """x [T][H][d], pos int [axes][T]."""
    x = np.asarray(x, np.float64)
    d = x.shape[-1]
    w, axis = axes_frequencies(d, theta, sections, own_spectrum)
    # positions times frequencies in extended precision: far positions turn many times
    ang = np.asarray(pos, np.longdouble)[axis].T * w.astype(np.longdouble)
    ang = np.fmod(ang, 2 * np.arctan(np.longdouble(1)) * 4).astype(np.float64)[:, None, :]
    c, s = np.cos(ang), np.sin(ang) * (-1.0 if inverse else 1.0)
    lo, hi = x[..., : d // 2], x[..., d // 2:]
    return np.concatenate([lo * c - hi * s, hi * c + lo * s], -1)


def places(tok_off, seq_len, block_table, block_tokens: int):
    """For every packed row: (sequence, logical position, physical block, row
    in it); rows of no sequence are left out."""
    out = {}
    for a in range(len(seq_len)):
        n = int(tok_off[a + 1]) - int(tok_off[a])
        for j in range(n):
            p = int(seq_len[a]) - n + j
            out[int(tok_off[a]) + j] = (a, p, int(block_table[a, p // block_tokens]), p % block_tokens)
    return out


def extend_attention(q, k_pool, v_pool, block_table, tok_off, seq_len, block_tokens: int, scale: float, causal: bool):
    """(out [T][Hq][d], mean absolute value weight sum_p p |V|, largest sum of
    |q_i k_i| * scale) in fp64; rows of no sequence are NaN."""
    q = np.asarray(q, np.float64)
    T, hq, d = q.shape
    hkv = k_pool.shape[1]
    g = hq // hkv
    out = np.full((T, hq, d), np.nan)
    mag = np.zeros((T, hq, d))
    big = 0.0
    for a in range(len(seq_len)):
        t0, t1, n = int(tok_off[a]), int(tok_off[a + 1]), int(seq_len[a])
        ids = block_table[a, : -(-n // block_tokens)]
        for h in range(hkv):
            K = k_pool[ids, h].reshape(-1, d)[:n].astype(np.float64)
            V = v_pool[ids, h].reshape(-1, d)[:n].astype(np.float64)
            for t in range(t0, t1):
                lim = n - (t1 - t0) + (t - t0) + 1 if causal else n
                for e in range(g):
                    if lim <= 0:
                        out[t, h * g + e] = 0.0
                        continue
                    s = K[:lim] @ q[t, h * g + e] * scale
                    big = max(big, float((np.abs(K[:lim]) @ np.abs(q[t, h * g + e])).max()) * scale)
                    p = np.exp(s - s.max())
                    p /= p.sum()
                    out[t, h * g + e] = p @ V[:lim]
                    mag[t, h * g + e] = p @ np.abs(V[:lim])
    return out, mag, big
