"""Plain, slow fp64 numpy form of the decode layer between its projections: the append to a paged
cache with its rotation, the attention of one token over that cache, and the residual step with its
norms. Written from the formulas; shares no code with the library.

Pools are dicts or arrays indexed [page, row, head, entry] of fp64 values (what the cache's elements
stand for).
"""
from __future__ import annotations

import numpy as np


def rotate(x, pos, inv_freq, interleaved):
    """x [tokens, heads, D] with its pairs turned by pos * f; entries past the pairs stay."""
    x = np.array(x, np.float64)
    for t in range(x.shape[0]):
        for i, f in enumerate(inv_freq):
            a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + len(inv_freq))
            ang = np.float64(pos[t]) * np.float64(f)
            c, s = np.cos(ang), np.sin(ang)
            xa, xb = x[t, :, a].copy(), x[t, :, b].copy()
            x[t, :, a] = xa * c - xb * s
            x[t, :, b] = xb * c + xa * s
    return x


def place(table, n_pages, page_size, seq, pos):
    """(page, row) of a token, or None for padding or anything out of range."""
    if pos < 0 or seq < 0 or seq >= len(table) or pos >= table.shape[1] * page_size:
        return None
    page = int(table[seq, pos // page_size])
    return (page, pos % page_size) if 0 <= page < n_pages else None


def attention(q, keys, values, table, lens, scale, window=0, softcap=0.0):
    """out [n, H, D], lse [n, H] and, for tolerances, the largest sum of |scale q_i k_i| over the
    positions seen [n, H] and sum_j p_j |v_j| [n, H, D]. Pages outside the pool are not seen; a
    length outside [0, pages * page_size] is 0."""
    n_pages, page_size, K, D = keys.shape
    n, H, _ = q.shape
    out = np.zeros((n, H, D))
    lse = np.full((n, H), -np.inf)
    size, spread = np.zeros((n, H)), np.zeros((n, H, D))
    for i in range(n):
        L = int(lens[i])
        if L < 0 or L > table.shape[1] * page_size:
            L = 0
        seen = []
        for j in range(max(0, L - window) if window > 0 else 0, L):
            at = place(table, n_pages, page_size, i, j)
            if at is not None:
                seen.append(at)
        if not seen:
            continue
        pg, rw = np.array(seen).T
        for h in range(H):
            kk, vv = keys[pg, rw, h // (H // K)], values[pg, rw, h // (H // K)]
            s = (kk @ q[i, h]) * scale
            size[i, h] = np.max(np.abs(kk) @ np.abs(q[i, h])) * abs(scale)
            if softcap > 0:
                s = softcap * np.tanh(s / softcap)
            m = np.max(s)
            p = np.exp(s - m)
            out[i, h] = (p @ vv) / p.sum()
            spread[i, h] = (p @ np.abs(vv)) / p.sum()
            lse[i, h] = m + np.log(p.sum())
    return out, lse, size, spread


def norm(z, weight, bias, eps, layer):
    z = np.asarray(z, np.float64)
    if layer:
        z = z - z.mean(-1, keepdims=True)
    z = z / np.sqrt((z * z).mean(-1, keepdims=True) + eps)
    z = z if weight is None else z * np.asarray(weight, np.float64)
    return z if bias is None else z + np.asarray(bias, np.float64)


def residual_norm(h, y, post=None, pre=None, gate=None, res_scale=1.0, out_scale=1.0):
    """(r, x); post and pre are functions of a row matrix or None."""
    r = np.float64(res_scale) * np.asarray(h, np.float64)
    if y is not None:
        z = np.asarray(y, np.float64)
        z = z if post is None else post(z)
        z = z if gate is None else z * np.asarray(gate, np.float64)
        r = r + np.float64(out_scale) * z
    return r, (r if pre is None else pre(r))
