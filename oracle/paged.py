"""The paged packed K/V cache by its definition, in numpy and 64 bits (test infrastructure, like the
rest of the oracle).

A pool is uint8 [n_pages, H, P, D*bits/8]; position p of sequence b is page table[b][p // P], slot
p % P; rows start[b] .. start[b+1]-1 of a ragged batch are the newest positions of sequence b, whose
length lens[b] counts them.  The quantizer is the dense cache's (oracle.kv_quant / kv_dequant).
"""
from __future__ import annotations

import numpy as np

import oracle


def _at(table, b, pos, P):
    return table[b, pos // P], pos % P


def append(pages, x, start, lens, table, labels, s, z, bits, weights=None):
    """x fp32 [T, H, D] into the pages (a copy is returned); weights' new positions become 0."""
    pages = pages.copy()
    weights = None if weights is None else weights.copy()
    P, D = pages.shape[2], x.shape[2]
    codes = oracle.kv_quant(np.ascontiguousarray(x.transpose(1, 0, 2)[None]), labels, s, z, bits)[0]  # [H, T, rb]
    assert codes.shape[2] == D * bits // 8
    for b in range(len(lens)):
        n = start[b + 1] - start[b]
        for i in range(n):
            pos = lens[b] - n + i
            if pos >= 0:
                pg, sl = _at(table, b, pos, P)
                pages[pg, :, sl] = codes[:, start[b] + i]
                if weights is not None:
                    weights[pg, :, sl] = 0
    return pages if weights is None else (pages, weights)


def gather(pages, table, b, n):
    """Rows [n, H, bytes] of the first n positions of sequence b."""
    pos = np.arange(n)
    pg, sl = _at(table, b, pos, pages.shape[2])
    return pages[pg, :, sl]


def values(pages, table, b, n, D, labels, s, z, bits):
    """fp32 [n, H, D]: the dequantized first n positions of sequence b."""
    r = np.ascontiguousarray(gather(pages, table, b, n).transpose(1, 0, 2)[None])
    if n == 0:
        return np.zeros((0, pages.shape[1], D), np.float32)
    return oracle.kv_dequant(r, D, labels, s, z, bits)[0].transpose(1, 0, 2)


def attention(q, start, lens, table, k_pages, v_pages, k_cal, v_cal, bits, scale=None, weights=None):
    """fp64 out [T, Hq, D] (NaN in rows of no sequence) and, where given, the grown running sums; also
    the probabilities' ingredients for error bounds: per sequence (K, V, x, w)."""
    T, Hq, D = q.shape
    H = k_pages.shape[1]
    G = Hq // H
    scale = 1.0 / np.sqrt(D) if not scale else scale
    out = np.full((T, Hq, D), np.nan)
    weights = None if weights is None else weights.astype(np.float64)
    parts = []
    for b in range(len(lens)):
        n, L = start[b + 1] - start[b], lens[b]
        K = values(k_pages, table, b, L, D, *k_cal, bits).astype(np.float64).repeat(G, axis=1)
        V = values(v_pages, table, b, L, D, *v_cal, bits).astype(np.float64).repeat(G, axis=1)
        qb = q[start[b]:start[b] + n].astype(np.float64)
        x = np.einsum("nad,pad->anp", qb, K) * scale
        vis = np.arange(L)[None, :] <= (L - n + np.arange(n))[:, None]
        x = np.where(vis, x, -np.inf)
        m = np.max(x, axis=2, keepdims=True, initial=-np.inf)
        e = np.where(vis, np.exp(x - np.where(np.isfinite(m), m, 0.0)), 0.0)
        t = e.sum(axis=2, keepdims=True)
        w = e / np.where(t > 0, t, 1.0)
        out[start[b]:start[b] + n] = np.einsum("anp,pad->nad", w, V)
        if weights is not None and n:
            pg, sl = _at(table, b, np.arange(L), k_pages.shape[2])
            weights[pg, :, sl] += w.reshape(H, G * n, L).sum(axis=1).T
        parts.append((K, V, x, w))
    return out, weights, parts


def evict(k_pages, v_pages, weights, lens, table, budget, recent):
    """(k_pages, v_pages, weights, new_lens, kept [B, H, budget]) after eviction."""
    k_pages, v_pages, weights = k_pages.copy(), v_pages.copy(), weights.copy()
    P, H = k_pages.shape[2], k_pages.shape[1]
    kept = np.full((len(lens), H, budget), -1, np.int32)
    new = np.minimum(lens, budget).astype(np.int32)
    for b, L in enumerate(lens):
        if L <= budget:
            kept[b, :, :L] = np.arange(L)
            continue
        pg, sl = _at(table, b, np.arange(L), P)
        for h in range(H):
            w = weights[pg, h, sl][:L - recent].astype(np.float64)
            w = np.where(np.isnan(w), -np.inf, w)
            nan = np.isnan(weights[pg, h, sl][:L - recent])
            order = np.lexsort((np.arange(w.size), nan, -w))  # larger first, NaN last, then the lower position
            keep = np.concatenate((np.sort(order[:budget - recent]), np.arange(L - recent, L)))
            kept[b, h] = keep
            j = np.arange(budget)
            for x in (k_pages, v_pages, weights):
                x[pg[j], h, sl[j]] = x[pg[keep], h, sl[keep]].copy()
    return k_pages, v_pages, weights, new, kept
