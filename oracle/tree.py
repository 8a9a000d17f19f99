"""Tree-drafted decoding in fp64 numpy -- TEST INFRASTRUCTURE ONLY.

The operators' definitions, one row, node or token at a time: norm and rotation, attention of a drafted tree over a
paged cache, verification of drafted tokens, and the commit of a kept path.  Pinned by ``tests/test_oracle_tree.py``.
"""
from __future__ import annotations

import numpy as np


def norm_rotate(x, weight, eps, angle, interleaved):
    """Head rows x [n][H][D] normed (weight [D] or None) and rotated by angle [n][pairs] (float64)."""
    y = np.asarray(x, np.float64)
    if weight is not None:
        y = y / np.sqrt((y * y).mean(-1, keepdims=True) + eps) * np.asarray(weight, np.float64)
    pairs = angle.shape[1]
    out = y.copy()
    for i in range(pairs):
        a, b = (2 * i, 2 * i + 1) if interleaved else (i, i + pairs)
        c, s = np.cos(angle[:, i])[:, None], np.sin(angle[:, i])[:, None]
        out[..., a] = y[..., a] * c - y[..., b] * s
        out[..., b] = y[..., b] * c + y[..., a] * s
    return out


def tree_masks(parents, lens=None):
    """Masks (uint64) and depths of trees given by parents [B][T]."""
    B, T = np.shape(parents)
    masks, depths = np.zeros((B, T), np.uint64), np.zeros((B, T), np.int32)
    for b in range(B):
        for t in range(T if lens is None else int(lens[b])):
            node, bits, depth = t, 1 << t, 0
            while node > 0:
                node = int(parents[b][node])
                bits |= 1 << node
                depth += 1
            masks[b, t], depths[b, t] = bits, depth
    return masks, depths


def rows_of(cache, table_row, count):
    """Rows 0 .. count - 1 of a sequence, [count][Hkv][D], from a paged layer [NB][Hkv][bs][D]."""
    bs = cache.shape[2]
    pos = np.arange(count)
    return cache[np.asarray(table_row)[pos // bs], :, pos % bs] if count else np.zeros((0,) + cache.shape[1::2])


def tree_attention(q, k_cache, v_cache, table, ctx, masks, lens, scale):
    """out [B][T][Hq][D] and, for tolerances, sum_i w_i |v_i| of the same shape; rows behind a tree are NaN."""
    B, T, Hq, D = q.shape
    G = Hq // k_cache.shape[1]
    out, spread = (np.full(q.shape, np.nan, np.float64) for _ in range(2))
    for b in range(B):
        n = int(ctx[b])
        K, V = (rows_of(c, table[b], n) for c in (k_cache, v_cache))
        hist = n - int(lens[b])
        for t in range(int(lens[b])):
            seen = [p for p in range(n) if p < hist or (int(masks[b, t]) >> (p - hist)) & 1]
            for h in range(Hq):
                if not seen:
                    out[b, t, h] = spread[b, t, h] = 0.0
                    continue
                k, v = K[seen, h // G].astype(np.float64), V[seen, h // G].astype(np.float64)
                x = k @ q[b, t, h].astype(np.float64) * scale
                w = np.exp(x - x.max())
                w /= w.sum()
                out[b, t, h], spread[b, t, h] = w @ v, w @ np.abs(v)
    return out, spread


def residual(p, q):
    """max(0, p - q) divided by its sum; None where nothing is left."""
    r = np.maximum(p - q, 0.0)
    return r / r.sum() if r.sum() > 0 else None


def verify(p, q, tokens, parents, u, distinct):
    """One sequence (p, q [T][V]): the kept nodes and the next token, by the definition: the target's and the draft's
    rows of the node are replaced after every refusal."""
    T, V = p.shape
    path, node = [0], 0
    while True:
        pk, qk, kept = p[node].astype(np.float64), q[node].astype(np.float64), None
        for c in range(node + 1, T):
            if parents[c] != node or pk is None or qk is None:
                continue
            x = tokens[c]
            if u[c] * qk[x] < pk[x]:
                kept = c
                break
            pk = residual(pk, qk)
            if distinct:
                rest = 1.0 - qk[x]
                qk = qk / rest if rest > 0 else None
                if qk is not None:
                    qk[x] = 0.0
        if kept is None:
            w = p[node].astype(np.float64) if pk is None else pk
            sums = np.cumsum(w)
            return path, int(np.searchsorted(sums, u[0] * sums[-1], side="right"))
        path.append(kept)
        node = kept


def commit(pools, table, ctx, lens, path, path_len):
    """pools: arrays [L][NB][Hkv][bs][D], changed in place; returns the new context lengths."""
    new = np.array(ctx, np.int32)
    for b in range(len(ctx)):
        base = int(ctx[b]) - int(lens[b])
        for pool in pools:
            bs = pool.shape[3]
            old = [pool[:, table[b][(base + n) // bs], :, (base + n) % bs].copy() for n in range(int(lens[b]))]
            for i in range(int(path_len[b])):
                pool[:, table[b][(base + i) // bs], :, (base + i) % bs] = old[int(path[b][i])]
        new[b] = base + int(path_len[b])
    return new
