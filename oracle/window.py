"""Windows, the block-scaled 8-bit cache and block tables in fp64 numpy -- TEST INFRASTRUCTURE ONLY.

The operators' definitions, one sequence, row or position at a time.  Pinned by ``tests/test_oracle_window.py``.
"""
from __future__ import annotations

import numpy as np

BS = 16
LEAST = -32  # exponent of the scale of a block of zeros
# what e4m3 holds: code (without its sign bit) -> value; 0x7f is NaN
E4M3 = np.array([np.ldexp(c & 7, -9) if c < 8 else np.ldexp(8 + (c & 7), (c >> 3) - 10) for c in range(127)])


def visible(n, window, sinks):
    """Positions that the query at position n - 1 sees (window 0: all)."""
    p = np.arange(n)
    return p if window == 0 else p[(p >= n - window) | (p < sinks)]


def attend(q, k, v, scale):
    """softmax(q k^T scale) v for one query row; a row without weights gives 0."""
    s = np.asarray(k, np.float64) @ np.asarray(q, np.float64) * scale
    if len(s) == 0 or np.all(s == -np.inf):
        return np.zeros(np.shape(v)[1])
    w = np.exp(s - s.max())
    return w @ np.asarray(v, np.float64) / w.sum()


def decode(q, rows, scale, window, sinks):
    """q [B][Hq][D]; rows(b, positions) -> k, v [n][Hkv][D] and the context's length through rows.ctx[b]."""
    q = np.asarray(q, np.float64)
    out = np.zeros(q.shape)
    for b in range(q.shape[0]):
        k, v = rows(b, visible(int(rows.ctx[b]), window, sinks))
        per = q.shape[1] // k.shape[1]
        for h in range(q.shape[1]):
            out[b, h] = attend(q[b, h], k[:, h // per], v[:, h // per], scale)
    return out


def prefill(q, k, v, lens, scale, window, sinks):
    """Packed segments, causal, every row over its visible ones."""
    q, k, v = (np.asarray(x, np.float64) for x in (q, k, v))
    out, at, per = np.zeros(q.shape), 0, q.shape[1] // k.shape[1]
    for n in lens:
        for h in range(q.shape[1]):
            kk, vv = k[at:at + n, h // per], v[at:at + n, h // per]
            for i in range(n):
                p = visible(i + 1, window, sinks)
                out[at + i, h] = attend(q[at + i, h], kk[p], vv[p], scale)
        at += n
    return out


def nearest_e4m3(x):
    """Codes (uint8) of the e4m3 values nearest to x (ties to the even code, beyond 448 to 448, NaN to 0x7f)."""
    x = np.asarray(x, np.float64)
    a = np.minimum(np.abs(x), E4M3[-1])
    up = np.clip(np.searchsorted(E4M3, a), 0, 126)
    down = np.maximum(up - 1, 0)
    take_up = (E4M3[up] - a < a - E4M3[down]) | ((E4M3[up] - a == a - E4M3[down]) & (up % 2 == 0))
    code = np.where(take_up, up, down) | np.where(np.signbit(x), 0x80, 0)
    return np.where(np.isnan(x), 0x7f | np.where(np.signbit(x), 0x80, 0), code).astype(np.uint8)


def e4m3_values(codes):
    c = np.asarray(codes, np.uint8)
    return np.where(c & 0x7f == 0x7f, np.nan, np.append(E4M3, np.nan)[c & 0x7f] * np.where(c & 0x80, -1.0, 1.0))


def exponent(x):
    """Least e for which no finite value of x exceeds 448 * 2^e."""
    a = np.abs(np.asarray(x, np.float64))
    top = a[np.isfinite(a)].max(initial=0.0)
    if top == 0:
        return LEAST
    e = LEAST
    while top > 448 * 2.0 ** e:
        e += 1
    return e


def append(k, v, slots, codes, scales):
    """Rows [n][Hkv][D] into codes [NB][Hkv][2][BS][D] (uint8) and scales [NB][Hkv][2], in place, run by run."""
    t = 0
    while t < len(slots):
        s = int(slots[t])
        if s < 0:
            t += 1
            continue
        n = 1
        while t + n < len(slots) and slots[t + n] == s + n and (s + n) // BS == s // BS:
            n += 1
        blk, first = s // BS, s % BS
        for h in range(codes.shape[1]):
            for c, rows in enumerate((k, v)):
                x = np.asarray(rows[t:t + n, h], np.float64)
                new = 2.0 ** exponent(x)
                old = float(scales[blk, h, c])
                tile = codes[blk, h, c]
                if first > 0 and old >= new:
                    new = old
                elif first > 0:
                    tile[:first] = nearest_e4m3(e4m3_values(tile[:first]) * (old / new))
                tile[first:first + n] = nearest_e4m3(x / new)
                scales[blk, h, c] = new
        t += n


def ring(window):
    """Blocks that a window's positions are ever in at once."""
    return max(len({p // BS for p in range(last - window + 1, last + 1)}) for last in range(window - 1, window + BS))


def block_tables(before, after, free, placed, table, window, sinks, num_slots):
    """New table, placed, cu_tokens, slots and positions; the step one block and one token at a time."""
    table = np.array(table)
    B, turn, first = len(after), ring(window) if window else 0, -(-sinks // BS)
    slots, positions = np.full(num_slots, -1, np.int64), np.zeros(num_slots, np.int32)
    cu, t, at, original = [0], 0, int(placed), table.copy()
    nothing = original, int(placed), np.zeros(B + 1, np.int32), np.full(num_slots, -1, np.int64), np.zeros(num_slots, np.int32)
    if not 0 <= at <= len(free):
        return nothing
    for b in range(B):
        lo, hi = (0 if before is None else int(before[b])), int(after[b])
        if lo < 0 or hi < lo or hi > table.shape[1] * BS:
            cu.append(t)
            continue
        blocks = -(-hi // BS)
        for j in range(-(-lo // BS), blocks):
            if window and j >= first + turn:
                table[b, j] = table[b, j - turn]
            else:
                if at == len(free):
                    return nothing
                table[b, j] = free[at]
                at += 1
        for p in range(lo, hi):
            if t == num_slots:
                return nothing
            positions[t] = p
            if not window or p // BS < first or p // BS >= blocks - turn:
                slots[t] = int(table[b, p // BS]) * BS + p % BS
            t += 1
        cu.append(t)
    return table, at, np.array(cu, np.int32), slots, positions
