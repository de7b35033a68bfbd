"""fp64 CPU oracle for the serving calls: block tables and slot maps, rows into
the 8-bit cache, and HCA attention over it.

TEST INFRASTRUCTURE ONLY.  Imported by ``tests/``; the product library never
imports or calls it and shares no code with it.  Plain numpy in float64, one
loop per request, one visibility predicate per (token, key): a token at position
i sees its request's raw row t iff i - W < t <= i and its compressed entry j iff
(j + 1) m <= i + 1 (the rule of the dense oracle with one document per request).

The cache is given by values: ``pool`` [nblocks, bs, D] holds the e4m3 values as
doubles (NaN included), ``scale`` [nblocks] one scale per block.
"""
from __future__ import annotations

import numpy as np


def e4m3_table() -> np.ndarray:
    """Values of the 256 e4m3 codes (sign, 4 exponent bits of bias 7, 3 mantissa
    bits; S.1111.111 is NaN, there are no infinities)."""
    v = np.empty(256)
    for c in range(256):
        e, f = (c >> 3) & 15, c & 7
        x = f * 2.0 ** -9 if e == 0 else (1 + f / 8) * 2.0 ** (e - 7)
        v[c] = np.nan if (e, f) == (15, 7) else (-x if c & 128 else x)
    return v


_POS = e4m3_table()[:127]  # ascending, 0 .. 448


def e4m3_round(x) -> np.ndarray:
    """Nearest e4m3 value, ties to the even code; |x| up to 448.  Infinities
    and NaN give NaN."""
    x = np.asarray(x, dtype=np.float64)
    a = np.where(np.isfinite(x), np.abs(x), 0.0)
    assert a.size == 0 or a.max() <= 448.0
    hi = np.searchsorted(_POS, a)                 # first value >= a
    lo = np.maximum(hi - 1, 0)
    dl, dh = a - _POS[lo], _POS[hi] - a
    pick = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi)
    r = np.copysign(_POS[pick], x)
    return np.where(np.isfinite(x), r, np.nan)


def block_scale(amax: float) -> float:
    """Smallest power of two s >= 2^-96 with amax <= 448 s."""
    s = 2.0 ** -96
    while amax > 448.0 * s:
        s *= 2.0
    return s


def plan(held, added, table, free_blocks, free_count, bs, nslots, m):
    """(start, slots, free_left, table), or None when it does not fit."""
    held, added, table = (np.array(a, dtype=np.int64) for a in (held, added, table))
    cols = table.shape[1]
    left, start, slots = int(free_count), [0], []
    for r in range(len(held)):
        a, b = int(held[r]) // m, int(held[r] + added[r]) // m
        for e in range(a, b):
            page = e // bs
            if e % bs == 0 and page < cols:  # the first entry of a column that was empty
                left -= 1
                if left < 0:
                    return None
                table[r, page] = free_blocks[left]
            last = (b - 1) // bs
            slots.append(int(table[r, page % cols]) * bs + e % bs if last - page < cols else -1)
        start.append(len(slots))
    if len(slots) > nslots:
        return None
    return start, slots + [-1] * (nslots - len(slots)), left, table


def append(x, slots, pool, scale):
    """(pool, scale) after the rows; runs in order of x."""
    x = np.asarray(x, dtype=np.float64)
    pool, scale = np.array(pool, dtype=np.float64), np.array(scale, dtype=np.float64)
    bs = pool.shape[1]
    t = 0
    while t < len(slots):
        s = int(slots[t])
        if s < 0:
            t += 1
            continue
        n = 1
        while t + n < len(slots) and slots[t + n] == s + n and (s + n) % bs:
            n += 1
        blk, off = divmod(s, bs)
        rows = x[t:t + n]
        fin = rows[np.isfinite(rows)]
        need = block_scale(float(np.abs(fin).max()) if fin.size else 0.0)
        if off == 0:
            new = need
        else:
            new = max(need, float(scale[blk]))
            if new > scale[blk]:
                pool[blk, :off] = e4m3_round(pool[blk, :off] * (scale[blk] / new))
        scale[blk] = new
        pool[blk, off:off + n] = e4m3_round(rows / new)
        t += n
    return pool, scale


def _rows(cache, r, entries):
    pool, scale, table = cache
    bs, cols = pool.shape[1], table.shape[1]
    out = np.empty((len(entries), pool.shape[2]))
    for i, e in enumerate(entries):
        blk = int(table[r, (e // bs) % cols])
        out[i] = pool[blk, e % bs] * scale[blk] if 0 <= blk < pool.shape[0] else np.nan
    return out


def attend(q, start, held, raw, comp, W, m, scale):
    """(out [N,H,D], lse [N,H], mass [N,H,D], spread [N,H]): mass is the
    probability-weighted mean of |key| (what the error of a probability
    multiplies), spread the largest over the visible keys of sum_d |q_d k_d|.
    Rows that belong to no request are NaN."""
    q = np.asarray(q, dtype=np.float64)
    N, H, D = q.shape
    out, mass = np.full((N, H, D), np.nan), np.full((N, H, D), np.nan)
    lse, spread = np.full((N, H), np.nan), np.full((N, H), np.nan)
    for r in range(len(held)):
        for t in range(int(start[r]), int(start[r + 1])):
            i = int(held[r]) + t - int(start[r])
            kv = _rows(raw, r, [p for p in range(max(0, i - W + 1), i + 1)])
            ents = [] if comp is None else [j for j in range((i + 1) // m + 1) if (j + 1) * m <= i + 1]
            if ents:
                kv = np.concatenate([kv, _rows(comp, r, ents)])
            s = scale * (q[t] @ kv.T)
            top = s.max(1, keepdims=True)
            p = np.exp(s - top)
            tot = p.sum(1, keepdims=True)
            out[t] = (p / tot) @ kv
            mass[t] = (p / tot) @ np.abs(kv)
            lse[t] = (top + np.log(tot))[:, 0]
            spread[t] = (np.abs(q[t]) @ np.abs(kv).T).max(1)
    return out, lse, mass, spread


def terms(q, start, held, raw, comp, W, m, scale):
    """For each query token of the requests, in order: (values [n,D] of the n keys
    that it sees, probabilities [H,n], lse [H], spread [H,n]), spread being
    sum_d |q_d k_d|."""
    q = np.asarray(q, dtype=np.float64)
    for r in range(len(held)):
        for t in range(int(start[r]), int(start[r + 1])):
            i = int(held[r]) + t - int(start[r])
            kv = _rows_at_once(raw, r, np.arange(max(0, i - W + 1), i + 1))
            if comp is not None and (i + 1) // m:
                kv = np.concatenate([kv, _rows_at_once(comp, r, np.arange((i + 1) // m))])
            s = scale * (q[t] @ kv.T)
            top = s.max(1, keepdims=True)
            p = np.exp(s - top)
            tot = p.sum(1, keepdims=True)
            yield kv, p / tot, (top + np.log(tot))[:, 0], np.abs(q[t]) @ np.abs(kv).T


def _rows_at_once(cache, r, entries):
    pool, scale, table = cache
    bs, cols = pool.shape[1], table.shape[1]
    blk = table[r, (entries // bs) % cols]
    return pool[blk, entries % bs] * scale[blk][:, None]
