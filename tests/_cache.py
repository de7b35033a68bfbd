"""Inputs and tolerances shared by the serving tests."""
import math

import numpy as np
import torch

from oracle import cache as OC

E4M3 = torch.float8_e4m3fn


def values(pool):
    return pool.float().cpu().double().numpy()


def make_cache(entries, cols, bs, D, seed, spare=2, spread=2, spill=True):
    """A CPU cache holding `entries[r]` random rows for each request: (pool
    e4m3, scale, table).  Blocks are in random order, scales differ by block,
    unused table columns are -1 and rows that belong to nobody are NaN."""
    g = torch.Generator().manual_seed(seed)
    rng = np.random.default_rng(seed)
    used = [min(-(-e // bs), cols) for e in entries]
    nblocks = sum(used) + spare
    perm = rng.permutation(nblocks)
    table = np.full((len(entries), cols), -1, dtype=np.int32)
    at = 0
    for r, n in enumerate(used):
        table[r, :n] = perm[at:at + n]
        at += n
    x = torch.randn(nblocks, bs, D, generator=g)
    scale = torch.exp2(torch.randint(-7 - spread, -6 + spread, (nblocks,), generator=g).float())
    pool = (x / torch.exp2(torch.tensor(-7.0))).clamp(-448, 448).to(E4M3)
    raw = pool.view(torch.uint8)
    if spill:
        live = np.zeros((nblocks, bs), dtype=bool)
        for r, e in enumerate(entries):
            for k in range(max(0, e - cols * bs), e):
                live[table[r, (k // bs) % cols], k % bs] = True
        raw[torch.from_numpy(~live)] = 0x7F
    return pool, scale, torch.from_numpy(table)


def oracle_cache(c):
    return None if c is None else (values(c[0]), c[1].double().numpy(), c[2].numpy())


def ring_cols(W, t, bs):
    return -(-(W - 1 + t) // bs) + 1


def attn_case(held, added, H, D, W, m, bs, dtype, seed, comp=True, ring=True, qscale=1.0, pad=0):
    """CPU inputs of one attention call: (q, start, held, raw, comp)."""
    total = [h + a for h, a in zip(held, added)]
    cols = -(-max(total + [1]) // bs)
    if ring:
        cols = min(cols, ring_cols(W, max(added), bs))
    raw = make_cache(total, cols, bs, D, seed)
    cmp_ = None
    if comp:
        ent = [t // m for t in total]
        cmp_ = make_cache(ent, max(1, -(-max(ent) // bs)), bs, D, seed + 1)
    g = torch.Generator().manual_seed(seed + 2)
    N = sum(added) + pad
    q = (torch.randn(N, H, D, generator=g) * qscale).to(dtype)
    start = torch.tensor(np.concatenate([[0], np.cumsum(added)]), dtype=torch.int32)
    return q, start, torch.tensor(held, dtype=torch.int32), raw, cmp_


def bounds(q, ref, nkeys, scale, dtype):
    """Elementwise bounds of |out - ref| and |lse - ref| for one call.

    Scores.  fp32 sums of D products, each rounding (or a truncation, on the
    tensor cores) at most 2^-23 of the sum of magnitudes: D 2^-23 scale spread.
    bf16: q goes in as fp16 with a power-of-two factor that puts a row's largest
    |q| at 224 .. 448, exact (8 bits) but for what falls below 2^-14, off by at
    most 2^-25 / 224 max|q| an element: scale max|q| D max|k| 2^-32.
    The exponent itself is a few roundings of the score in base 2: 8 2^-24 |s|.
    A probability is off by that, relatively; so is lse, absolutely, plus the
    sum's roundings.

    Output.  bf16: p as fp16 is off by 2^-11, or by 2^-25 of the largest where it
    is tiny, once a key: 2^-20 for values that differ by up to 2^5; the result is
    rounded by 2^-8.  fp32: nkeys roundings of 2^-24."""
    out, lse, mass, spread = ref
    D = q.shape[2]
    e = D * 2.0 ** -23 * abs(scale) * spread + 8 * 2.0 ** -24 * (np.abs(lse) + abs(scale) * spread)
    if dtype == torch.bfloat16:
        qmax = float(q.float().abs().max())
        kmax = 448.0 * 2.0 ** -6 * 2  # largest key of make_cache
        e = e + abs(scale) * qmax * D * kmax * 2.0 ** -32
    lse_tol = e + 2.0 ** -22 * (np.abs(lse) + 1.0)
    p = 2 * e + 2.0 ** -20
    if dtype == torch.bfloat16:
        p = p + 2.0 ** -11 + nkeys * 2.0 ** -20
        out_tol = 2.0 ** -8 * np.abs(out) + p[..., None] * 2 * mass
    else:
        out_tol = 2.0 ** -22 * np.abs(out) + (p + nkeys * 2.0 ** -24)[..., None] * 2 * mass
    return out_tol, lse_tol


def check_attn(got, q, start, held, raw, comp, W, m, scale, dtype):
    ref = OC.attend(q.float().double().numpy(), start.numpy(), held.numpy(), oracle_cache(raw), oracle_cache(comp), W, m,
                    scale)
    n = int(start[-1])
    last = int((held + start[1:] - start[:-1]).max()) if len(held) else 0
    nkeys = min(W, last) + (last // m if comp is not None else 0)
    out_tol, lse_tol = bounds(q, ref, nkeys, scale, dtype)
    out, lse = got[0].float().cpu().double().numpy(), got[1].cpu().double().numpy()
    for name, g, r, tol in (("out", out, ref[0], out_tol), ("lse", lse, ref[1], lse_tol)):
        g, r, tol = g[:n], r[:n], tol[:n]
        assert np.all(np.isfinite(g)), f"{name}: {np.argwhere(~np.isfinite(g))[:4].tolist()} not finite"
        bad = np.argwhere(np.abs(g - r) > tol)
        assert not len(bad), (f"{name}: {len(bad)} of {g.size} off, first {bad[0].tolist()}: {g[tuple(bad[0])]} for "
                              f"{r[tuple(bad[0])]}, bound {tol[tuple(bad[0])]}")


def scale_of(D):
    return 1.0 / math.sqrt(D)
