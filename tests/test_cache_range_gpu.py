"""Attention over the cache where block scales, probabilities and scores lie far
apart, against the fp64 oracle, token by token and key by key."""
import numpy as np
import pytest
import torch

from _cache import E4M3, attn_case, make_cache, oracle_cache, scale_of
from block_sparse_compressed_gb300 import hca
from oracle import cache as OC

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


def dev(c):
    return None if c is None else tuple(t.to(DEV) for t in c)


def tolerances(kv, p, lse, spread, scale, dtype, qmax):
    """Bounds of |out - ref| [H,D] and |lse - ref| [H] of one token.

    Scores.  fp32 sums of D products, each rounding or truncation at most 2^-23 of
    the sum of magnitudes, and a few roundings of the score in base 2: a key's
    score is off by e = |scale| (D + 8) 2^-23 spread.  bf16: q's elements below
    2^-14 of fp16, where a row's largest is at least 224, lose 2^-25 / 224 of it:
    |scale| max|q| 2^-32 sum_d |k_d|.
    Probabilities.  Relatively off by 2 e and 2^-21; bf16: rounded to fp16, by
    2^-11, or by 2^-25 of the row's largest where they are tiny.
    lse is off by the probability-weighted e, roundings of the reference (2^-23 of
    it) and of n sums of positive terms; the largest e bounds the weighted one.
    Output.  What the probabilities' errors multiply, |k|, plus the sum's own
    roundings in fp32: n / 16 partial sums on the tensor cores, n otherwise, each
    2^-23 of the mass; the denominator's error; the rounding of the result."""
    n = kv.shape[0]
    e = abs(scale) * (kv.shape[1] + 8) * 2.0 ** -23 * spread
    if dtype == BF16:
        e = e + abs(scale) * qmax[:, None] * 2.0 ** -32 * np.abs(kv).sum(1)[None]
    e = np.minimum(e, 1.0)
    # a key that hardly counts may be off by more than one that does
    we = (p * 2 * e).sum(1)
    off = p * (2 * e + 2.0 ** -21)
    if dtype == BF16:
        off = off + np.maximum(p * 2.0 ** -11, 2.0 ** -25 * p.max(1, keepdims=True))
    mass, out = p @ np.abs(kv), p @ kv
    steps = n / 16 + 16 if dtype == BF16 else n
    lse_tol = we + 2.0 ** -22 * (np.abs(lse) + 1) + n * 2.0 ** -24
    out_tol = off @ np.abs(kv) + steps * 2.0 ** -23 * mass + (2 * we + n * 2.0 ** -24)[:, None] * np.abs(out)
    # the output's own rounding, below its type's smallest normal too
    return out_tol + (2.0 ** -8 if dtype == BF16 else 2.0 ** -22) * np.abs(out) + 2.0 ** -133, lse_tol, out


def run(q, start, h, raw, c, W, m, scale):
    return hca.hca_cache_attn(q.to(DEV), start.to(DEV), h.to(DEV), dev(raw), dev(c), W, m, scale, check=True)


def check(got, q, start, h, raw, c, W, m, scale):
    dtype = q.dtype
    out, lse = got[0].float().cpu().double().numpy(), got[1].cpu().double().numpy()
    qd = q.float().double().numpy()
    for t, (kv, p, rl, spread) in enumerate(OC.terms(qd, start.numpy(), h.numpy(), oracle_cache(raw), oracle_cache(c), W, m, scale)):
        out_tol, lse_tol, ref = tolerances(kv, p, rl, spread, scale, dtype, np.abs(qd[t]).max(1))
        for name, g, r, tol in (("out", out[t], ref, out_tol), ("lse", lse[t], rl, lse_tol)):
            bad = np.argwhere(~(np.abs(g - r) <= tol))
            assert not len(bad), (f"token {t} {name}: {len(bad)} of {g.size} off, first {bad[0].tolist()}: {g[tuple(bad[0])]} "
                                  f"for {r[tuple(bad[0])]}, bound {tol[tuple(bad[0])]}")


def along(H, D, seed, dtype, strength):
    """(u, q): a direction of length 1 and H queries along it, each of score `strength` with a key u."""
    g = torch.Generator().manual_seed(seed)
    u = torch.randn(D, generator=g)
    u /= u.norm()
    return u, (u[None] * strength / scale_of(D) * torch.linspace(0.9, 1.1, H)[:, None])[None].to(dtype)


def flat_cache(n, bs, D, u, along_u, seed):
    """A full-table cache of n rows along_u * u + noise in blocks of scale 2^-7."""
    g = torch.Generator().manual_seed(seed)
    pool, scale, table = make_cache([n], -(-n // bs), bs, D, seed)
    for b in range(-(-n // bs)):
        x = along_u * u[None] + 0.2 * torch.randn(bs, D, generator=g) / D ** 0.5
        pool[int(table[0, b])] = (x * 2.0 ** 7).clamp(-448, 448).to(E4M3)
    scale.fill_(2.0 ** -7)
    if n % bs:
        pool.view(torch.uint8)[int(table[0, -1]), n % bs:] = 0x7F
    return pool, scale, table


GROUPS = [(BF16, 16, 64), (BF16, 64, 128), (BF16, 128, 64), (F32, 4, 64)]


@pytest.mark.parametrize("dtype,H,D", GROUPS)
@pytest.mark.parametrize("ratio,tail", [(10, 16), (13, 13), (16, 10), (16, 13), (20, 8)])
@pytest.mark.parametrize("place", [0, 7, 200])
def test_a_peaked_small_row_in_a_block_of_great_scale(dtype, H, D, ratio, tail, place):
    # a row of zeros has the largest score of a long flat tail; its block's scale is
    # 2^ratio times the others'
    n, bs = 20000, 64
    u, q = along(H, D, 3, dtype, tail * np.log(2.0))
    raw = flat_cache(n, bs, D, u, -1.0, 4)
    b = int(raw[2][0, place])
    raw[0].view(torch.uint8)[b] = 0                       # rows of zeros
    raw[0][b, 0] = (-u * 200).to(E4M3)                   # one so large that its score leaves it no probability
    raw[1][b] = 2.0 ** (ratio - 7)
    start, held = torch.tensor([0, 1], dtype=torch.int32), torch.tensor([n - 1], dtype=torch.int32)
    a = (q, start, held, raw, None, 1 << 30, 4, scale_of(D))
    check(run(*a), *a)


@pytest.mark.parametrize("dtype,H,D", GROUPS)
@pytest.mark.parametrize("bs", [16, 128])
@pytest.mark.parametrize("exps", [(-89,), (105,), (-60, 0), (0, -60, -96), (0, 9, -9), (-9, 0, 6, 12), (40, 55), (-20, 1, -7)])
def test_block_scales_of_any_size(dtype, H, D, bs, exps):
    # blocks of 2^exps in turn, the queries such that scores stay ordinary
    held, added, W, m = [2500, 700], [1, 2], 300, 2
    q, start, h, raw, c = attn_case(held, added, H, D, W, m, bs, dtype, 11, ring=False)
    for cache in (raw, c):
        for r in range(2):
            ids = cache[2][r][cache[2][r] >= 0].long()
            cache[1][ids] = torch.tensor([2.0 ** (exps[(k // 3) % len(exps)] - 7) for k in range(len(ids))])
    q = (q.float() * 2.0 ** -max(exps)).to(dtype)
    a = (q, start, h, raw, c, W, m, scale_of(D))
    check(run(*a), *a)


@pytest.mark.parametrize("dtype,H,D", GROUPS)
@pytest.mark.parametrize("big", [20, 60])
def test_rows_of_zeros_count_in_the_sum(dtype, H, D, big):
    # blocks of zeros have the smallest scale; beside rows of great values and scores they keep their weight
    n, bs = 9000, 32
    u, q = along(H, D, 5, dtype, 7.0)
    q = (q.float() * 2.0 ** -big).to(dtype)
    raw = flat_cache(n, bs, D, u, 1.0, 6)
    raw[1].fill_(2.0 ** (big - 7))
    ids = raw[2][0].long()
    zero = ids[torch.arange(len(ids)) % 40 != 3]
    raw[0].view(torch.uint8)[zero] = 0
    raw[1][zero] = 2.0 ** -96
    start, held = torch.tensor([0, 1], dtype=torch.int32), torch.tensor([n - 1], dtype=torch.int32)
    a = (q, start, held, raw, None, 1 << 30, 4, scale_of(D))
    check(run(*a), *a)


@pytest.mark.parametrize("dtype,H,D", GROUPS)
@pytest.mark.parametrize("order", ["rise", "fall"])
@pytest.mark.parametrize("step", [3, 5])
def test_scales_that_change_all_along(dtype, H, D, order, step):
    # every 40 blocks the scale grows (shrinks) by 2^step, over several tiles and parts
    n, bs = 12000, 16
    g = torch.Generator().manual_seed(8)
    q, start, h, raw, c = attn_case([n - 1], [1], H, D, 1 << 30, 4, bs, dtype, 8, comp=False, ring=False)
    ids = raw[2][0].long()
    k = torch.arange(len(ids)) // 40
    raw[1][ids] = torch.exp2((k if order == "rise" else k.max() - k).float() * step - 40)
    q = (torch.randn(q.shape, generator=g) * 2.0 ** (33 - step * int(k.max()))).to(dtype)
    a = (q, start, h, raw, None, 1 << 30, 4, scale_of(D))
    check(run(*a), *a)


@pytest.mark.parametrize("dtype,H,D", GROUPS)
def test_scales_that_are_no_powers_of_two(dtype, H, D):
    held, added, W, m, bs = [1500, 40], [1, 3], 200, 2, 16
    q, start, h, raw, c = attn_case(held, added, H, D, W, m, bs, dtype, 12)
    g = torch.Generator().manual_seed(9)
    for cache in (raw, c):
        cache[1].mul_(1 + torch.rand(cache[1].shape, generator=g))
    a = (q, start, h, raw, c, W, m, scale_of(D))
    check(run(*a), *a)


@pytest.mark.parametrize("H,D,T,held,W,m", [(16, 64, 1, [9000, 40], 128, 4), (64, 128, 1, [30000, 700], 128, 2), (64, 128, 3, [3000, 5], 500, 4),
                                            (128, 64, 2, [0, 9000], 1 << 30, 4), (5, 64, 40, [0, 300], 33, 3)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_ordinary_caches_within_the_bounds_of_each_token(dtype, H, D, T, held, W, m):
    q, start, h, raw, c = attn_case(held, [T] * len(held), H, D, W, m, 32, dtype, 21, ring=W < 1000)
    a = (q, start, h, raw, c, W, m, scale_of(D))
    check(run(*a), *a)


@pytest.mark.parametrize("H,D", [(16, 64), (64, 128), (128, 64)])
@pytest.mark.parametrize("sign", [1.0, -1.0])
def test_scores_up_to_the_stated_limit(H, D, sign):
    # scores of 0.1 to 0.995 of 2^24 that differ by 13 to 19 in base 2, where fp32 has
    # steps of 1 and 2: whatever the order that is left, every output is a mean of rows
    n, bs = 2000, 16
    raw = make_cache([n], -(-n // bs), bs, D, 3)
    raw[0].view(torch.uint8)[:] = 0
    v = torch.zeros(n, D)
    v[:, 0] = 448.0
    steps = torch.tensor([192.0, 208.0, 224.0, 240.0, 256.0])    # of 448, which is 32 in base 2
    k = torch.arange(n)
    v[:, 1] = torch.where(k < 300, 0.0, steps[(k // 7) % 5])
    v[:, 2:] = torch.randn(n, D - 2, generator=torch.Generator().manual_seed(1)).abs() * 100
    v.clamp_(max=448)
    for r in range(n):
        raw[0][int(raw[2][0, r // bs]), r % bs] = v[r].to(E4M3)
    raw[1].fill_(2.0 ** -7)
    q = torch.zeros(1, H, D)
    q[0, :, 0] = sign * torch.linspace(0.1, 0.995, H) * 2.0 ** 24 / scale_of(D) / 3.5
    q[0, :, 1] = 32 * np.log(2.0) / scale_of(D) / 3.5
    q = q.to(BF16)
    start, held = torch.tensor([0, 1], dtype=torch.int32), torch.tensor([n - 1], dtype=torch.int32)
    out, lse = run(q, start, held, raw, None, 1 << 30, 4, scale_of(D))
    assert bool(torch.isfinite(lse).all()) and bool(torch.isfinite(out).all())
    # a column of equal values is their mean, up to the sum's and the result's roundings
    assert float((out[..., 0].float() - 3.5).abs().max()) <= 3.5 * (2.0 ** -8 + 2.0 ** -10)
    assert float(out[..., 2:].float().max()) <= 3.5 * (1 + 2.0 ** -8 + 2.0 ** -10) and float(out[..., 2:].float().min()) >= 0
    top = q[0, :, 0].double() * 3.5 * scale_of(D)
    # the reference, the score and what follows: a few roundings of fp32 at 2^24 in base 2
    assert float((lse[0].double().cpu() - top).abs().max()) <= 32 + 16


@pytest.mark.parametrize("D", [144, 256])
def test_fp32_of_wide_heads_in_many_groups(D):
    # so many requests, a few of them long, that the join of many groups takes rows of more than 128
    held = [(k * 613) % 500 + (20000 if k % 31 == 0 else 0) for k in range(70)]
    q, start, h, raw, c = attn_case(held, [1] * 70, 3, D, 64, 4, 16, F32, 5)
    a = (q, start, h, raw, c, 64, 4, scale_of(D))
    check(run(*a), *a)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("N", [5, 700])
def test_append_keeps_a_scale_that_is_no_power_of_two(dtype, N):
    # rows behind others in blocks of scales 1 .. 2 and large enough: x times fp32's 1 / s
    bs, D = 32, 64
    nblocks = -(-N // 5)
    g = torch.Generator().manual_seed(4)
    x = torch.randn(N, D, generator=g).to(dtype)
    slots = torch.tensor([k // 5 * bs + 11 + k % 5 for k in range(N)], dtype=torch.int32)
    pool = (torch.randn(nblocks, bs, D, generator=g) * 100).clamp(-448, 448).to(E4M3)
    scale = 1 + torch.rand(nblocks, generator=g)
    p, s = pool.to(DEV), scale.to(DEV)
    hca.hca_cache_append(x.to(DEV), slots.to(DEV), p, s, check=True)
    want = pool.float().double().numpy()
    inv = (1 / scale).double().numpy()[slots.numpy() // bs]
    scaled = (x.float() * torch.from_numpy(inv).float()[:, None]).double().numpy()
    want.reshape(-1, D)[slots.numpy()] = OC.e4m3_round(scaled)
    assert torch.equal(s.cpu(), scale)
    np.testing.assert_array_equal(p.float().cpu().double().numpy(), want)


@pytest.mark.parametrize("H,D", [(16, 64), (64, 128), (128, 64)])
def test_probabilities_beside_other_scales_are_rounded_once(H, D):
    # blocks of scales 1 .. 2.  A token sees a key with the top score and values of 0 and
    # two of nearly equal scores and opposite values, so that the result is the
    # difference of two probabilities, and what their roundings leave of it shows
    R, bs, W, half = 150, 16, 3, D // 2
    g = torch.Generator().manual_seed(6)
    raw = make_cache([3] * R, 1, bs, D, 6)
    u = torch.randn(half, generator=g)
    raw[1].copy_(2.0 ** -7 * (1 + torch.rand(raw[1].shape, generator=g)))
    for r in range(R):
        k = torch.zeros(3, D)
        k[0, :half] = 100 * u + 10 * torch.randn(half, generator=g)
        k[1, :half] = 40 * u + 10 * torch.randn(half, generator=g)
        k[2, :half] = k[1, :half]
        k[2, r % half] *= 1.15                      # one step of e4m3 or two
        k[1, half:] = 300 * torch.randn(half, generator=g).sign()
        k[2, half:] = -k[1, half:]
        raw[0][int(raw[2][r, 0]), :3] = k.clamp(-448, 448).to(E4M3)
    q = torch.zeros(R, H, D)
    q[..., :half] = u / half ** 0.5 * (1 + torch.rand(R, H, 1, generator=g))
    q = q.to(BF16)
    start, held = torch.arange(R + 1, dtype=torch.int32), torch.full((R,), 2, dtype=torch.int32)
    a = (q, start, held, raw, None, W, 4, scale_of(D))
    check(run(*a), *a)
