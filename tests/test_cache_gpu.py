"""GPU parity of the serving calls (hca_cache_plan, hca_cache_append,
hca_cache_attn) against the fp64 oracle in oracle/cache.py.  Slots, tables and
cache bytes have to be equal; attention outputs lie within the bounds derived in
_cache.bounds."""
import numpy as np
import pytest
import torch

from _cache import E4M3, attn_case, check_attn, make_cache, ring_cols, scale_of, values
from block_sparse_compressed_gb300 import hca
from oracle import cache as OC

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
E_CAP, E_CACHE = 11, 12


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def dev(c):
    return None if c is None else tuple(t.to(DEV) for t in c)


# ---------------------------------------------------------------------------
# plan
# ---------------------------------------------------------------------------
def _plan_inputs(R, len_hi, add_hi, bs, m, cols, seed, spare=5):
    rng = np.random.default_rng(seed)
    held, added = rng.integers(0, len_hi + 1, R), rng.integers(0, add_hi + 1, R)
    need = np.minimum(-(-((held + added) // m) // bs), cols)
    used = np.minimum(-(-(held // m) // bs), cols)
    nblocks = int(need.sum()) + spare
    perm = rng.permutation(nblocks).astype(np.int32)
    table = np.full((R, cols), -1, dtype=np.int32)
    at = 0
    for r in range(R):
        table[r, :used[r]] = perm[at:at + used[r]]
        at += used[r]
    return held, added, table, perm[at:].copy(), nblocks, int(((held + added) // m - held // m).sum())


@pytest.mark.parametrize("R,len_hi,add_hi,bs,m,cols,extra", [
    (1, 0, 1, 16, 1, 1, 0),
    (1, 0, 700, 16, 1, 44, 3),         # a prompt
    (64, 60000, 1, 64, 1, 3, 0),       # decode into rings
    (64, 60000, 1, 64, 128, 8, 64),    # decode: most requests complete no window
    (37, 300, 500, 16, 1, 2, 9),       # ring narrower than the step: entries overwritten at once
    (1500, 100, 5, 32, 4, 4, 1),       # more requests than threads
    (5, 10, 30000, 128, 1, 300, 0),    # slots by many CTAs
    (9, 0, 0, 16, 1, 1, 4),            # nothing to add
])
def test_plan_matches_oracle(R, len_hi, add_hi, bs, m, cols, extra):
    held, added, table, free, nblocks, n = _plan_inputs(R, len_hi, add_hi, bs, m, cols, R + bs + m)
    start, slots, left, want = OC.plan(held, added, table, free, len(free), bs, n + extra, m)
    t = torch.from_numpy(table).to(DEV)
    count = i32([len(free)])
    got = hca.hca_cache_plan(i32(held), i32(added), t, i32(free), count, nblocks, bs, n + extra, m=m, check=True)
    assert got[0].tolist() == start
    assert got[1].tolist() == slots
    assert got[2].tolist() == [left] and count.tolist() == [len(free)]
    assert np.array_equal(t.cpu().numpy(), want)
    live = [s for s in slots if s >= 0]
    assert len(set(live)) == len(live)


def test_plan_counts_in_place_and_follows_itself():
    # steps one after the other, the count of free blocks updated where it is
    held, table, count = i32([0, 0, 0]), torch.full((3, 8), -1, dtype=torch.int32, device=DEV), i32([12])
    free = i32(list(range(12)))
    ref = (np.zeros(3, dtype=np.int64), np.full((3, 8), -1), 12)
    for step, added in enumerate(([40, 0, 3], [1, 1, 1], [0, 60, 20], [17, 0, 0])):
        a = i32(added)
        start, slots, left = hca.hca_cache_plan(held, a, table, free, count, 12, 16, 90, free_left=count, check=True)
        s0, s1, l1, t1 = OC.plan(ref[0], added, ref[1], list(range(12)), ref[2], 16, 90, 1)
        assert start.tolist() == s0 and slots.tolist() == s1 and count.tolist() == [l1]
        assert np.array_equal(table.cpu().numpy(), t1)
        held += a
        ref = (ref[0] + np.array(added), t1, l1)


@pytest.mark.parametrize("what,status", [("blocks", E_CAP), ("slots", E_CAP), ("negative", E_CACHE), ("count", E_CACHE),
                                         ("long", E_CACHE), ("minus", E_CACHE)])
@pytest.mark.parametrize("big", [False, True])
def test_plan_that_does_not_fit_changes_nothing(what, status, big):
    R, bs, cols = 5, 16, 400
    held, added = [0] * R, [1000 if big else 100] * R
    table = torch.full((R, cols), -1, dtype=torch.int32, device=DEV)
    nslots, nfree, count = R * added[0], 400, 400
    if what == "blocks":
        count = R * -(-added[0] // bs) - 1
    if what == "slots":
        nslots -= 1
    if what == "negative":
        added[3] = -1
    if what == "minus":
        held[2] = -5
    if what == "count":
        count = nfree + 1
    if what == "long":
        held[1] = (1 << 30) - 50
    ws = torch.empty(hca.load().hca_cache_plan_workspace_size(R), dtype=torch.uint8, device=DEV)
    start, slots, left = hca.hca_cache_plan(i32(held), i32(added), table, i32(list(range(nfree))), i32([count]), nfree, bs,
                                            nslots, ws=ws)
    assert hca.hca_workspace_status(ws) == status
    assert start.tolist() == [0] * (R + 1) and left.tolist() == [count]
    assert bool((slots == -1).all()) and bool((table == -1).all())


def test_plan_gives_no_slot_for_a_bad_block():
    table = torch.full((2, 3), -1, dtype=torch.int32, device=DEV)
    ws = torch.empty(512, dtype=torch.uint8, device=DEV)
    _, slots, _ = hca.hca_cache_plan(i32([0, 0]), i32([20, 3]), table, i32([1, 99, 0]), i32([3]), 8, 16, 23, ws=ws)
    assert hca.hca_workspace_status(ws) == E_CACHE
    assert slots.tolist() == [0 * 16 + k for k in range(16)] + [-1] * 4 + [16, 17, 18]


def test_plan_without_requests():
    start, slots, left = hca.hca_cache_plan(i32([]), i32([]), torch.empty(0, 2, dtype=torch.int32, device=DEV), i32([4, 5]),
                                            i32([2]), 8, 16, 3, check=True)
    assert start.tolist() == [0] and slots.tolist() == [-1] * 3 and left.tolist() == [2]


# ---------------------------------------------------------------------------
# append
# ---------------------------------------------------------------------------
def _append_inputs(N, D, bs, dtype, seed, runs, nblocks):
    """`runs`: (block, first row, rows), in the order of x."""
    g = torch.Generator().manual_seed(seed)
    x = torch.randn(N, D, generator=g) * torch.exp2(torch.randint(-9, 9, (N, 1), generator=g).float())
    pool = (torch.randn(nblocks, bs, D, generator=g) * 100).clamp(-448, 448).to(E4M3)
    scale = torch.exp2(torch.randint(-12, 3, (nblocks,), generator=g).float())
    slots = [b * bs + o + k for b, o, n in runs for k in range(n)]
    return x.to(dtype), slots, pool, scale


@pytest.mark.parametrize("D", [16, 64, 128, 208, 256])
@pytest.mark.parametrize("bs", [16, 64, 128])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_append_matches_oracle(D, bs, dtype):
    runs = [(3, 0, bs), (0, 0, 5), (7, bs - 1, 1), (6, 2, bs - 2), (1, 5, 1), (5, 0, 1), (9, bs // 2, 3)]
    pad = 4
    N = sum(n for _, _, n in runs) + pad
    x, slots, pool, scale = _append_inputs(N, D, bs, dtype, D + bs, runs, 11)
    slots = slots[:bs + 5] + [-1, -1] + slots[bs + 5:] + [-1, -1]     # padding between requests and behind the last
    want, ws = OC.append(x.float().double().numpy(), slots, values(pool), scale.double().numpy())
    p, s = pool.to(DEV), scale.to(DEV)
    hca.hca_cache_append(x.to(DEV), i32(slots), p, s, check=True)
    np.testing.assert_array_equal(s.cpu().double().numpy(), ws)
    np.testing.assert_array_equal(values(p), want)
    again, s2 = pool.to(DEV), scale.to(DEV)
    hca.hca_cache_append(x.to(DEV), i32(slots), again, s2)
    assert torch.equal(again.view(torch.uint8), p.view(torch.uint8)) and torch.equal(s, s2)


@pytest.mark.parametrize("N", [1500, 20011, 70001])
def test_append_many_rows(N):
    # a long prompt: blocks in random order, whole and cut ones
    D, bs, nblocks = 128, 64, N // 64 + 90
    perm = np.random.default_rng(1).permutation(nblocks)
    slots = [int(perm[(k + 37) // bs]) * bs + (k + 37) % bs for k in range(N)]
    x, _, pool, scale = _append_inputs(N, D, bs, BF16, 9, [], nblocks)
    want, ws = OC.append(x.float().double().numpy(), slots, values(pool), scale.double().numpy())
    p, s = pool.to(DEV), scale.to(DEV)
    hca.hca_cache_append(x.to(DEV), i32(slots), p, s, check=True)
    np.testing.assert_array_equal(s.cpu().double().numpy(), ws)
    np.testing.assert_array_equal(values(p), want)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_append_values_at_the_edges(dtype):
    bs, D = 16, 16
    big = torch.finfo(dtype).max
    x = torch.zeros(8, D)
    x[0, :4] = torch.tensor([448.0, -448.0, 2.0 ** -10, -0.0])  # exactly at the border, a tie to zero
    x[1, 0] = 449.0                                             # beyond it in fp32; bf16 has steps of 2 here and rounds it to 448
    x[2, :3] = torch.tensor([float("inf"), float("-inf"), float("nan")])
    x[3, 0] = big
    x[4, 0] = 1e-38
    x[5] = 0.0                                                  # a block of zeros
    x[6, 0] = float("nan")                                      # nothing finite but zeros
    x[7] = torch.linspace(-1, 1, D)
    x = x.to(dtype)
    slots = [k * bs for k in range(8)]
    pool, scale = torch.zeros(8, bs, D).to(E4M3), torch.ones(8)
    want, ws = OC.append(x.float().double().numpy(), slots, values(pool), scale.double().numpy())
    p, s = pool.to(DEV), scale.to(DEV)
    hca.hca_cache_append(x.to(DEV), i32(slots), p, s, check=True)
    np.testing.assert_array_equal(s.cpu().double().numpy(), ws)
    np.testing.assert_array_equal(values(p), want)
    assert ws[0] == 1.0 and ws[1] == (1.0 if dtype == BF16 else 2.0) and ws[5] == 2.0 ** -96


@pytest.mark.parametrize("N", [255, 256, 257, 1025])
def test_append_single_rows(N):
    # a decode step: every row a run of its own, in a block that holds others
    D, bs, nblocks = 64, 16, N + 3
    perm = np.random.default_rng(N).permutation(nblocks)
    slots = [int(perm[k]) * bs + (5 * k) % bs for k in range(N)]
    x, _, pool, scale = _append_inputs(N, D, bs, BF16, N, [], nblocks)
    want, ws = OC.append(x.float().double().numpy(), slots, values(pool), scale.double().numpy())
    p, s = pool.to(DEV), scale.to(DEV)
    hca.hca_cache_append(x.to(DEV), i32(slots), p, s, check=True)
    np.testing.assert_array_equal(s.cpu().double().numpy(), ws)
    np.testing.assert_array_equal(values(p), want)
    # one slot again at the end: reported, whichever way the rows are taken
    ws = torch.empty(hca.load().hca_cache_append_workspace_size(nblocks), dtype=torch.uint8, device=DEV)
    hca.hca_cache_append(x.to(DEV), i32(slots[:-1] + [slots[0]]), p, s, ws=ws)
    assert hca.hca_workspace_status(ws) == E_CACHE


def test_append_touches_nothing_else():
    bs, D, nblocks = 32, 64, 6
    x, slots, pool, scale = _append_inputs(9, D, bs, BF16, 4, [(2, 20, 9)], nblocks)
    pool.view(torch.uint8)[2, 29:] = 0x7F
    p, s = pool.to(DEV), scale.to(DEV)
    hca.hca_cache_append((x * 2 ** 12).to(BF16).to(DEV), i32(slots), p, s, check=True)
    a, b = p.cpu().view(torch.uint8), pool.view(torch.uint8)
    assert bool((a[2, 29:] == 0x7F).all())
    keep = [0, 1, 3, 4, 5]
    assert torch.equal(a[keep], b[keep]) and torch.equal(s.cpu()[keep], scale[keep])
    assert float(s[2]) > float(scale[2])


def test_append_refuses_on_the_device():
    bs, D, nblocks = 16, 64, 4
    ws = torch.empty(hca.load().hca_cache_append_workspace_size(nblocks), dtype=torch.uint8, device=DEV)
    x, _, pool, scale = _append_inputs(6, D, bs, F32, 4, [], nblocks)

    def call(slots, scale=scale):
        p, s = pool.to(DEV), scale.to(DEV)
        hca.hca_cache_append(x.to(DEV), i32(slots), p, s, ws=ws)
        return hca.hca_workspace_status(ws), p.cpu().view(torch.uint8), s.cpu()

    assert call([0, 1, -1, 16, 17, -5])[0] == 0
    st, p, _ = call([0, 1, nblocks * bs, 2 ** 31 - 1, 16, 17])      # slots behind the pool are skipped
    assert st == E_CACHE and torch.equal(p[2:], pool.view(torch.uint8)[2:])
    # the same slot twice, and a block's rows apart: reported; other blocks are written
    for slots in ([5, 5, 33, 34, 35, 36], [5, 6, 33, 34, 35, 7], [0, 1, 33, 34, 0, 1]):
        st, p, s = call(slots)
        want, sw = OC.append(x[2:5].double().numpy() if slots[4] == 35 else x[2:4].double().numpy(),
                             [33, 34, 35] if slots[4] == 35 else [33, 34], values(pool), scale.double().numpy())
        if slots[5] == 36:
            want, sw = OC.append(x[2:6].double().numpy(), [33, 34, 35, 36], values(pool), scale.double().numpy())
        assert st == E_CACHE
        np.testing.assert_array_equal(values(p.view(E4M3))[1:], want[1:])
        np.testing.assert_array_equal(s.double().numpy()[1:], sw[1:])
    for bad in (float("nan"), 0.0, -1.0, float("inf")):
        sc = scale.clone()
        sc[0] = bad
        st, p, s = call([3, 4, -1, -1, -1, -1], sc)
        assert st == E_CACHE and float(s[0]) == OC.block_scale(float(x[:2].abs().max()))
    assert call([0, 1, 2, 3, 4, 5])[0] == 0          # the workspace keeps nothing of it


def test_append_refuses_padding_inside_a_block():
    # rows of one block are adjacent: a skipped row among them makes two runs of it
    D, bs = 16, 16
    x, slots, pool, scale = _append_inputs(bs + 2, D, bs, BF16, 32, [(3, 0, bs)], 11)
    p, s = pool.to(DEV), scale.to(DEV)
    with pytest.raises(hca.HCAError) as e:
        hca.hca_cache_append(x.to(DEV), i32(slots[:7] + [-1, -1] + slots[7:]), p, s, check=True)
    assert e.value.status == E_CACHE


def test_append_of_nothing():
    pool, scale = torch.zeros(2, 16, 64, device=DEV).to(E4M3), torch.ones(2, device=DEV)
    hca.hca_cache_append(torch.zeros(0, 64, device=DEV), i32([]), pool, scale, check=True)


# ---------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------
CASES = [
    # held, added, H, D, W, m, bs
    ([0], [1], 64, 128, 128, 128, 64),                             # the first token
    ([0, 1, 126, 127, 128, 255], [1] * 6, 16, 128, 128, 128, 64),  # windows about to complete
    ([700, 3, 0, 1291], [1, 1, 1, 1], 64, 128, 128, 4, 64),        # several tiles
    ([700, 3, 0, 1291], [3, 0, 5, 1], 64, 128, 128, 4, 64),        # ragged, one request without tokens
    ([40, 500], [2, 7], 128, 128, 64, 16, 16),
    ([300, 90, 17], [1, 1, 1], 5, 64, 64, 16, 32),                 # odd head count
    ([300, 90, 17], [4, 1, 9], 5, 64, 64, 16, 16),
    ([129], [130], 1, 128, 33, 8, 128),                            # one head, many positions a group
    ([20, 400], [3, 1], 200, 64, 50, 16, 32),                      # more heads than a group has columns
    ([20, 400], [1, 1], 96, 128, 50, 16, 64),
    ([20, 400], [1, 2], 24, 128, 1, 1, 16),                        # W = 1, every row its own entry
    ([0, 0], [70, 301], 8, 64, 7, 3, 16),                          # prompts from nothing
]


@pytest.mark.parametrize("held,added,H,D,W,m,bs", CASES)
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("comp", [True, False])
def test_attention_matches_oracle(held, added, H, D, W, m, bs, dtype, comp):
    q, start, h, raw, c = attn_case(held, added, H, D, W, m, bs, dtype, sum(held) + H, comp=comp)
    got = hca.hca_cache_attn(q.to(DEV), start.to(DEV), h.to(DEV), dev(raw), dev(c), W, m, scale_of(D), check=True)
    check_attn(got, q, start, h, raw, c, W, m, scale_of(D), dtype)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("H,T", [(3, 1), (40, 1), (64, 1), (64, 2), (128, 1)])
def test_attention_of_every_block_size_and_group(D, bs, H, T):
    held = [5 * bs + 3, 0, 700]
    q, start, h, raw, c = attn_case(held, [T, 1, T], H, D, 150, 2, bs, BF16, bs + H + T)
    got = hca.hca_cache_attn(q.to(DEV), start.to(DEV), h.to(DEV), dev(raw), dev(c), 150, 2, scale_of(D), check=True)
    check_attn(got, q, start, h, raw, c, 150, 2, scale_of(D), BF16)


@pytest.mark.parametrize("D", [16, 48, 80, 256])
def test_fp32_attention_of_other_head_dims(D):
    held, added, H, W, m, bs = [77, 300], [2, 1], 3, 40, 8, 16
    q, start, h, raw, c = attn_case(held, added, H, D, W, m, bs, F32, D)
    got = hca.hca_cache_attn(q.to(DEV), start.to(DEV), h.to(DEV), dev(raw), dev(c), W, m, scale_of(D), check=True)
    check_attn(got, q, start, h, raw, c, W, m, scale_of(D), F32)


@pytest.mark.parametrize("dtype,H,D,qscale", [(BF16, 64, 128, 8.0), (BF16, 16, 64, 20.0), (F32, 4, 64, 8.0)])
@pytest.mark.parametrize("W", [128, 1 << 30])
def test_attention_with_peaked_scores(dtype, H, D, qscale, W):
    # the largest score moves from tile to tile and far beyond the first one's
    held, added, m, bs = [9000, 2500], [1, 2], 4, 64
    q, start, h, raw, c = attn_case(held, added, H, D, W, m, bs, dtype, 3, ring=W < 1000, qscale=qscale)
    got = hca.hca_cache_attn(q.to(DEV), start.to(DEV), h.to(DEV), dev(raw), dev(c), W, m, scale_of(D), check=True)
    check_attn(got, q, start, h, raw, c, W, m, scale_of(D), dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_with_scores_that_rise(dtype):
    # keys along q, later ones larger: every tile beats the reference of all before it
    held, added, H, D, W, m, bs = [4000], [1], 16, 128, 1 << 20, 4, 64
    q, start, h, raw, c = attn_case(held, added, H, D, W, m, bs, dtype, 8, ring=False)
    dirn = torch.randn(D, generator=torch.Generator().manual_seed(1))
    for pool, sc, table in (raw, c):
        n = 4001 if pool is raw[0] else 1000
        for k in range(n):
            b = int(table[0, k // bs])
            pool[b, k % bs] = (dirn * (20 + 300 * k / n)).clamp(-448, 448).to(E4M3)
        sc.fill_(2.0 ** -7)
    q = (dirn * torch.linspace(-2, 2, H)[:, None])[None].to(dtype)
    got = hca.hca_cache_attn(q.to(DEV), start.to(DEV), h.to(DEV), dev(raw), dev(c), W, m, scale_of(D), check=True)
    check_attn(got, q, start, h, raw, c, W, m, scale_of(D), dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("scale", [-0.09, 0.0])
def test_attention_with_other_scales(dtype, scale):
    held, added, H, D, W, m, bs = [600, 30], [1, 3], 16, 64, 64, 4, 16
    q, start, h, raw, c = attn_case(held, added, H, D, W, m, bs, dtype, 6)
    got = hca.hca_cache_attn(q.to(DEV), start.to(DEV), h.to(DEV), dev(raw), dev(c), W, m, scale, check=True)
    check_attn(got, q, start, h, raw, c, W, m, scale, dtype)


@pytest.mark.parametrize("dtype,H,D", [(BF16, 64, 128), (BF16, 16, 64), (F32, 4, 64)])
def test_attention_with_block_scales_far_apart(dtype, H, D):
    # a block of tiny rows beside one of ordinary ones, zeros at the smallest scale
    held, added, W, m, bs = [2000], [1], 128, 4, 16
    q, start, h, raw, c = attn_case(held, added, H, D, W, m, bs, dtype, 12)
    c[1][::3] = 2.0 ** -60
    c[1][1::5] = 2.0 ** -96
    c[0][int(c[2][0, 4])] = 0.0
    got = hca.hca_cache_attn(q.to(DEV), start.to(DEV), h.to(DEV), dev(raw), dev(c), W, m, scale_of(D), check=True)
    check_attn(got, q, start, h, raw, c, W, m, scale_of(D), dtype)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_rows_behind_the_last_token_are_left(dtype):
    held, added, H, D, W, m, bs = [50, 8], [1, 2], 16, 64, 32, 4, 16
    q, start, h, raw, c = attn_case(held, added, H, D, W, m, bs, dtype, 2, pad=5)
    q[3:] = float("nan")
    out = torch.full_like(q, 7.0).to(DEV)
    lse = torch.full((8, H), 7.0, device=DEV)
    hca.hca_cache_attn(q.to(DEV), start.to(DEV), h.to(DEV), dev(raw), dev(c), W, m, scale_of(D), out=out, lse=lse, check=True)
    check_attn((out, lse), q[:3], start, h, raw, c, W, m, scale_of(D), dtype)
    assert bool((out[3:] == 7).all()) and bool((lse[3:] == 7).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_nan_in_one_query_row_stays_there(dtype):
    held, added, H, D, W, m, bs = [500, 300], [1, 1], 16, 64, 64, 4, 16
    q, start, h, raw, c = attn_case(held, added, H, D, W, m, bs, dtype, 2)
    q[0, 3, 5] = float("nan")
    q[1, 7, 9] = float("inf")
    out, lse = hca.hca_cache_attn(q.to(DEV), start.to(DEV), h.to(DEV), dev(raw), dev(c), W, m, scale_of(D), check=True)
    bad = ~torch.isfinite(lse)
    assert bad.nonzero().tolist() == [[0, 3], [1, 7]]
    q[0, 3], q[1, 7] = 0, 0
    out[0, 3], out[1, 7] = 0, 0
    fin = torch.isfinite(out).all(2)
    assert bool(fin.all())
    ref = OC.attend(q.float().double().numpy(), start.numpy(), h.numpy(), *[(values(x[0]), x[1].double().numpy(), x[2].numpy())
                                                                          for x in (raw, c)], W, m, scale_of(D))
    err = np.abs(out.float().cpu().double().numpy() - ref[0])
    err[0, 3], err[1, 7] = 0, 0
    assert err.max() < 0.05


@pytest.mark.parametrize("dtype,H,D", [(BF16, 16, 64), (BF16, 64, 128), (F32, 4, 64)])
def test_nan_in_a_row_reaches_only_the_tokens_that_see_it(dtype, H, D):
    # four tokens in one step; the third one's own row and the entry that it
    # completes hold NaN, the row at the window's far end of the first too
    held, added, W, m, bs = [77], [4], 30, 8, 16
    q, start, h, raw, c = attn_case(held, added, H, D, W, m, bs, dtype, 2, ring=False)
    clean = tuple(t.clone() for t in raw), tuple(t.clone() for t in c)
    for cache, e in ((raw, 79), (raw, 48), (c, 9)):
        cache[0].view(torch.uint8)[int(cache[2][0, e // bs]), e % bs, 5] = 0xFF
    out, lse = hca.hca_cache_attn(q.to(DEV), start.to(DEV), h.to(DEV), dev(raw), dev(c), W, m, scale_of(D), check=True)
    want, wl = hca.hca_cache_attn(q.to(DEV), start.to(DEV), h.to(DEV), dev(clean[0]), dev(clean[1]), W, m, scale_of(D))
    # row 48 is in the window of token 77 only, row 79 and entry 9 are seen from token 79 on
    for t in (0, 2, 3):
        assert bool(torch.isnan(out[t]).all()) and bool(torch.isnan(lse[t]).all())
    assert torch.equal(out[1], want[1]) and torch.equal(lse[1], wl[1])


def _status_case(dtype=BF16):
    held, added, H, D, W, m, bs = [500, 300, 40], [1, 1, 2], 16, 64, 64, 4, 16
    q, start, h, raw, c = attn_case(held, added, H, D, W, m, bs, dtype, 2)
    n = hca.load().hca_cache_attn_workspace_size(q.shape[0], 3, H, D, 0 if dtype == BF16 else 1)
    ws = torch.empty(n, dtype=torch.uint8, device=DEV)

    def call(start=start, h=h, raw=raw, c=c):
        out, lse = torch.full_like(q, 7.0).to(DEV), torch.full((4, H), 7.0, device=DEV)
        hca.hca_cache_attn(q.to(DEV), start.to(DEV), h.to(DEV), dev(raw), dev(c), W, m, scale_of(D), out=out, lse=lse, ws=ws)
        return hca.hca_workspace_status(ws), out.float().cpu(), lse.cpu()

    return call, start, h, raw, c


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_attention_refuses_bad_lengths_on_the_device(dtype):
    call, start, h, raw, c = _status_case(dtype)
    good = call()
    assert good[0] == 0 and bool(torch.isfinite(good[1]).all())
    t = lambda *v: torch.tensor(v, dtype=torch.int32)  # noqa: E731
    narrow = (raw[0], raw[1], raw[2][:, :3].contiguous())
    short = (c[0], c[1], c[2][:, :7].contiguous())
    for kw in (dict(start=t(0, 2, 1, 4)), dict(start=t(1, 2, 3, 4)), dict(start=t(0, 1, 2, 5)), dict(start=t(0, -1, 2, 4)),
               dict(h=t(500, -1, 40)), dict(h=t(500, 300, (1 << 30) - 1)), dict(raw=narrow), dict(c=short)):
        st, out, lse = call(**kw)
        assert st == E_CACHE, kw
        assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all()), kw
    again = call()
    assert again[0] == 0 and torch.equal(again[1], good[1]) and torch.equal(again[2], good[2])


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bad", [-1, 10 ** 6, -2 ** 31, 2 ** 31 - 1])
def test_a_bad_block_id_is_reported(dtype, bad):
    call, start, h, raw, c = _status_case(dtype)
    good = call()
    table = c[2].clone()
    table[1, 2] = bad
    st, out, lse = call(c=(c[0], c[1], table))
    assert st == E_CACHE
    assert bool(torch.isnan(out[1]).all()) and bool(torch.isnan(lse[1]).all())
    for k in (0, 2, 3):
        assert torch.equal(out[k], good[1][k]) and torch.equal(lse[k], good[2][k])
    table = raw[2].clone()
    table[2, 0] = bad
    st, out, lse = call(raw=(raw[0], raw[1], table))
    assert st == E_CACHE and bool(torch.isnan(out[2:]).all()) and bool(torch.isfinite(out[:2]).all())
    assert call()[0] == 0


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("bad", [0.0, -1.0, float("inf"), float("nan")])
def test_a_bad_scale_is_reported(dtype, bad):
    call, start, h, raw, c = _status_case(dtype)
    good = call()
    scale = c[1].clone()
    scale[int(c[2][0, 3])] = bad
    st, out, lse = call(c=(c[0], scale, c[2]))
    assert st == E_CACHE and bool(torch.isnan(out[0]).all()) and bool(torch.isnan(lse[0]).all())
    assert torch.equal(out[1:], good[1][1:]) and torch.equal(lse[1:], good[2][1:])


def test_attention_without_tokens():
    q, start, h, raw, c = attn_case([5, 9], [0, 0], 16, 64, 32, 4, 16, BF16, 2)
    out, lse = hca.hca_cache_attn(q.to(DEV), start.to(DEV), h.to(DEV), dev(raw), dev(c), 32, 4, 0.1, check=True)
    assert out.shape == (0, 16, 64) and lse.shape == (0, 16)
    q = torch.zeros(3, 16, 64, dtype=BF16, device=DEV)
    out = torch.full_like(q, 5.0)
    hca.hca_cache_attn(q, start.to(DEV), h.to(DEV), dev(raw), dev(c), 32, 4, 0.1, out=out, check=True)
    assert bool((out == 5).all())


@pytest.mark.parametrize("dtype,H,D,T", [(BF16, 64, 128, 1), (BF16, 128, 128, 1), (BF16, 16, 64, 3), (F32, 4, 64, 1)])
def test_attention_of_many_requests_gives_the_same_bits_twice(dtype, H, D, T):
    R, W, m, bs = 90, 128, 16, 32
    held = [(k * 977) % 3001 for k in range(R)]
    q, start, h, raw, c = attn_case(held, [T] * R, H, D, W, m, bs, dtype, 4)
    args = (q.to(DEV), start.to(DEV), h.to(DEV), dev(raw), dev(c), W, m, scale_of(D))
    a = hca.hca_cache_attn(*args, check=True)
    b = hca.hca_cache_attn(*args, check=True)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check_attn(a, q, start, h, raw, c, W, m, scale_of(D), dtype)


def test_requests_do_not_depend_on_their_neighbours():
    # a request alone gives what it gives in a batch, up to the order of a split sum
    R, H, D, W, m, bs = 40, 64, 128, 128, 8, 64
    held = [(k * 613) % 6000 for k in range(R)]
    q, start, h, raw, c = attn_case(held, [1] * R, H, D, W, m, bs, BF16, 14)
    a, la = hca.hca_cache_attn(q.to(DEV), start.to(DEV), h.to(DEV), dev(raw), dev(c), W, m, scale_of(D), check=True)
    for r in (0, 7, 39):
        one = (torch.tensor([0, 1], dtype=torch.int32, device=DEV), h[r:r + 1].to(DEV))
        b, lb = hca.hca_cache_attn(q[r:r + 1].to(DEV), one[0], one[1], (raw[0].to(DEV), raw[1].to(DEV), raw[2][r:r + 1].to(DEV)),
                                   (c[0].to(DEV), c[1].to(DEV), c[2][r:r + 1].to(DEV)), W, m, scale_of(D), check=True)
        assert float((a[r:r + 1].float() - b.float()).abs().max()) <= 2 * 2.0 ** -8 * float(b.float().abs().max())
        assert float((la[r:r + 1] - lb).abs().max()) <= 1e-5 * float(lb.abs().max())


def test_cache_beyond_32_bit_offsets():
    # a pool of over 4 GB, the request's blocks at both of its ends
    bs, D, H, W, m = 128, 128, 16, 128, 4
    nblocks = (1 << 32) // (bs * D) + 700
    pool = torch.empty(nblocks, bs, D, dtype=torch.uint8, device=DEV)
    pool[:300] = 0x7F
    pool[-600:] = 0x7F
    pool = pool.view(E4M3)
    scale = torch.ones(nblocks, device=DEV)
    n = 1000
    x = torch.randn(n, D, generator=torch.Generator().manual_seed(1)).to(BF16)
    ids = [nblocks - 1, 3, nblocks - 300, nblocks - 2, 0, nblocks - 599, 17, nblocks - 5]
    slots = [ids[k // bs] * bs + k % bs for k in range(n)]
    hca.hca_cache_append(x.to(DEV), i32(slots), pool, scale, check=True)
    small = torch.empty(8, bs, D, dtype=torch.uint8)
    for k, b in enumerate(ids):
        small[k] = pool[b].view(torch.uint8).cpu()
    sc = scale[torch.tensor(ids, device=DEV)].cpu()
    want, sw = OC.append(x.float().double().numpy(), list(range(n)), np.zeros((8, bs, D)), np.ones(8))
    np.testing.assert_array_equal(values(small.view(E4M3)).reshape(-1, D)[:n], want.reshape(-1, D)[:n])
    np.testing.assert_array_equal(sc.double().numpy(), sw)
    q = torch.randn(1, H, D, generator=torch.Generator().manual_seed(2)).to(BF16)
    start, held = torch.tensor([0, 1], dtype=torch.int32), torch.tensor([n - 1], dtype=torch.int32)
    got = hca.hca_cache_attn(q.to(DEV), start.to(DEV), held.to(DEV), (pool, scale, i32([ids])), None, 1 << 30, m, scale_of(D),
                             check=True)
    check_attn(got, q, start, held, (small.view(E4M3), sc, torch.arange(8, dtype=torch.int32)[None]), None, 1 << 30, m,
               scale_of(D), BF16)


# ---------------------------------------------------------------------------
# together
# ---------------------------------------------------------------------------
class Server:
    """What a serving program keeps: a shared pool for raw rows and entries, two
    tables, one free list; prompts and tokens go through plan, append, attend.
    Compressed entries come from the compressor on the last m rows."""

    def __init__(self, R, H, D, W, m, bs, dtype, t_max, len_max, graph=False):
        self.R, self.H, self.D, self.W, self.m, self.bs = R, H, D, W, m, bs
        self.cols, self.ccols = ring_cols(W, t_max, bs), -(-(len_max // m + 1) // bs)
        self.nblocks = R * (self.cols + self.ccols)
        self.pool = torch.full((self.nblocks, bs, D), 0x7F, dtype=torch.uint8, device=DEV).view(E4M3)
        self.scale = torch.ones(self.nblocks, device=DEV)
        full = lambda c: torch.full((R, c), -1, dtype=torch.int32, device=DEV)  # noqa: E731
        self.raw_table, self.comp_table = full(self.cols), full(self.ccols)
        self.free = i32(np.random.default_rng(0).permutation(self.nblocks))
        self.count = i32([self.nblocks])
        self.held = i32([0] * R)
        self.nslots = R * t_max

    def step(self, x, ent, q, added):
        """x, q rows packed by request; ent: compressed entries that complete, packed."""
        W, m, bs = self.W, self.m, self.bs
        start, slots, _ = hca.hca_cache_plan(self.held, added, self.raw_table, self.free, self.count, self.nblocks, bs,
                                             x.shape[0], free_left=self.count)
        _, cslots, _ = hca.hca_cache_plan(self.held, added, self.comp_table, self.free, self.count, self.nblocks, bs,
                                          ent.shape[0], m=m, free_left=self.count)
        hca.hca_cache_append(x, slots, self.pool, self.scale)
        hca.hca_cache_append(ent, cslots, self.pool, self.scale)
        out, lse = hca.hca_cache_attn(q, start, self.held, (self.pool, self.scale, self.raw_table),
                                      (self.pool, self.scale, self.comp_table), W, m, scale_of(self.D))
        self.held += added
        return out, lse




@pytest.mark.parametrize("dtype,H,D", [(BF16, 64, 128), (F32, 4, 64)])
def test_prompts_then_tokens(dtype, H, D):
    R, W, m, bs, T = 3, 40, 8, 16, 90
    g = torch.Generator().manual_seed(0)
    sv = Server(R, H, D, W, m, bs, dtype, T, 200)
    kv = [torch.randn(200, D, generator=g).clamp(-1.7, 1.7).to(dtype) for _ in range(R)]
    for r in range(R):
        kv[r][:, 0] = 1.75          # every row reaches 448 at the block's scale, so a block's scale never grows
    qs = [torch.randn(200, H, D, generator=g).to(dtype) for _ in range(R)]
    gate, bias = torch.randn(R, 200, generator=g), torch.zeros(m)
    comp = [hca.hca_compress_fwd(kv[r][None].to(DEV), gate[r:r + 1].to(DEV), bias.to(DEV), None, m)[0].cpu() for r in range(R)]
    for ck in comp:
        ck[:, 0] = 1.75
    held = [0] * R
    for added in ([90, 13, 0], [1, 1, 1], [1, 1, 1], [5, 0, 30], [1, 1, 1], [0, 64, 2]):
        x = torch.cat([kv[r][held[r]:held[r] + n] for r, n in enumerate(added)])
        q = torch.cat([qs[r][held[r]:held[r] + n] for r, n in enumerate(added)])
        ent = torch.cat([comp[r][held[r] // m:(held[r] + n) // m] for r, n in enumerate(added)])
        pad = torch.zeros(3, D, dtype=dtype)
        got = sv.step(torch.cat([x, pad]).to(DEV), torch.cat([ent, pad]).to(DEV), q.to(DEV), i32(added))
        # a plain cache of the same rows: request r's rows in order, quantised block by block
        raws, comps = [], []
        for r in range(R):
            n = held[r] + added[r]
            for rows, into in ((kv[r][:n], raws), (comp[r][:n // m], comps)):
                k = -(-max(1, len(rows)) // bs)
                p, s = np.zeros((k, bs, D)), np.ones(k)
                p, s = OC.append(rows.float().double().numpy(), list(range(len(rows))), p, s)
                into.append((p, s))
        start = torch.tensor(np.concatenate([[0], np.cumsum(added)]), dtype=torch.int32)

        def join(parts):
            k = max(len(s) for _, s in parts)
            table, at = np.full((R, k), -1), 0
            for r, (p, s) in enumerate(parts):
                table[r, :len(s)] = np.arange(at, at + len(s))
                at += len(s)
            pool = torch.from_numpy(np.concatenate([p for p, _ in parts])).float().to(E4M3)
            return pool, torch.from_numpy(np.concatenate([s for _, s in parts])).float(), torch.from_numpy(table).int()

        check_attn(got, q, start, torch.tensor(held, dtype=torch.int32), join(raws), join(comps), W, m, scale_of(D), dtype)
        held = [h + n for h, n in zip(held, added)]


def test_a_captured_step_serves_the_next_tokens():
    # one decode step captured once, replayed with the lengths it finds: the same
    # bits as eager steps, with compressed entries completing on the way
    R, H, D, W, m, bs, steps = 4, 64, 128, 40, 8, 16, 21
    g = torch.Generator().manual_seed(5)
    prompt = [37, 5, 64, 15]
    n0 = sum(prompt)
    x0, q0 = torch.randn(n0, D, generator=g).to(BF16).to(DEV), torch.randn(n0, H, D, generator=g).to(BF16).to(DEV)
    e0 = torch.randn(n0 // m, D, generator=g).to(BF16).to(DEV)
    xs = torch.randn(steps, R, D, generator=g).to(BF16).to(DEV)
    es = torch.randn(steps, R, D, generator=g).to(BF16).to(DEV)
    qs = torch.randn(steps, R, H, D, generator=g).to(BF16).to(DEV)

    def fresh():
        sv = Server(R, H, D, W, m, bs, BF16, 64, 200)
        sv.step(x0, e0, q0, i32(prompt))
        return sv

    one = i32([1] * R)
    eager, sv = [], fresh()
    for k in range(steps):
        eager.append([t.clone() for t in sv.step(xs[k], es[k], qs[k], one)])
    sv = fresh()
    x, e, q = xs[0].clone(), es[0].clone(), qs[0].clone()
    state = [t.clone() for t in (sv.pool.view(torch.uint8), sv.scale, sv.raw_table, sv.comp_table, sv.count, sv.held)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sv.step(x, e, q, one)
    torch.cuda.current_stream().wait_stream(side)
    for t, s in zip((sv.pool.view(torch.uint8), sv.scale, sv.raw_table, sv.comp_table, sv.count, sv.held), state):
        t.copy_(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = sv.step(x, e, q, one)
    for k in range(steps):
        x.copy_(xs[k]); e.copy_(es[k]); q.copy_(qs[k])
        graph.replay()
        assert torch.equal(out, eager[k][0]) and torch.equal(lse, eager[k][1]), k


def test_two_streams_at_once():
    # two calls in flight on two streams with workspaces of their own
    cases = []
    for seed, (H, D, dtype) in enumerate(((64, 128, BF16), (16, 64, BF16), (4, 64, F32))):
        held = [(k * 331 + seed) % 2000 for k in range(20)]
        q, start, h, raw, c = attn_case(held, [1] * 20, H, D, 64, 8, 32, dtype, seed)
        args = (q.to(DEV), start.to(DEV), h.to(DEV), dev(raw), dev(c), 64, 8, scale_of(D))
        cases.append((args, hca.hca_cache_attn(*args, check=True)))
    streams = [torch.cuda.Stream() for _ in cases]
    torch.cuda.synchronize()
    got = []
    for _ in range(5):
        for (args, _), s in zip(cases, streams):
            with torch.cuda.stream(s):
                got.append(hca.hca_cache_attn(*args))
    torch.cuda.synchronize()
    for k, (out, lse) in enumerate(got):
        want = cases[k % len(cases)][1]
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


# ---------------------------------------------------------------------------
# the binding, failures, shapes of the schedule
# ---------------------------------------------------------------------------
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_both_ways_of_the_binding_give_the_same(dtype, monkeypatch):
    hca.load()
    short = hca._py
    if short is None:
        pytest.skip("built without the headers of Python or torch")
    R, H, D, W, m, bs = 5, 8, 64, 40, 8, 16
    held, added = [70, 0, 12, 333, 5], [1, 9, 0, 2, 40]
    q, start, h, raw, c = attn_case(held, added, H, D, W, m, bs, dtype, 3)
    rows = torch.randn(sum(added), D, generator=torch.Generator().manual_seed(1)).to(dtype).to(DEV)
    seen = []

    class Spy:
        def __getattr__(self, name):
            def call(*a):
                r = getattr(short, name)(*a)
                seen.append(r is not None)
                return r
            return call

    results = []
    for py in (Spy(), None):
        monkeypatch.setattr(hca, "_py", py)
        table = torch.full((R, 40), -1, dtype=torch.int32, device=DEV)
        for r, n in enumerate(held):
            for k in range(-(-n // bs)):
                table[r, k] = 25 * r + k
        plan = hca.hca_cache_plan(i32(held), i32(added), table, i32(list(range(125, 160))), i32([35]), 160, bs, sum(added), check=True)
        pool, scale = torch.zeros(160, bs, D, device=DEV).to(E4M3), torch.ones(160, device=DEV)
        hca.hca_cache_append(rows, plan[1], pool, scale, check=True)
        attn = hca.hca_cache_attn(q.to(DEV), start.to(DEV), h.to(DEV), dev(raw), dev(c), W, m, scale_of(D), check=True)
        bare = hca.hca_cache_attn(q.to(DEV), start.to(DEV), h.to(DEV), dev(raw), None, W, m, scale_of(D), check=True)
        results.append([*plan, table, pool.view(torch.uint8), scale, *attn, *bare])
    assert seen == [True] * 4
    assert len(results[0]) == len(results[1])
    for a, b in zip(*results):
        assert a.dtype == b.dtype and torch.equal(a, b)


def test_results_go_into_the_callers_tensors():
    q, start, h, raw, c = attn_case([70, 9], [1, 2], 8, 64, 40, 8, 16, BF16, 3)
    args = (q.to(DEV), start.to(DEV), h.to(DEV), dev(raw), dev(c), 40, 8, scale_of(64))
    want = hca.hca_cache_attn(*args)
    out, lse = torch.empty_like(want[0]), torch.empty_like(want[1])
    ws = torch.empty(hca.load().hca_cache_attn_workspace_size(3, 2, 8, 64, 0), dtype=torch.uint8, device=DEV)
    got = hca.hca_cache_attn(*args, out=out, lse=lse, ws=ws, check=True)
    assert got[0] is out and got[1] is lse and torch.equal(out, want[0]) and torch.equal(lse, want[1])
    with pytest.raises(hca.HCAError):
        hca.hca_cache_attn(*args, ws=ws[:-1])
    with pytest.raises(ValueError):
        hca.hca_cache_attn(*args, ws=ws.cpu())
    with pytest.raises(TypeError):
        hca.hca_cache_attn(*args, ws=ws.float())
    none = hca.hca_cache_attn(*args[:6], 1 << 40, args[7], check=True)   # a ratio that no length reaches
    bare = hca.hca_cache_attn(*args[:4], None, 40, 1, args[7], check=True)
    assert torch.equal(none[0], bare[0]) and torch.equal(none[1], bare[1])
    with pytest.raises(ValueError):
        hca.hca_cache_attn(*args, out=out[:2])
    with pytest.raises(TypeError):
        hca.hca_cache_attn(*args, lse=lse.double())
    with pytest.raises(ValueError):
        hca.hca_cache_attn(args[0], args[1].cpu(), *args[2:])
    with pytest.raises(ValueError):
        hca.hca_cache_attn(args[0].transpose(0, 1).contiguous().transpose(0, 1), *args[1:])
    with pytest.raises(hca.HCAError):
        hca.hca_cache_attn(*args[:5], 0, *args[6:])
    with pytest.raises(hca.HCAError):
        hca.hca_cache_attn(*args[:7], float("nan"))


@pytest.mark.parametrize("H,D,T", [(64, 128, 1), (16, 64, 2), (200, 64, 1)])
def test_a_stalled_attention_times_out(H, D, T):
    # the tensor-core warp waits for what never comes: every wait ends, the status
    # says so and no stale number is left; the next call works
    held = [3000, 17, 260]
    q, start, h, raw, c = attn_case(held, [T] * 3, H, D, 64, 4, 16, BF16, 2)
    args = (q.to(DEV), start.to(DEV), h.to(DEV), dev(raw), dev(c), 64, 4, scale_of(D))
    want = hca.hca_cache_attn(*args, check=True)
    hca.hca_test_inject(hca.INJECT_WAIT_LIMIT_NS, 30_000_000)
    hca.hca_test_inject(hca.INJECT_STALL, 1)
    try:
        ws = torch.empty(hca.load().hca_cache_attn_workspace_size(3 * T, 3, H, D, 0), dtype=torch.uint8, device=DEV)
        out, lse = hca.hca_cache_attn(*args, ws=ws)
        assert hca.hca_workspace_status(ws) == 10
        assert bool(torch.isnan(out).all()) and bool(torch.isnan(lse).all())
    finally:
        hca.hca_test_inject(hca.INJECT_RESET, 0)
    got = hca.hca_cache_attn(*args, check=True)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_a_failed_launch_is_reported():
    q, start, h, raw, c = attn_case([70, 9], [1, 2], 8, 64, 40, 8, 16, BF16, 3)
    args = (q.to(DEV), start.to(DEV), h.to(DEV), dev(raw), dev(c), 40, 8, scale_of(64))
    for call in (lambda: hca.hca_cache_attn(*args),
                 lambda: hca.hca_cache_append(q[:, 0].contiguous().to(DEV), i32([-1, -1, -1]), *dev(c)[:2]),
                 lambda: hca.hca_cache_plan(i32([1]), i32([1]), i32([[0, -1]]), i32([1, 2]), i32([2]), 3, 16, 1)):
        hca.hca_test_inject(hca.INJECT_LAUNCH_FAILURE, 1)
        try:
            with pytest.raises(hca.HCAError):
                call()
        finally:
            hca.hca_test_inject(hca.INJECT_RESET, 0)
        call()


@pytest.mark.parametrize("dtype,H,D", [(BF16, 64, 128), (BF16, 1, 64), (F32, 2, 64)])
def test_more_requests_than_threads(dtype, H, D):
    held = [(k * 37) % 300 for k in range(401)]
    q, start, h, raw, c = attn_case(held, [1] * 401, H, D, 48, 8, 16, dtype, 6)
    got = hca.hca_cache_attn(q.to(DEV), start.to(DEV), h.to(DEV), dev(raw), dev(c), 48, 8, scale_of(D), check=True)
    check_attn(got, q, start, h, raw, c, 48, 8, scale_of(D), dtype)


def test_more_groups_for_a_block_than_it_lists():
    # one tile a request, more than 64 requests to a block of 304
    R, H, D, W, m, bs = 21000, 1, 64, 8, 4, 16
    held = [k % 5 for k in range(R)]
    q, start, h, raw, c = attn_case(held, [1] * R, H, D, W, m, bs, BF16, 6)
    got = hca.hca_cache_attn(q.to(DEV), start.to(DEV), h.to(DEV), dev(raw), dev(c), W, m, scale_of(D), check=True)
    check_attn(got, q, start, h, raw, c, W, m, scale_of(D), BF16)


@pytest.mark.parametrize("dtype,H,D,T", [(BF16, 64, 128, 1), (BF16, 200, 128, 1), (BF16, 16, 64, 3), (BF16, 128, 64, 2), (F32, 4, 64, 1)])
def test_one_long_request_in_many_parts(dtype, H, D, T):
    held = [9001, 20]
    q, start, h, raw, c = attn_case(held, [T, 1], H, D, 300, 2, 32, dtype, 8)
    got = hca.hca_cache_attn(q.to(DEV), start.to(DEV), h.to(DEV), dev(raw), dev(c), 300, 2, scale_of(D), check=True)
    check_attn(got, q, start, h, raw, c, 300, 2, scale_of(D), dtype)


def test_two_graphs_share_a_workspace():
    cases = [attn_case(held, [1] * len(held), 16, 64, 64, 4, 16, BF16, 5) for held in ([900, 3, 77], [12, 2500, 40])]
    ws = torch.empty(hca.load().hca_cache_attn_workspace_size(3, 3, 16, 64, 0), dtype=torch.uint8, device=DEV)
    graphs, outs, wants = [], [], []
    for q, start, h, raw, c in cases:
        args = (q.to(DEV), start.to(DEV), h.to(DEV), dev(raw), dev(c), 64, 4, scale_of(64))
        wants.append(hca.hca_cache_attn(*args, check=True))
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            outs.append(hca.hca_cache_attn(*args, ws=ws))
        graphs.append((g, args))
    for k in (0, 1, 1, 0, 1, 0, 0):
        for t in outs[k]:
            t.fill_(7)
        graphs[k][0].replay()
        assert torch.equal(outs[k][0], wants[k][0]) and torch.equal(outs[k][1], wants[k][1])
    assert hca.hca_workspace_status(ws) == 0


@pytest.mark.parametrize("H,D,held,added", [(64, 64, [3, 0, 900], [700, 1, 640]), (200, 64, [50, 0], [333, 12]), (128, 128, [0], [620])])
def test_prompts_of_more_groups_than_blocks(H, D, held, added):
    # two groups and more for each block: the line is cut between them
    q, start, h, raw, c = attn_case(held, added, H, D, 70, 4, 32, BF16, 9)
    got = hca.hca_cache_attn(q.to(DEV), start.to(DEV), h.to(DEV), dev(raw), dev(c), 70, 4, scale_of(D), check=True)
    check_attn(got, q, start, h, raw, c, 70, 4, scale_of(D), BF16)


def test_prompts_beside_a_long_request():
    # one group with far more tiles than a block's share: it has to be divided
    H, D = 128, 64
    held, added = [0, 30000], [640, 1]
    q, start, h, raw, c = attn_case(held, added, H, D, 70, 1, 64, BF16, 9)
    got = hca.hca_cache_attn(q.to(DEV), start.to(DEV), h.to(DEV), dev(raw), dev(c), 70, 1, scale_of(D), check=True)
    check_attn(got, q, start, h, raw, c, 70, 1, scale_of(D), BF16)


@pytest.mark.parametrize("fill", [0x00, 0x7F, 0xFF])
def test_what_a_workspace_holds_does_not_matter(fill):
    lib = hca.load()
    for dtype, H, D, held, added in ((BF16, 64, 128, [3000, 5, 700], [1, 1, 1]), (BF16, 64, 64, [3, 0, 900], [700, 1, 640]),
                                     (BF16, 200, 64, [20, 400], [3, 1]), (F32, 4, 64, [500, 20], [1, 2]),
                                     (F32, 4, 64, [k % 70 for k in range(200)], [1] * 200)):
        q, start, h, raw, c = attn_case(held, added, H, D, 70, 4, 32, dtype, 9)
        args = (q.to(DEV), start.to(DEV), h.to(DEV), dev(raw), dev(c), 70, 4, scale_of(D))
        want = hca.hca_cache_attn(*args, check=True)
        n = lib.hca_cache_attn_workspace_size(q.shape[0], len(held), H, D, 0 if dtype == BF16 else 1)
        ws = torch.full((n,), fill, dtype=torch.uint8, device=DEV)
        got = hca.hca_cache_attn(*args, ws=ws, check=True)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    for N in (40, 2000):
        x = torch.randn(N, 64, generator=torch.Generator().manual_seed(3)).to(BF16).to(DEV)
        slots = torch.randperm(-(-N // 16), generator=torch.Generator().manual_seed(4))
        slots = (slots[:, None] * 16 + torch.arange(16)).flatten()[:N].int().to(DEV)
        pools = []
        for ws in (None, torch.full((lib.hca_cache_append_workspace_size(200),), fill, dtype=torch.uint8, device=DEV)):
            pool, scale = torch.zeros(200, 16, 64, device=DEV).to(E4M3), torch.ones(200, device=DEV)
            hca.hca_cache_append(x, slots, pool, scale, ws=ws, check=True)
            pools.append((pool.view(torch.uint8), scale))
        assert torch.equal(pools[0][0], pools[1][0]) and torch.equal(pools[0][1], pools[1][1])
    for add in (3, 9000):
        plans = []
        for ws in (None, torch.full((lib.hca_cache_plan_workspace_size(2),), fill, dtype=torch.uint8, device=DEV)):
            table = torch.full((2, 700), -1, dtype=torch.int32, device=DEV)
            got = hca.hca_cache_plan(i32([0, 0]), i32([add, add]), table, i32(list(range(1400))), i32([1400]), 1400, 16, 2 * add + 5,
                                     ws=ws, check=True)
            plans.append([*got, table])
        for a, b in zip(*plans):
            assert torch.equal(a, b)


def test_threads_that_call_at_once():
    # host threads on streams of their own: the calls share nothing but the library
    import threading
    cases = []
    for seed, (H, D, dtype) in enumerate(((64, 128, BF16), (16, 64, BF16), (4, 64, F32))):
        q, start, h, raw, c = attn_case([900, 3, 77], [1, 2, 1], H, D, 64, 4, 16, dtype, seed)
        args = (q.to(DEV), start.to(DEV), h.to(DEV), dev(raw), dev(c), 64, 4, scale_of(D))
        cases.append((args, hca.hca_cache_attn(*args, check=True)))
    torch.cuda.synchronize()
    bad = []

    def work(args, want):
        try:
            with torch.cuda.stream(torch.cuda.Stream()):
                for _ in range(20):
                    out, lse = hca.hca_cache_attn(*args, check=True)
                    if not (torch.equal(out, want[0]) and torch.equal(lse, want[1])):
                        bad.append("differs")
        except Exception as e:  # noqa: BLE001
            bad.append(repr(e))

    ts = [threading.Thread(target=work, args=c) for c in cases for _ in range(2)]
    for t in ts:
        t.start()
    for t in ts:
        t.join(60)
    assert not bad, bad[:3]


def test_scores_of_great_magnitude():
    # up to 2^24 the order of the scores decides, and nothing overflows on the way
    H, D = 64, 128
    q, start, h, raw, c = attn_case([500, 40], [1, 2], H, D, 64, 4, 16, BF16, 12)
    for big in (2.0 ** 4, 2.0 ** 10, 2.0 ** 16):
        out, lse = hca.hca_cache_attn((q.float() * big).to(BF16).to(DEV), start.to(DEV), h.to(DEV), dev(raw), dev(c), 64, 4,
                                      scale_of(D), check=True)
        assert bool(torch.isfinite(out).all()) and bool(torch.isfinite(lse).all())
        assert float(lse.abs().max()) < 2.0 ** 24
        # every output is a mean of cache rows, none of which is beyond 448 times the largest scale
        assert float(out.float().abs().max()) <= 448 * float(max(raw[1].max(), c[1].max()))


def test_a_captured_prompt_step():
    # the kernels of long prompts, each set up while the one in front of it runs, in a graph
    R, H, D, W, m, bs, added = 2, 8, 64, 40, 8, 16, [2500, 2101]
    g = torch.Generator().manual_seed(6)
    n, e = sum(added), sum(a // m for a in added)
    xs, es = torch.randn(2, n, D, generator=g).to(BF16).to(DEV), torch.randn(2, e, D, generator=g).to(BF16).to(DEV)
    qs, add = torch.randn(2, n, H, D, generator=g).to(BF16).to(DEV), i32(added)

    def fresh():
        return Server(R, H, D, W, m, bs, BF16, max(added), max(added) + 1)

    def state(sv):
        return [sv.pool.view(torch.uint8), sv.scale, sv.raw_table, sv.comp_table, sv.count, sv.held]

    eager = []
    for k in range(2):
        sv = fresh()
        eager.append([t.clone() for t in (*sv.step(xs[k], es[k], qs[k], add), *state(sv))])
    sv = fresh()
    start = [t.clone() for t in state(sv)]
    x, ent, q = xs[0].clone(), es[0].clone(), qs[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        sv.step(x, ent, q, add)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse = sv.step(x, ent, q, add)
    for k in (0, 1, 1, 0):
        for t, s in zip(state(sv), start):
            t.copy_(s)
        x.copy_(xs[k]); ent.copy_(es[k]); q.copy_(qs[k])
        graph.replay()
        for a, b in zip((out, lse, *state(sv)), eager[k]):
            assert torch.equal(a, b), k
