"""Attention over the cache for requests with common prefixes, against the fp64
oracle, which attends every request's own table."""
import numpy as np
import pytest
import torch

from _cache import E4M3, attn_case, check_attn, scale_of
from block_sparse_compressed_gb300 import hca

pytestmark = pytest.mark.gpu
DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32
E_CACHE = 12


@pytest.fixture(autouse=True)
def apart():
    """The common entries are attended apart however few they are; the argument of the
    function is another HCA_INJECT_SHARED_PATH."""
    hca.hca_test_inject(hca.INJECT_SHARED_PATH, 1)
    yield lambda v: hca.hca_test_inject(hca.INJECT_SHARED_PATH, v)
    hca.hca_test_inject(hca.INJECT_RESET)


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


def dev(c):
    return tuple(t.to(DEV) for t in c)


def shared_case(prefixes, behind, added, H, D, W, m, bs, dtype, seed, pad=0, qscale=1.0):
    """CPU inputs of a call: prefixes is a list of (requests, common columns), behind
    the tokens that each request holds behind its prefix."""
    cols = [c for n, c in prefixes for _ in range(n)]
    held = [c * bs * m + b for c, b in zip(cols, behind)]
    q, start, h, raw, comp = attn_case(held, added, H, D, W, m, bs, dtype, seed, pad=pad, qscale=qscale)
    table = comp[2]
    r = 0
    for n, c in prefixes:
        if n:
            table[r:r + n, :c] = table[r, :c].clone()
        r += n
    first = np.concatenate([[0], np.cumsum([n for n, _ in prefixes])]).tolist()
    return (q, start, h, raw, comp), i32(first), i32([c for _, c in prefixes])


def call(case, first, cols, W, m, check=True, **k):
    q, start, held, raw, comp = case
    return hca.hca_cache_attn_shared(q.to(DEV), start.to(DEV), held.to(DEV), dev(raw), dev(comp), first, cols, W, m, scale_of(q.shape[2]),
                                     check=check, **k)


CASES = [  # prefixes, tokens behind them, new tokens, H, D, W, m, bs
    ([(1, 1)], [0], [1], 1, 64, 16, 1, 16),
    ([(3, 2)], [0, 5, 63], [1, 1, 1], 8, 128, 32, 4, 16),
    ([(2, 3), (1, 0), (4, 1)], [0, 3, 40, 1, 7, 0, 100], [1] * 7, 64, 128, 128, 4, 32),
    ([(2, 9), (3, 5)], [10, 0, 33, 2, 64], [3, 1, 4, 2, 5], 16, 64, 64, 4, 64),
    ([(5, 7)], [0, 1, 2, 3, 1000], [1, 0, 2, 0, 1], 5, 128, 16, 2, 128),
    ([(2, 40)], [0, 17], [40, 23], 64, 128, 128, 2, 16),       # chunks: many row tiles
    ([(9, 33)], list(range(9)), [1] * 9, 32, 128, 8, 1, 16),    # 288 rows, units cut between CTAs
    ([(1, 0), (1, 0)], [5, 900], [1, 3], 24, 64, 64, 4, 16),    # nothing shared
    ([(2, 1), (0, 3), (1, 2)], [50, 0, 9], [2, 1, 1], 130, 64, 33, 3, 16),
]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("prefixes,behind,added,H,D,W,m,bs", CASES)
def test_matches_oracle(prefixes, behind, added, H, D, W, m, bs, dtype):
    case, first, cols = shared_case(prefixes, behind, added, H, D, W, m, bs, dtype, 3)
    check_attn(call(case, first, cols, W, m), *case, W, m, scale_of(D), dtype)


@pytest.mark.parametrize("path", [0, 2])
@pytest.mark.parametrize("prefixes,behind,added,H,D,W,m,bs", CASES[2:5])
def test_other_ways(prefixes, behind, added, H, D, W, m, bs, path, apart):
    apart(path)
    case, first, cols = shared_case(prefixes, behind, added, H, D, W, m, bs, BF16, 3)
    check_attn(call(case, first, cols, W, m), *case, W, m, scale_of(D), BF16)
    out, lse = call(case, first, cols + 1000, W, m, check=False)
    assert bool(out.isnan().all()) and bool(lse.isnan().all())


def test_the_way_is_picked_by_the_sizes(apart):
    """Both ways of the default, told apart by what the calls launch."""
    apart(0)
    hca.hca_profile_enable(True)
    try:
        case, first, cols = shared_case([(40, 512)], [0] * 40, [1] * 40, 8, 64, 16, 1, 16, BF16, 21)
        check_attn(call(case, first, cols, 16, 1), *case, 16, 1, scale_of(64), BF16)
        assert hca.hca_profile_read()["hca_cache_prefix"][0] == 1
        case, first, cols = shared_case([(2, 3)], [0, 1], [1, 1], 8, 64, 16, 1, 16, BF16, 22)
        check_attn(call(case, first, cols, 16, 1), *case, 16, 1, scale_of(64), BF16)
        assert hca.hca_profile_read()["hca_cache_prefix"][0] == 1
    finally:
        hca.hca_profile_enable(False)


@pytest.mark.parametrize("dtype", [BF16, F32])
def test_without_tokens(dtype):
    case, first, cols = shared_case([(2, 3)], [4, 7], [0, 0], 8, 64, 16, 4, 16, dtype, 4)
    out, lse = call(case, first, cols, 16, 4)
    assert out.shape == (0, 8, 64) and lse.shape == (0, 8)
    # room for tokens, but none of them there
    case, first, cols = shared_case([(2, 3)], [4, 7], [0, 0], 8, 64, 16, 4, 16, dtype, 4, pad=3)
    out, lse = torch.full((3, 8, 64), 2.0, dtype=dtype, device=DEV), torch.full((3, 8), 2.0, device=DEV)
    call(case, first, cols, 16, 4, out=out, lse=lse)
    assert bool((out == 2).all()) and bool((lse == 2).all())


@pytest.mark.parametrize("bs", [16, 32, 64, 128])
@pytest.mark.parametrize("D", [64, 128])
def test_every_block_size_and_odd_ends(D, bs):
    """Prefixes that end inside a tile of keys, rows that end inside a tile of rows."""
    for pages in (1, 128 // bs, 128 // bs + 1, 300 // bs):
        case, first, cols = shared_case([(3, pages)], [0, 20, 130], [1, 2, 1], 33, D, 64, 1, bs, BF16, pages + bs)
        check_attn(call(case, first, cols, 64, 1), *case, 64, 1, scale_of(D), BF16)


@pytest.mark.parametrize("qscale", [0.0, 1e-30, 30.0, 1e4])
def test_scores_of_any_size(qscale):
    case, first, cols = shared_case([(4, 20)], [0, 50, 100, 3], [1] * 4, 64, 128, 64, 1, 16, BF16, 5, qscale=qscale)
    check_attn(call(case, first, cols, 64, 1), *case, 64, 1, scale_of(128), BF16)


@pytest.mark.parametrize("D", [64, 128])
def test_scores_that_rise_along_the_prefix(D):
    """Every later page beats the reference, so O follows again and again."""
    case, first, cols = shared_case([(3, 24)], [0, 9, 40], [1, 2, 1], 40, D, 16, 1, 16, BF16, 6, qscale=2.0)
    pool, scale, table = case[4]
    q = case[0]
    q.copy_(q.abs())  # all scores positive, growing with the scales
    pool.copy_(pool.float().abs().to(E4M3))
    for page in range(24):
        scale[table[0, page]] = 2.0 ** (page / 2 - 9) if page % 2 == 0 else 2.0 ** ((page - 1) / 2 - 9)
    check_attn(call(case, first, cols, 16, 1), *case, 16, 1, scale_of(D), BF16)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("what", ["far", "odd", "tiny"])
def test_block_scales(what, D):
    case, first, cols = shared_case([(3, 30), (2, 11)], [0, 9, 40, 5, 5], [1, 2, 1, 1, 1], 40, D, 16, 1, 16, BF16, 7)
    scale = case[4][1]
    g = torch.Generator().manual_seed(8)
    if what == "far":      # beyond 2^-15 of the largest
        scale.copy_(torch.exp2(torch.randint(-40, -4, scale.shape, generator=g).float()))
    elif what == "odd":    # no powers of two
        scale.mul_(1 + torch.rand(scale.shape, generator=g))
    else:
        scale.fill_(2.0 ** -96)
    check_attn(call(case, first, cols, 16, 1), *case, 16, 1, scale_of(D), BF16)


def test_where_nothing_is_shared(apart):
    """Each request's own is then all there is; attended with it (2) it is the call without prefixes, bit for bit."""
    case, first, cols = shared_case([(6, 0)], [5, 900, 3, 77, 128, 4000], [1, 3, 1, 0, 2, 1], 64, 128, 64, 4, 32, BF16, 9)
    q, start, held, raw, comp = case
    want = hca.hca_cache_attn(q.to(DEV), start.to(DEV), held.to(DEV), dev(raw), dev(comp), 64, 4, scale_of(128))
    check_attn(call(case, first, cols, 64, 4), *case, 64, 4, scale_of(128), BF16)
    apart(2)
    got = call(case, first, cols, 64, 4)
    assert torch.equal(want[0], got[0]) and torch.equal(want[1], got[1])
    none = call(case, i32([0]), i32([]), 64, 4)
    assert torch.equal(want[0], none[0]) and torch.equal(want[1], none[1])


def test_rows_behind_the_last_token_are_left():
    case, first, cols = shared_case([(2, 3)], [4, 7], [1, 2], 8, 64, 16, 4, 16, BF16, 10, pad=5)
    out, lse = torch.full((8, 8, 64), 3.0, dtype=BF16, device=DEV), torch.full((8, 8), 3.0, device=DEV)
    call(case, first, cols, 16, 4, out=out, lse=lse)
    assert bool((out[3:] == 3).all()) and bool((lse[3:] == 3).all())
    check_attn((out[:3], lse[:3]), case[0][:3], *case[1:], 16, 4, scale_of(64), BF16)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("change", [
    dict(first=[0, 3, 5]), dict(first=[1, 2, 4]), dict(first=[0, 5, 4]), dict(first=[0, -1, 4]), dict(first=[0, 2, 3]),
    dict(cols=[-1, 1]), dict(cols=[1000, 1]), dict(cols=[2 ** 31 - 1, 1]), dict(cols=[4, 1]), dict(cols=[3, 2]), dict(held=1),
    dict(start=[0, 1, 0, 3, 4]), dict(start=[0, 1, 2, 3, 99]), dict(start=[-4, 1, 2, 3, 4])])
def test_values_that_do_not_fit_are_refused(change, dtype):
    case, first, cols = shared_case([(2, 3), (2, 1)], [4, 7, 2, 5], [1] * 4, 8, 64, 16, 4, 16, dtype, 11)
    q, start, held, raw, comp = case
    if "first" in change:
        first = i32(change["first"])
    if "cols" in change:
        cols = i32(change["cols"])
    if "held" in change:
        held = held.clone()
        held[0] = 3 * 16 * 4 - 2  # one token short of the prefix
    if "start" in change:
        start = torch.tensor(change["start"], dtype=torch.int32)
    ws = torch.empty(hca.load().hca_cache_attn_shared_workspace_size(4, 4, 8, 64, 2, 1 if dtype == F32 else 0), dtype=torch.uint8, device=DEV)
    out, lse = call((q, start, held, raw, comp), first, cols, 16, 4, check=False, ws=ws)
    assert hca.hca_workspace_status(ws) == E_CACHE
    assert bool(out.isnan().all()) and bool(lse.isnan().all())
    good = call(case, *[i32(v) for v in ([0, 2, 4], [3, 1])], 16, 4)  # the next call is an ordinary one
    check_attn(good, *case, 16, 4, scale_of(64), dtype)


@pytest.mark.parametrize("bad", ["id", "scale"])
def test_a_bad_common_block_reaches_its_prefix_only(bad):
    case, first, cols = shared_case([(2, 6), (2, 4)], [4, 7, 2, 5], [1] * 4, 8, 64, 16, 4, 16, BF16, 12)
    want = call(case, first, cols, 16, 4)
    comp = case[4]
    if bad == "id":
        comp[2][0:2, 3] = len(comp[0])
    else:
        comp[1][comp[2][0, 3]] = 0.0
    ws = torch.empty(hca.load().hca_cache_attn_shared_workspace_size(4, 4, 8, 64, 2, 0), dtype=torch.uint8, device=DEV)
    out, lse = call(case, first, cols, 16, 4, check=False, ws=ws)
    assert hca.hca_workspace_status(ws) == E_CACHE
    assert bool(out[:2].isnan().all()) and bool(lse[:2].isnan().all())
    assert torch.equal(out[2:], want[0][2:])


def test_nan_in_the_cache_and_in_queries():
    case, first, cols = shared_case([(2, 6), (2, 4)], [4, 7, 2, 5], [1] * 4, 8, 64, 16, 4, 16, BF16, 13)
    want = call(case, first, cols, 16, 4)
    case[0][1, 3, 5] = float("nan")
    out, _ = call(case, first, cols, 16, 4)
    assert bool(out[1, 3].isnan().all())
    keep = torch.ones(4, 8, dtype=torch.bool, device=DEV)
    keep[1, 3] = False
    assert torch.equal(out[keep], want[0][keep])
    pool, _, table = case[4]
    pool.view(torch.uint8)[table[2, 1], 5, 7] = 0x7F  # seen by the second prefix's requests
    out, _ = call(case, first, cols, 16, 4)
    assert bool(out[2:].isnan().all()) and torch.equal(out[0], want[0][0])


def test_same_bits_twice_and_captured():
    case, first, cols = shared_case([(20, 37), (11, 9)], [(37 * r) % 300 for r in range(31)], [1 + r % 3 for r in range(31)], 64, 128, 128, 4,
                                    16, BF16, 14)
    q, start, held, raw, comp = case[0].to(DEV), case[1].to(DEV), case[2].to(DEV), dev(case[3]), dev(case[4])
    args = (q, start, held, raw, comp, first, cols, 128, 4, scale_of(128))
    a = hca.hca_cache_attn_shared(*args)
    b = hca.hca_cache_attn_shared(*args)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    check_attn(a, *case, 128, 4, scale_of(128), BF16)
    ws = torch.empty(hca.load().hca_cache_attn_shared_workspace_size(q.shape[0], 31, 64, 128, 2, 0), dtype=torch.uint8, device=DEV)
    graphs = []
    for _ in range(2):  # two graphs that share a workspace
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = hca.hca_cache_attn_shared(*args, ws=ws)
        graphs.append((g, out))
    q.mul_(0.5)
    ws.fill_(255)
    want = hca.hca_cache_attn_shared(*args)
    for g, out in graphs:
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out[0], want[0]) and torch.equal(out[1], want[1])


def test_other_streams_at_once():
    case, first, cols = shared_case([(9, 33)], list(range(9)), [1] * 9, 32, 128, 8, 1, 16, BF16, 15)
    args = (case[0].to(DEV), case[1].to(DEV), case[2].to(DEV), dev(case[3]), dev(case[4]), first, cols, 8, 1, scale_of(128))
    want = hca.hca_cache_attn_shared(*args)
    torch.cuda.synchronize()
    streams, outs = [torch.cuda.Stream() for _ in range(3)], []
    for _ in range(10):
        for s in streams:
            with torch.cuda.stream(s):
                outs.append(hca.hca_cache_attn_shared(*args))
    torch.cuda.synchronize()
    assert all(torch.equal(o[0], want[0]) for o in outs)


def test_many_prefixes_and_requests():
    """As many prefixes as are allowed, more requests than threads."""
    rng = np.random.default_rng(16)
    prefixes = [(int(n), int(c)) for n, c in zip(rng.integers(0, 4, 256), rng.integers(0, 4, 256))]
    R = sum(n for n, _ in prefixes)
    case, first, cols = shared_case(prefixes, rng.integers(0, 50, R).tolist(), [1] * R, 4, 64, 16, 2, 16, BF16, 17)
    check_attn(call(case, first, cols, 16, 2), *case, 16, 2, scale_of(64), BF16)
    with pytest.raises(hca.HCAError):
        call(case, i32([0] * 257 + [R]), i32([0] * 257), 16, 2)


def test_long_prefix_of_many_rows():
    """A prefix of 6,000 entries for 96 tokens of 3 requests, in all SMs."""
    case, first, cols = shared_case([(3, 375)], [0, 1, 2], [30, 33, 33], 16, 128, 16, 1, 16, BF16, 18)
    check_attn(call(case, first, cols, 16, 1), *case, 16, 1, scale_of(128), BF16)


@pytest.mark.parametrize("D", [64, 128])
def test_more_row_tiles_than_blocks(D):
    """Most row tiles are finished by the block that has them, some are cut, one prefix
    has no common entries."""
    case, first, cols = shared_case([(2, 5), (1, 0), (1, 9)], [0, 30, 17, 5], [101, 97, 50, 73], 128, D, 16, 1, 32, BF16, 20, pad=3)
    out, lse = torch.full((324, 128, D), 4.0, dtype=BF16, device=DEV), torch.full((324, 128), 4.0, device=DEV)
    call(case, first, cols, 16, 1, out=out, lse=lse)
    assert bool((out[321:] == 4).all()) and bool((lse[321:] == 4).all())
    check_attn((out[:321], lse[:321]), case[0][:321], *case[1:], 16, 1, scale_of(D), BF16)
    again = call(case, first, cols, 16, 1)
    assert torch.equal(again[0][:321], out[:321]) and torch.equal(again[1][:321], lse[:321])
    # refused: all rows
    out, lse = call(case, first, cols + 1, 16, 1, check=False)
    assert bool(out.isnan().all()) and bool(lse.isnan().all())
    # a bad block reaches its prefix only
    case[4][2][3, 4] = -7
    bad, _ = call(case, first, cols, 16, 1, check=False)
    assert bool(bad[248:321].isnan().all()) and torch.equal(bad[:248], again[0][:248])


@pytest.mark.parametrize("path", [1, 2])
def test_requests_without_tokens_need_no_table(path, apart):
    """A batch of fixed size: places that are not taken, before, between and behind the others."""
    apart(path)
    case, first, cols = shared_case([(4, 5), (3, 9), (2, 2)], [3, 0, 6, 0, 0, 40, 0, 0, 0], [0, 1, 2, 0, 0, 1, 0, 0, 0], 16, 64, 16, 1, 16, BF16, 25)
    want = call(case, first, cols, 16, 1)
    check_attn(want, *case, 16, 1, scale_of(64), BF16)
    q, start, held, raw, comp = case
    for r in (0, 3, 4, 6, 7, 8):
        raw[2][r], comp[2][r], held[r] = -1, -1, 0
    got = call(case, first, cols, 16, 1)
    assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_few_rows_over_a_long_prefix():
    """A row tile in as many parts as the join takes."""
    case, first, cols = shared_case([(2, 300)], [5, 40], [1, 1], 8, 64, 16, 1, 64, BF16, 23)
    check_attn(call(case, first, cols, 16, 1), *case, 16, 1, scale_of(64), BF16)


def test_more_parts_than_lanes():
    """The prefix in 65 parts and a request's own keys in more than 16, which the join's lanes
    take in turns."""
    case, first, cols = shared_case([(2, 520)], [6000, 3], [1, 2], 8, 64, 16, 1, 128, BF16, 26)
    check_attn(call(case, first, cols, 16, 1), *case, 16, 1, scale_of(64), BF16)


@pytest.mark.parametrize("H,D,added", [(64, 128, [70, 61]), (96, 64, [70, 61]), (64, 128, [31, 20]), (20, 128, [31, 20])])
def test_numbers_of_rows_between(H, D, added):
    """Joins of their own launch, of some and of few rows."""
    case, first, cols = shared_case([(2, 37)], [9, 500], added, H, D, 40, 1, 16, BF16, 27)
    check_attn(call(case, first, cols, 40, 1), *case, 40, 1, scale_of(D), BF16)


def test_both_ways_of_the_binding_give_the_same(monkeypatch):
    case, first, cols = shared_case([(2, 3), (1, 2)], [4, 7, 9], [1, 2, 1], 8, 64, 16, 4, 16, BF16, 24)
    a = call(case, first, cols, 16, 4)
    if hca._py is None:
        pytest.skip("built without the headers of Python or torch")
    monkeypatch.setattr(hca, "_py", None)
    b = call(case, first, cols, 16, 4)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    with pytest.raises(ValueError):
        hca.hca_cache_attn_shared(case[0].to(DEV), case[1].to(DEV), case[2].to(DEV), dev(case[3]), None, first, cols, 16, 4, 0.1)
    with pytest.raises(ValueError):
        call(case, first[:-1], cols, 16, 4)
    with pytest.raises(TypeError):
        call(case, first, cols.long(), 16, 4)


def test_a_stalled_wait_times_out():
    case, first, cols = shared_case([(3, 12)], [0, 1, 2], [1, 2, 1], 16, 128, 16, 1, 16, BF16, 19)
    ws = torch.empty(hca.load().hca_cache_attn_shared_workspace_size(4, 3, 16, 128, 1, 0), dtype=torch.uint8, device=DEV)
    try:
        hca.hca_test_inject(hca.INJECT_WAIT_LIMIT_NS, 2_000_000)
        hca.hca_test_inject(hca.INJECT_STALL, 1)
        out, lse = call(case, first, cols, 16, 1, check=False, ws=ws)
        assert hca.hca_workspace_status(ws) == 10
        assert bool(out.isnan().all()) and bool(lse.isnan().all())
    finally:
        hca.hca_test_inject(hca.INJECT_RESET)
        hca.hca_test_inject(hca.INJECT_SHARED_PATH, 1)
    check_attn(call(case, first, cols, 16, 1, ws=ws), *case, 16, 1, scale_of(128), BF16)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("tokens", [100, 200])
@pytest.mark.parametrize("limit", [1, 5000])
def test_waits_that_give_up_before_the_first_pages(limit, tokens, D):
    """A CTA's part of the prefix is some 2,700 pages, whose scales are all looked at before
    the first page is handed on: the waits for it end first.  100 and 200 tokens of 2 requests:
    beside the own keys, and behind them."""
    case, first, cols = shared_case([(2, 4096)], [1, 2], [tokens, tokens], 128, D, 16, 1, 16, BF16, 28)
    args = tuple(t.to(DEV) for t in case[:3]) + (dev(case[3]), dev(case[4]), first, cols, 16, 1, scale_of(D))
    ws = torch.empty(hca.load().hca_cache_attn_shared_workspace_size(2 * tokens, 2, 128, D, 1, 0), dtype=torch.uint8, device=DEV)
    want = hca.hca_cache_attn_shared(*args, ws=ws, check=True)
    try:
        hca.hca_test_inject(hca.INJECT_WAIT_LIMIT_NS, limit)
        out, lse = hca.hca_cache_attn_shared(*args, ws=ws)
        assert hca.hca_workspace_status(ws) == 10
        assert bool(out.isnan().all()) and bool(lse.isnan().all())
    finally:
        hca.hca_test_inject(hca.INJECT_WAIT_LIMIT_NS, 0)
    again = hca.hca_cache_attn_shared(*args, ws=ws, check=True)
    assert torch.equal(again[0], want[0]) and torch.equal(again[1], want[1])


@pytest.mark.parametrize("prefixes,launches", [([(1, 512)] * 40, 0), ([(10, 512)] * 4, 1)])
def test_the_way_is_picked_by_the_prefixes(prefixes, launches, apart):
    """40 tokens over 64 key tiles: one row tile each where every request has a prefix of its
    own, which is slower apart (55 us for 30), and a row tile for every ten of them."""
    apart(0)
    hca.hca_profile_enable(True)
    try:
        case, first, cols = shared_case(prefixes, [0] * 40, [1] * 40, 8, 64, 16, 1, 16, BF16, 29)
        check_attn(call(case, first, cols, 16, 1), *case, 16, 1, scale_of(64), BF16)
        assert hca.hca_profile_read().get("hca_cache_prefix", (0,))[0] == launches
    finally:
        hca.hca_profile_enable(False)


def test_many_places_that_are_not_taken():
    """20,000 requests without tokens in front of a prefix's others take no longer than behind
    them (21 us): one after the other a load for each is 1.2 ms."""
    case, first, cols = shared_case([(4, 40)], [0, 3, 40, 9], [1, 2, 1, 1], 16, 64, 16, 1, 16, BF16, 30)
    q, start, held, raw, comp = case
    n = 20000
    none = torch.zeros(n, dtype=torch.int32)
    times = []
    for front in (False, True):
        join = lambda a, b: torch.cat([b, a] if front else [a, b])  # noqa: E731
        big = (q, join(start, none if front else none + start[-1]), join(held, none),
               *((c[0], c[1], join(c[2], torch.full((n, c[2].shape[1]), -1, dtype=torch.int32))) for c in (raw, comp)))
        took = []
        for _ in range(6):
            hca.hca_profile_enable(True)
            try:
                got = call(big, i32([0, n + 4]), cols, 16, 1)
                took.append(hca.hca_profile_read()["hca_cache_prefix"][1])
            finally:
                hca.hca_profile_enable(False)
        times.append(min(took))
        check_attn(got, *case, 16, 1, scale_of(64), BF16)
    assert times[1] < 5 * times[0], times
