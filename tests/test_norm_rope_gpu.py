"""Norms with positions and the rotation alone against the fp64 oracle."""
import ctypes

import numpy as np
import pytest
import torch

from block_sparse_compressed_gb300 import hca
from oracle import norm_rope as ON

pytestmark = pytest.mark.gpu
BF16, F32 = torch.bfloat16, torch.float32
EPS = 1e-6


def f64(t):
    return t.detach().float().cpu().double().numpy()


def close(name, got, ref, tol, dtype):
    """One rounding to the type on top of the arithmetic's bound."""
    got = f64(got)
    tol = torch.finfo(dtype).eps / 2 * (np.abs(ref) + tol) + tol
    assert got.shape == ref.shape, (name, got.shape, ref.shape)
    bad = np.argwhere(~(np.abs(got - ref) <= tol))
    assert not len(bad), f"{name}: {len(bad)} of {got.size} off, first {bad[0].tolist()}: {got[tuple(bad[0])]} for {ref[tuple(bad[0])]}"


def make(B, H, S, D, rot, dtype, seed, axes=1, weight=True, token_major=True, far=1000):
    g = torch.Generator().manual_seed(seed)
    rnd = lambda *s: torch.randn(*s, generator=g)  # noqa: E731
    q = (rnd(B, S, H, D) * torch.exp2(rnd(H, 1))).to(dtype).cuda().transpose(1, 2)
    if not token_major:
        q = q.contiguous()
    kv = rnd(B, S, D).to(dtype).cuda()
    w = [(1 + 0.3 * rnd(D)).cuda() if weight else None for _ in range(2)]
    pos = torch.randint(-far, far, (axes, B, S), generator=g, dtype=torch.int32).cuda()
    freq = (rnd(axes, rot // 2).abs() ** 3).cuda()
    dq, dkv = rnd(B, H, S, D).to(dtype).cuda(), rnd(B, S, D).to(dtype).cuda()
    return q, kv, w[0], w[1], pos, freq, dq, dkv


def host(w):
    return None if w is None else w.cpu().double().numpy()


def check_fwd(x, w, theta, first, halves, got, name, eps=EPS):
    x, w = f64(x), host(w)
    close(name, got, ON.forward(x, w, eps, theta, first, halves), ON.forward_bound(x, w, eps, theta, first, halves), got.dtype)


def check_bwd(x, w, theta, first, halves, g, dx, dw, name):
    x, w, g = f64(x), host(w), f64(g)
    rdx, rdw = ON.backward(x, w, EPS, theta, first, halves, g)
    tdx, tdw = ON.backward_bound(x, w, EPS, theta, first, halves, g)
    close("d" + name, dx, rdx, tdx, dx.dtype)
    if w is None:
        assert dw is None
    else:
        close("dw" + name, dw, rdw, tdw, F32)


SHAPES = [  # B, H, S, D, rot, first, halves, axes, weight
    (1, 1, 1, 64, 64, 0, False, 1, True), (2, 3, 17, 64, 32, 32, False, 1, True), (1, 64, 5, 128, 64, 64, False, 1, True),
    (2, 5, 33, 128, 128, 0, True, 2, False), (1, 2, 70, 72, 48, 16, True, 3, True), (3, 7, 9, 8, 8, 0, False, 1, True),
    (1, 4, 19, 200, 40, 96, False, 4, True), (2, 1, 31, 256, 256, 0, True, 1, True), (1, 3, 11, 512, 512, 0, True, 1, False),
    (1, 3, 11, 512, 64, 448, False, 1, True), (1, 2, 6, 392, 272, 64, True, 2, True), (2, 2, 4, 16, 0, 0, False, 1, True),
    (1, 130, 3, 32, 16, 8, True, 1, True), (5, 1, 1, 128, 64, 0, False, 1, False)]


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", SHAPES)
def test_forward_and_backward(shape, dtype):
    B, H, S, D, rot, first, halves, axes, weight = shape
    q, kv, wq, wkv, pos, freq, dq, dkv = make(B, H, S, D, rot, dtype, 1, axes, weight, token_major=S % 2 == 1)
    th = ON.angles(pos.cpu().numpy(), freq.cpu().numpy())
    kw = dict(first=first, halves=halves)
    qo, kvo = hca.hca_norm_rope_fwd(q, kv, wq, wkv, pos, freq, EPS, **kw)
    assert qo.is_contiguous() and kvo.is_contiguous()
    check_fwd(q, wq, th[:, None], first, halves, qo, "q")
    check_fwd(kv, wkv, th, first, halves, kvo, "kv")
    gq, gkv, gwq, gwkv = hca.hca_norm_rope_bwd(q, kv, wq, wkv, pos, freq, EPS, dq, dkv, **kw)
    assert gq.stride() == q.stride() or q.numel() == 0 or min(q.shape) == 1
    check_bwd(q, wq, th[:, None], first, halves, dq, gq, gwq, "q")
    check_bwd(kv, wkv, th, first, halves, dkv, gkv, gwkv, "kv")
    again = hca.hca_norm_rope_bwd(q, kv, wq, wkv, pos, freq, EPS, dq, dkv, **kw)
    for a, b in zip((gq, gkv, gwq, gwkv), again):
        assert a is None or torch.equal(a, b)


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("shape", SHAPES)
def test_rotation_alone(shape, dtype):
    B, H, S, D, rot, first, halves, axes, _ = shape
    x, _, _, _, pos, freq, _, _ = make(B, H, S, D, rot, dtype, 2, axes)
    th = ON.angles(pos.cpu().numpy(), freq.cpu().numpy())[:, None]
    for inverse in (False, True):
        y = hca.hca_rope(x, pos, freq, inverse=inverse, first=first, halves=halves)
        t = -th if inverse else th
        close("y", y, ON.rotate(f64(x), t, first, halves), ON.rotate_bound(f64(x), t, first, halves), dtype)
    # columns that do not turn keep their bits
    u, v = ON.columns(rot // 2, first, halves)
    still = np.setdiff1d(np.arange(D), np.concatenate([u, v]))
    assert torch.equal(y[..., still], x[..., still])


def test_far_positions_and_fast_frequencies():
    pos = torch.tensor([[[0, 1, -1, 2 ** 31 - 1, -2 ** 31, 123456789, 10 ** 6]]], dtype=torch.int32).cuda()
    freq = torch.tensor([[1.0, 6.2831855, 3.0e-5, 1e4, 0.0, 1e-9, 77.7, 4.0e9]]).cuda()
    x = torch.randn(1, 2, 7, 16, generator=torch.Generator().manual_seed(3)).cuda()
    th = ON.angles(pos.cpu().numpy(), freq.cpu().numpy())[:, None]
    for halves in (False, True):
        y = hca.hca_rope(x, pos, freq, halves=halves)
        close("y", y, ON.rotate(f64(x), th, 0, halves), ON.rotate_bound(f64(x), th, 0, halves), F32)


def test_default_positions_columns_and_single_tensors():
    q, kv, wq, wkv, _, freq, dq, dkv = make(2, 4, 23, 64, 32, BF16, 4)
    pos = torch.arange(23, dtype=torch.int32).repeat(2, 1).cuda()
    a = hca.hca_norm_rope_fwd(q, kv, wq, wkv, None, freq[0], EPS)
    b = hca.hca_norm_rope_fwd(q, kv, wq, wkv, pos, freq, EPS, first=32)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    assert torch.equal(hca.hca_norm_rope_fwd(q, None, wq, None, pos, freq, EPS)[0], a[0])
    only = hca.hca_norm_rope_fwd(None, kv, None, wkv, pos, freq, EPS)
    assert only[0] is None and torch.equal(only[1], a[1])
    full = hca.hca_norm_rope_bwd(q, kv, wq, wkv, pos, freq, EPS, dq, dkv)
    one = hca.hca_norm_rope_bwd(None, kv, None, wkv, pos, freq, EPS, None, dkv)
    assert one[0] is None and one[2] is None and torch.equal(one[1], full[1])
    close("dwkv", one[3], f64(full[3]), 2.0 ** -20 * np.abs(f64(full[3])) + 1e-4, F32)


def test_strides():
    g = torch.Generator().manual_seed(5)
    base = torch.randn(2, 9, 5, 3, 72, generator=g).to(BF16).cuda()
    freq = torch.rand(1, 16, generator=g).cuda()
    q = base[:, :, 1:4, 1, 8:72].transpose(1, 2)  # [2, 3, 9, 64], columns in the middle of wider rows
    assert q.data_ptr() % 16 == 0
    want = hca.hca_norm_rope_fwd(q.contiguous(), None, None, None, None, freq, EPS)[0]
    assert torch.equal(hca.hca_norm_rope_fwd(q, None, None, None, None, freq, EPS)[0], want)
    # a broadcast input: one row for all heads
    x = torch.randn(2, 1, 9, 64, generator=g).to(BF16).cuda().expand(2, 3, 9, 64)
    want = hca.hca_norm_rope_fwd(x.contiguous(), None, None, None, None, freq, EPS)[0]
    assert torch.equal(hca.hca_norm_rope_fwd(x, None, None, None, None, freq, EPS)[0], want)
    dq = hca.hca_norm_rope_bwd(x, None, None, None, None, freq, EPS, want, None)[0]
    assert dq.is_contiguous()
    assert torch.equal(dq, hca.hca_norm_rope_bwd(x.contiguous(), None, None, None, None, freq, EPS, want, None)[0])
    # results between other data
    out = torch.full((2, 9, 4, 64), 7.0, dtype=BF16, device="cuda")
    y = hca.hca_rope(q, None, freq, y=out[:, :, :3].transpose(1, 2))
    assert torch.equal(y, hca.hca_rope(q.contiguous(), None, freq)) and bool((out[:, :, 3] == 7).all())
    with pytest.raises(hca.HCAError) as e:  # rows of the result over one another
        hca.hca_rope(q, None, freq, y=torch.empty(2, 1, 9, 64, dtype=BF16, device="cuda").expand(2, 3, 9, 64))
    assert e.value.status == 5
    with pytest.raises(hca.HCAError) as e:  # 8 bytes beside a 16-byte boundary
        hca.hca_rope(base.flatten()[4:4 + 9 * 64].view(1, 1, 9, 64), None, freq)
    assert e.value.status == 4
    with pytest.raises(ValueError):
        hca.hca_rope(q.transpose(2, 3), None, freq)


def test_in_place_and_back():
    x = torch.randn(2, 3, 40, 128, generator=torch.Generator().manual_seed(6)).cuda()
    freq = torch.rand(2, 32, generator=torch.Generator().manual_seed(7)).cuda()
    pos = torch.randint(0, 5000, (2, 2, 40), dtype=torch.int32).cuda()
    keep = x.clone()
    want = hca.hca_rope(x, pos, freq)
    assert hca.hca_rope(x, pos, freq, y=x) is x and torch.equal(x, want)
    hca.hca_rope(x, pos, freq, inverse=True, y=x)
    th = ON.angles(pos.cpu().numpy(), freq.cpu().numpy())[:, None]
    b = ON.rotate_bound(f64(keep), th, 64, False)
    close("x", x, f64(keep), 4 * b, F32)
    q = keep.clone()
    want = hca.hca_norm_rope_fwd(q, None, None, None, pos, freq, EPS)[0]
    assert torch.equal(hca.hca_norm_rope_fwd(q, None, None, None, pos, freq, EPS, qo=q)[0], want)
    g = torch.randn_like(keep)
    want = hca.hca_norm_rope_bwd(keep, None, None, None, pos, freq, EPS, g, None)[0]
    assert torch.equal(hca.hca_norm_rope_bwd(keep, None, None, None, pos, freq, EPS, g, None, dq=g)[0], want)


def test_rows_keep_to_themselves():
    q, kv, wq, wkv, pos, freq, dq, dkv = make(1, 4, 50, 128, 64, F32, 8)
    q = q.contiguous()
    clean = hca.hca_norm_rope_fwd(q, kv, wq, wkv, pos, freq, EPS)[0]
    q[0, 1, 7, 3], q[0, 2, 9, 100] = float("nan"), float("inf")
    got = hca.hca_norm_rope_fwd(q, kv, wq, wkv, pos, freq, EPS)[0]
    bad = torch.zeros(1, 4, 50, dtype=torch.bool, device="cuda")
    bad[0, 1, 7] = bad[0, 2, 9] = True
    assert torch.equal(got[~bad], clean[~bad])
    assert bool(got[0, 1, 7].isnan().all()) and bool(got[0, 2, 9, 100].isnan())
    # a row of zeros is a row of zeros; without eps it is 0 / 0
    q[0, 3, 3] = 0
    assert bool((hca.hca_norm_rope_fwd(q, kv, wq, wkv, pos, freq, EPS)[0][0, 3, 3] == 0).all())
    zero = hca.hca_norm_rope_fwd(q, kv, wq, wkv, pos, freq, 0.0)[0]
    assert bool(zero[0, 3, 3].isnan().all()) and bool(zero[0, 0].isfinite().all())
    # the rotation passes infinities of still columns through
    x = torch.ones(1, 1, 2, 128, device="cuda")
    x[0, 0, 0, 5] = float("inf")
    y = hca.hca_rope(x, None, freq)
    assert y[0, 0, 0, 5] == float("inf") and bool(y[0, 0, 1].isfinite().all()) and bool((y[0, 0, 0, :5] == 1).all())


def test_scaled_rows_and_small_eps():
    """Magnitudes at the ends of the stated range."""
    x = torch.randn(1, 1, 3, 64, generator=torch.Generator().manual_seed(9)).cuda()
    x = x / x.abs().amax(-1, keepdim=True)
    x[0, 0, 0] *= 2.0 ** 60
    x[0, 0, 1] *= 2.0 ** -59
    freq = torch.rand(1, 16).cuda()
    th = ON.angles(np.arange(3)[None, None], freq.cpu().numpy())[:, None]
    qo = hca.hca_norm_rope_fwd(x, None, None, None, None, freq, 0.0)[0]
    check_fwd(x, None, th, 32, False, qo, "q", eps=0.0)


def serve_case(add, held, H, D, rot, dtype, seed, pad=0, axes=1):
    g = torch.Generator().manual_seed(seed)
    n = sum(add) + pad
    q, kv = torch.randn(n, H, D, generator=g).to(dtype).cuda(), torch.randn(n, D, generator=g).to(dtype).cuda()
    start = torch.tensor(np.concatenate([[0], np.cumsum(add)]), dtype=torch.int32).cuda()
    freq = torch.rand(axes, rot // 2, generator=g).cuda()
    pos = np.concatenate([np.arange(h, h + a) for h, a in zip(held, add)] + [np.zeros(pad)]).astype(np.int64)
    return q, kv, start, torch.tensor(held, dtype=torch.int32).cuda(), freq, pos, (1 + 0.2 * torch.randn(D, generator=g)).cuda()


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("add,held,H,D,rot,halves,pad", [
    ([1], [0], 64, 128, 64, False, 0), ([1] * 64, list(range(0, 64 * 2003, 2003)), 16, 128, 64, False, 7),
    ([0, 5, 0, 0, 33, 1, 0], [9, 100000, 3, 0, 2 ** 30 - 40, 7, 1], 3, 64, 64, True, 3), ([700, 1, 90], [5, 70000, 0], 2, 72, 16, False, 0),
    ([1, 0, 2] * 500, list(range(1500)), 1, 64, 32, False, 5), ([3] * 1024, list(range(1024)), 1, 512, 64, True, 1)])
def test_packed_tokens(add, held, H, D, rot, halves, pad, dtype):
    q, kv, start, h, freq, pos, w = serve_case(add, held, H, D, rot, dtype, 10, pad)
    n = sum(add)
    th = ON.angles(pos[None], freq.cpu().numpy())
    qo, kvo = torch.full_like(q, 5), torch.full_like(kv, 5)
    hca.hca_cache_norm_rope(q, kv, start, h, w, w, freq, EPS, halves=halves, qo=qo, kvo=kvo)
    check_fwd(q[:n], w, th[:n, None], D - rot, halves, qo[:n], "q")
    check_fwd(kv[:n], w, th[:n], D - rot, halves, kvo[:n], "kv")
    y = torch.full_like(q, 5)
    hca.hca_cache_rope(q, start, h, freq, inverse=True, halves=halves, y=y)
    close("y", y[:n], ON.rotate(f64(q[:n]), -th[:n, None], D - rot, halves), ON.rotate_bound(f64(q[:n]), th[:n, None], D - rot, halves), dtype)
    for t in (qo, kvo, y):  # rows behind the last request
        assert bool((t[n:] == 5).all())


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("halves", [False, True])
def test_wide_rows_of_few_heads(halves, dtype):
    """More tiles of 8 tokens than blocks, which take several each."""
    add, held = [1200, 0, 1701, 3], [70, 5, 0, 900000]
    q, kv, start, h, freq, pos, w = serve_case(add, held, 2, 512, 64, dtype, 17, 300)
    n = sum(add)
    th = ON.angles(pos[None], freq.cpu().numpy())
    qo, kvo = torch.full_like(q, 5), torch.full_like(kv, 5)
    hca.hca_cache_norm_rope(q, kv, start, h, w, w, freq, EPS, halves=halves, qo=qo, kvo=kvo)
    check_fwd(q[:n], w, th[:n, None], 448, halves, qo[:n], "q")
    check_fwd(kv[:n], w, th[:n], 448, halves, kvo[:n], "kv")
    assert bool((qo[n:] == 5).all()) and bool((kvo[n:] == 5).all())
    q, kv, wq, wkv, pos, freq, _, _ = make(3, 1, 1111, 320, 32, dtype, 18)
    th = ON.angles(pos.cpu().numpy(), freq.cpu().numpy())
    qo, kvo = hca.hca_norm_rope_fwd(q, kv, wq, wkv, pos, freq, EPS, halves=halves)
    check_fwd(q, wq, th[:, None], 288, halves, qo, "q")
    check_fwd(kv, wkv, th, 288, halves, kvo, "kv")


def test_packed_coordinates_and_strides():
    q, kv, start, held, freq, _, w = serve_case([4, 9], [3, 8], 5, 64, 32, BF16, 11, 2, axes=3)
    pos = torch.randint(0, 999, (3, 15), dtype=torch.int32).cuda()
    th = ON.angles(pos.cpu().numpy(), freq.cpu().numpy())
    wide = torch.zeros(15, 7, 64, dtype=BF16, device="cuda")
    wide[:, :5] = q
    wide[:, 5] = kv
    qo, kvo = hca.hca_cache_norm_rope(wide[:, :5], wide[:, 5], start, None, w, None, freq, EPS, pos=pos)
    check_fwd(q[:13], w, th[:13, None], 32, False, qo[:13], "q")
    check_fwd(kv[:13], None, th[:13], 32, False, kvo[:13], "kv")
    one = pos[0].contiguous()
    a = hca.hca_cache_rope(q, start, None, freq[0], pos=one)
    b = hca.hca_rope(q.transpose(0, 1)[None], one[None], freq[0])[0].transpose(0, 1)
    assert torch.equal(a[:13], b[:13])


def test_values_out_of_order_touch_nothing_else():
    """Lengths that mean nothing give positions that mean nothing."""
    q, kv, _, held, freq, _, w = serve_case([4, 9], [3, 8], 5, 64, 32, BF16, 12, 2)
    for start in ([0, 9, 4], [-5, 100, 15], [3, 2 ** 31 - 1, 2 ** 31 - 1], [0, 7, -3]):
        s = torch.tensor(start, dtype=torch.int32).cuda()
        buf = torch.full((3, 15, 5, 64), 5.0, dtype=BF16, device="cuda")
        hca.hca_cache_norm_rope(q, None, s, held, w, None, freq, EPS, qo=buf[1])
        torch.cuda.synchronize()
        assert bool((buf[0] == 5).all()) and bool((buf[2] == 5).all())
        live = max(0, min(15, start[-1]))
        assert bool((buf[1, live:] == 5).all()) and bool(buf[1].isfinite().all())


def test_other_stream_and_captured():
    q, kv, wq, wkv, pos, freq, dq, dkv = make(2, 8, 70, 128, 64, BF16, 13)
    want = hca.hca_norm_rope_fwd(q, kv, wq, wkv, pos, freq, EPS)
    wantb = hca.hca_norm_rope_bwd(q, kv, wq, wkv, pos, freq, EPS, dq, dkv)
    st = torch.cuda.Stream()
    st.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(st):
        a = hca.hca_norm_rope_fwd(q, kv, wq, wkv, pos, freq, EPS)
        b = hca.hca_norm_rope_bwd(q, kv, wq, wkv, pos, freq, EPS, dq, dkv)
    st.synchronize()
    assert all(torch.equal(x, y) for x, y in zip((*a, *b), (*want, *wantb)))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        a = hca.hca_norm_rope_fwd(q, kv, wq, wkv, pos, freq, EPS)
        b = hca.hca_norm_rope_bwd(q, kv, wq, wkv, pos, freq, EPS, dq, dkv)
    pos += 3
    q.mul_(1.5)
    graph.replay()
    torch.cuda.synchronize()
    want = hca.hca_norm_rope_fwd(q, kv, wq, wkv, pos, freq, EPS)
    wantb = hca.hca_norm_rope_bwd(q, kv, wq, wkv, pos, freq, EPS, dq, dkv)
    assert all(torch.equal(x, y) for x, y in zip((*a, *b), (*want, *wantb)))


def test_long_sequence_many_tiles():
    """More tiles than blocks of the backward, batch rows and head ranges among them, against itself in pieces."""
    q, kv, wq, wkv, pos, freq, dq, dkv = make(3, 20, 9001, 64, 48, BF16, 14, axes=2)
    out = hca.hca_norm_rope_fwd(q, kv, wq, wkv, pos, freq, EPS)
    back = hca.hca_norm_rope_bwd(q, kv, wq, wkv, pos, freq, EPS, dq, dkv)
    sq, skv = 0.0, 0.0
    for i in range(3):
        for a, b in ((0, 4500), (4500, 9001)):
            args = (q[i:i + 1, :, a:b], kv[i:i + 1, a:b], wq, wkv, pos[:, i:i + 1, a:b].contiguous(), freq, EPS)
            o = hca.hca_norm_rope_fwd(*args)
            assert torch.equal(o[0], out[0][i:i + 1, :, a:b]) and torch.equal(o[1], out[1][i:i + 1, a:b])
            d = hca.hca_norm_rope_bwd(*args, dq[i:i + 1, :, a:b].contiguous(), dkv[i:i + 1, a:b].contiguous())
            assert torch.equal(d[0], back[0][i:i + 1, :, a:b]) and torch.equal(d[1], back[1][i:i + 1, a:b])
            sq, skv = sq + d[2].double(), skv + d[3].double()
    # sums of 540,060 and 27,003 terms of the size of a product of two normal numbers: a chain of
    # roundings, each 2^-24 of a partial sum that stays below some sqrt(n) * 10
    for name, got, ref, n in (("dwq", back[2], sq, 540060), ("dwkv", back[3], skv, 27003)):
        assert float((got.double() - ref).abs().max()) <= n ** 0.5 * 10 * 2000 * 2.0 ** -24, name


def test_both_ways_of_the_binding_give_the_same(monkeypatch):
    if hca.load() and hca._py is None:
        pytest.skip("built without the headers of Python or torch")
    q, kv, wq, wkv, pos, freq, dq, dkv = make(2, 3, 21, 128, 64, BF16, 15, axes=2)
    sq, skv, start, held, sfreq, _, w = serve_case([4, 9], [3, 8], 5, 64, 32, F32, 16, 2)
    wide = torch.zeros(15, 6, 64, device="cuda")
    wide[:, 1:] = sq
    spos = torch.arange(15, dtype=torch.int32).cuda() * 7

    def calls():
        r = [*hca.hca_norm_rope_fwd(q, kv, wq, None, pos, freq, EPS, halves=True), *hca.hca_norm_rope_bwd(q, kv, wq, None, pos, freq, EPS, dq, dkv),
             hca.hca_rope(q, pos, freq, inverse=True, first=0), hca.hca_rope(q, pos, freq, y=torch.empty_like(q)),
             hca.hca_norm_rope_bwd(q[:, :1].expand(2, 3, 21, 128), None, None, None, pos, freq, EPS, dq, None)[0]]
        out = torch.zeros_like(sq), torch.zeros_like(skv), torch.zeros_like(sq)
        hca.hca_cache_norm_rope(wide[:, 1:], skv, start, held, w, w, sfreq, EPS, qo=out[0], kvo=out[1])
        hca.hca_cache_rope(wide[:, 1:], start, None, sfreq[0], pos=spos, y=out[2])
        return r + list(out)

    a = calls()
    monkeypatch.setattr(hca, "_py", None)
    for x, y in zip(a, calls()):
        assert (x is None and y is None) or (torch.equal(x, y) and x.stride() == y.stride())


def test_the_binding_refuses():
    q, kv, wq, wkv, pos, freq, dq, dkv = make(2, 3, 21, 128, 64, BF16, 17)
    f = hca.hca_norm_rope_fwd
    for bad, error in (((q, kv[:, :20], wq, wkv, pos, freq), ValueError), ((q, kv.float(), wq, wkv, pos, freq), TypeError),
                       ((q, kv, wq.bfloat16(), wkv, pos, freq), TypeError), ((q, kv, wq[:64], wkv, pos, freq), ValueError),
                       ((q, kv, wq, wkv, pos.long(), freq), TypeError), ((q, kv, wq, wkv, pos[:, :, :9], freq), ValueError),
                       ((q, kv, wq, wkv, pos, freq.double()), TypeError), ((q, kv, wq, wkv, None, freq.expand(2, 32).contiguous()), ValueError),
                       ((q, kv, wq, wkv, pos, freq.cpu()), ValueError), ((q.half(), kv.half(), wq, wkv, pos, freq), TypeError),
                       ((q, kv, wq, wkv, pos, None), ValueError), ((q[..., ::2], kv, wq, wkv, pos, freq), ValueError)):
        with pytest.raises(error):
            f(*bad, EPS)
    with pytest.raises(hca.HCAError):
        f(q, kv, wq, wkv, pos, freq, -1.0)
    with pytest.raises(hca.HCAError):
        f(q, kv, wq, wkv, pos, freq, EPS, first=72)
    with pytest.raises(ValueError):
        hca.hca_norm_rope_bwd(q, kv, wq, None, pos, freq, EPS, dq, dkv, dwkv=torch.empty(128, device="cuda"))
    with pytest.raises(ValueError):
        hca.hca_norm_rope_bwd(q, kv, wq, wkv, pos, freq, EPS, dq[:, :2], dkv)
    with pytest.raises(hca.HCAError) as e:
        hca.hca_norm_rope_bwd(q, kv, wq, wkv, pos, freq, EPS, dq, dkv, ws=torch.empty(64, dtype=torch.uint8, device="cuda"))
    assert e.value.status == 7
    with pytest.raises(ValueError):
        hca.hca_cache_rope(q[0].transpose(0, 1), None, None, freq)
    with pytest.raises(ValueError):  # a batch is not packed tokens
        hca.hca_cache_rope(q, None, None, freq)
    with pytest.raises(ValueError):
        hca.hca_cache_norm_rope(q, kv, None, None, None, None, freq, EPS)
    with pytest.raises(ValueError):
        hca.hca_cache_norm_rope(q[0].transpose(0, 1), None, torch.zeros(2, dtype=torch.int32, device="cuda"), None, None, None, freq, EPS)


def test_offsets_beyond_32_bits():
    """2.35e9 elements, turned in place; rows at both ends and around 2^31."""
    B, H, S, D = 2, 70, 32768, 512
    x = torch.empty(B, H, S, D, dtype=BF16, device="cuda")
    assert x.numel() > 2 ** 31
    g = torch.Generator(device="cuda").manual_seed(19)
    some = [(0, 0, 0), (0, 69, 32767), (1, 57, 32766), (1, 58, 32767), (1, 69, 32767), (1, 3, 5)]
    x.zero_()
    rows = torch.randn(len(some), D, generator=g, device="cuda").to(BF16)
    for (b, h, s), r in zip(some, rows):
        x[b, h, s] = r
    freq = torch.rand(32, generator=g, device="cuda")
    pos = torch.randint(0, 10 ** 6, (B, S), dtype=torch.int32, device="cuda", generator=g)
    hca.hca_rope(x, pos, freq, y=x)
    for (b, h, s), r in zip(some, rows):
        th = ON.angles(pos[b, s].cpu().numpy()[None], freq.cpu().numpy()[None])
        close("x", x[b, h, s], ON.rotate(f64(r), th, D - 64, False), ON.rotate_bound(f64(r), th, D - 64, False), BF16)
    assert int((x != 0).any(-1).sum()) == len(some)
    out = hca.hca_norm_rope_fwd(x, None, None, None, pos, freq, EPS)[0]
    for b, h, s in some:
        th = ON.angles(pos[b, s].cpu().numpy()[None], freq.cpu().numpy()[None])
        check_fwd(x[b, h, s], None, th, D - 64, False, out[b, h, s], "q")
    assert int((out != 0).any(-1).sum()) == len(some)


def test_threads_that_call_at_once():
    import threading
    q, kv, wq, wkv, pos, freq, dq, dkv = make(1, 4, 300, 64, 32, BF16, 18)
    want = hca.hca_norm_rope_bwd(q, kv, wq, wkv, pos, freq, EPS, dq, dkv)
    bad = []

    def work():
        with torch.cuda.stream(torch.cuda.Stream()):
            for _ in range(20):
                got = hca.hca_norm_rope_bwd(q, kv, wq, wkv, pos, freq, EPS, dq, dkv)
                torch.cuda.current_stream().synchronize()
                bad.extend(1 for a, b in zip(got, want) if not torch.equal(a, b))

    torch.cuda.synchronize()
    threads = [threading.Thread(target=work) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not bad


@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("R", [1, 1024, 1025, 3000])
def test_packed_norms_that_do_not_turn_need_no_lengths(R, dtype):
    """The C call takes held = NULL where rot is 0, for any number of requests."""
    q, kv, start, _, _, _, w = serve_case([1, 2, 0][:R] + [1] * (R - 3), [0] * R, 2, 64, 16, dtype, 20, pad=3)
    n, N = int(start[-1]), q.shape[0]
    qo, kvo, y = torch.full_like(q, 5), torch.full_like(kv, 5), torch.full_like(q, 5)
    lib, code, st = hca.load(), 1 if dtype == F32 else 0, torch.cuda.current_stream().cuda_stream
    assert lib.hca_norm_rope_fwd(q.data_ptr(), (ctypes.c_int64 * 3)(0, 64, 128), w.data_ptr(), qo.data_ptr(), kv.data_ptr(), None, None,
                                 kvo.data_ptr(), None, None, start.data_ptr(), None, 1, 2, N, 64, R, 1, 0, 0, 0, EPS, code, st) == 0
    assert lib.hca_rope(q.data_ptr(), None, y.data_ptr(), None, None, None, start.data_ptr(), None, 1, 2, N, 64, R, 1, 0, 0, 0, 0, code, st) == 0
    th = np.zeros((n, 0))
    check_fwd(q[:n], w, th[:, None], 0, False, qo[:n], "q")
    check_fwd(kv[:n], None, th, 0, False, kvo[:n], "kv")
    assert torch.equal(y[:n], q[:n])
    for t in (qo, kvo, y):
        assert bool((t[n:] == 5).all())


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 2.0 ** 64, -3e38])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("D,rot,halves,axes,at", [(64, 64, False, 1, 0), (64, 32, True, 2, 31), (512, 512, False, 4, 1023), (512, 256, True, 4, 300)])
def test_frequencies_without_an_angle(D, rot, halves, axes, at, dtype, bad):
    """All columns that turn are NaN then, at position 0 too; the others stay as they are."""
    q, kv, wq, wkv, pos, freq, dq, dkv = make(2, 3, 37, D, rot, dtype, 21, axes=axes)
    pos[:, 0, :5] = 0
    calls = lambda: hca.hca_norm_rope_fwd(q, kv, wq, wkv, pos, freq, EPS, halves=halves) + (  # noqa: E731
        hca.hca_rope(q, pos, freq, halves=halves, inverse=True),)
    want, back = calls(), hca.hca_norm_rope_bwd(q, kv, wq, wkv, pos, freq, EPS, dq, dkv, halves=halves)
    freq.view(-1)[at] = bad
    first = D - rot
    for a, b in zip(calls(), want):
        assert bool(a[..., first:].isnan().all()) and torch.equal(a[..., :first], b[..., :first])
    gq, gkv, gwq, gwkv = hca.hca_norm_rope_bwd(q, kv, wq, wkv, pos, freq, EPS, dq, dkv, halves=halves)
    assert bool(gq.isnan().all()) and bool(gkv.isnan().all())  # a row's mean has them all
    for a, b in ((gwq, back[2]), (gwkv, back[3])):
        assert bool(a[first:].isnan().all()) and torch.equal(a[:first], b[:first])


def test_dw_of_a_long_sequence_keeps_its_bits():
    """8.4e6 equal terms in each column, c x r with x = r = 1.  A thread adds up its rows of a
    tile of tokens (a head each), then its tiles, of which a block has S / 32 / SMs at most, as a
    block has 32 rows of 8 columns at once: each of these additions is off by 2^-24 of a sum of
    positive terms at most.  The sums over a block's rows and over blocks carry what they round
    off: 2 each, and 2 for r.  (In one sum over all rows of a thread: 133 units in column 0.)"""
    H, S, D = 32, 262144, 8
    c = torch.tensor([1.1, 0.7654321, 1.7, 1.2345678, 1.3333334, 1.0000001, 0.9, 1.9])
    x, g = torch.ones(1, H, S, D, device="cuda"), c.cuda().expand(1, H, S, D).contiguous()
    dw = hca.hca_norm_rope_bwd(x, None, torch.ones(D, device="cuda"), None, None, torch.zeros(0, device="cuda"), 0.0, g, None)[2]
    units = H + -(-S // 32 // torch.cuda.get_device_properties(0).multi_processor_count) + 6
    ref = c.double() * H * S
    assert bool(((dw.cpu().double() - ref).abs() <= units * 2.0 ** -24 * ref).all()), (dw.cpu().double() / ref - 1) * 2 ** 24


@pytest.mark.parametrize("halves", [False, True])
@pytest.mark.parametrize("axes", [2, 3, 4])
def test_far_coordinates_of_several_axes(axes, halves):
    """Each axis at the ends of 32 bits, with frequencies up to the stated 2^32: what is cut off
    adds up over the axes."""
    g = torch.Generator().manual_seed(22)
    ends = torch.tensor([2 ** 31 - 1, -2 ** 31, 2 ** 31 - 12345, -2 ** 31 + 777, 0, -1], dtype=torch.int64)
    pos = ends[torch.randint(0, len(ends), (axes, 1, 400), generator=g)].to(torch.int32).cuda()
    freq = torch.exp2(torch.rand(axes, 64, generator=g) * 62 - 30).cuda()  # 2^-30 .. 2^32
    freq *= torch.where(torch.rand(axes, 64, generator=g) < 0.3, -1.0, 1.0).cuda()
    x = torch.randn(1, 3, 400, 128, generator=g).cuda()
    th = ON.angles(pos.cpu().numpy(), freq.cpu().numpy())[:, None]
    for inverse in (False, True):
        y = hca.hca_rope(x, pos, freq, halves=halves, inverse=inverse)
        t = -th if inverse else th
        close("y", y, ON.rotate(f64(x), t, 0, halves), ON.rotate_bound(f64(x), t, 0, halves), F32)
