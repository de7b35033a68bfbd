"""The calls of a layer one after the other, as a program uses them: training, where
the gradients are those of the whole in 64 bits, and serving, where a captured step
with a common prefix is replayed."""
import math

import numpy as np
import pytest
import torch

from block_sparse_compressed_gb300 import hca
from oracle import norm_rope as ON

pytestmark = pytest.mark.gpu
DEV, BF16, F32 = "cuda", torch.bfloat16, torch.float32
EPS = 1e-6


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


# ---------------------------------------------------------------------------
# training: norm and rotation, compressor, attention, rotation back
# ---------------------------------------------------------------------------
def _turn(x, e, first):
    """Pairs of neighbours from column `first` on as complex numbers times e."""
    n = e.shape[-1]
    z = torch.view_as_complex(x[..., first:first + 2 * n].unflatten(-1, (n, 2)).contiguous()) * e
    return torch.cat([x[..., :first], torch.view_as_real(z).flatten(-2), x[..., first + 2 * n:]], -1)


def _norm(x, w):
    return x / torch.sqrt((x * x).mean(-1, keepdim=True) + EPS) * w


def _layer64(q, kv, g, wq, wkv, bias, e, W, m, scale, first):
    """The layer in 64 bits: q [B,H,S,D], kv [B,S,D] raw; out [B,H,S,D]."""
    B, H, S, D = q.shape
    q, kv = _turn(_norm(q, wq), e[:, None], first), _turn(_norm(kv, wkv), e, first)
    Sc = S // m  # whole windows: the rest is never seen
    a = torch.softmax(g[:, :Sc * m].reshape(B, Sc, m) + bias, -1)
    ckv = torch.einsum("bjr,bjrd->bjd", a, kv[:, :Sc * m].reshape(B, Sc, m, D))
    i = torch.arange(S)
    raw = (i[None, :] <= i[:, None]) & (i[None, :] > i[:, None] - W)
    comp = (torch.arange(Sc)[None, :] + 1) * m <= i[:, None] + 1
    keys, vis = torch.cat([kv, ckv], 1), torch.cat([raw, comp], 1)
    s = torch.einsum("bhsd,bkd->bhsk", q, keys) * scale
    p = torch.softmax(s.masked_fill(~vis, -math.inf), -1)
    return _turn(torch.einsum("bhsk,bkd->bhsd", p, keys), e[:, None].conj(), first)


@pytest.mark.parametrize("dtype", [F32, BF16])
def test_a_layer_and_its_gradients(dtype):
    B, H, S, D, W, m, rot = 2, 4, 90, 64, 16, 8, 32
    first, scale = D - rot, 1 / math.sqrt(D)
    gen = torch.Generator().manual_seed(1)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    q, kv, g, dout = rnd(B, S, H, D).to(dtype), rnd(B, S, D).to(dtype), rnd(B, S), rnd(B, S, H, D).to(dtype)
    wq, wkv, bias, freq = 1 + 0.2 * rnd(D), 1 + 0.2 * rnd(D), 0.3 * rnd(m), rnd(1, rot // 2).abs()
    pos = (torch.arange(S) + 1000).int().repeat(B, 1)
    # the calls; q, out and their gradients token by token, as the projections have them
    c = lambda t: t.to(DEV)  # noqa: E731
    qg, kvg, gg, doutg, p = c(q).transpose(1, 2), c(kv), c(g), c(dout).transpose(1, 2), c(pos)
    ws = [c(wq), c(wkv), c(bias), c(freq)]
    qr, kvr = hca.hca_norm_rope_fwd(qg, kvg, ws[0], ws[1], p, ws[3], EPS)
    ckv = hca.hca_compress_fwd(kvr, gg, ws[2], None, m)
    o, lse = hca.hca_attn_fwd(qr, kvr, ckv, None, W, m, scale, check=True)
    y = torch.empty(B, S, H, D, dtype=dtype, device=DEV)
    hca.hca_rope(o, p, ws[3], inverse=True, y=y.transpose(1, 2))
    do = hca.hca_rope(doutg, p, ws[3])  # the gradient of the rotation back is the rotation
    assert do.is_contiguous()
    dqr, dkvr, dckv = hca.hca_attn_bwd(qr, kvr, ckv, None, o, lse, do, W, m, scale, check=True)
    dx, dg, dbias = hca.hca_compress_bwd(kvr, gg, ws[2], None, m, dckv)
    dq, dkv, dwq, dwkv = hca.hca_norm_rope_bwd(qg, kvg, ws[0], ws[1], p, ws[3], EPS, dqr, (dkvr.float() + dx.float()).to(dtype))
    # the same in 64 bits
    leaves = [t.double().requires_grad_(True) for t in (q.transpose(1, 2), kv, g, wq, wkv, bias)]
    th = torch.from_numpy(ON.angles(pos.numpy()[None], freq.numpy()))
    ref = _layer64(*leaves, torch.polar(torch.ones_like(th), th), W, m, scale, first)
    grads = torch.autograd.grad(ref, leaves, dout.double().transpose(1, 2))
    got = (y.transpose(1, 2), dq, dkv, dg, dwq, dwkv, dbias)
    # fp32: some hundred roundings of 2^-24 a value, along a chain of five calls.  bf16: a
    # dozen tensors in between are rounded by 2^-8 of their values; a result is a sum of many
    # products of them, whose errors add up like their squares: 2^-8 times the root of 12,
    # times 4 for the largest of some thousand values, of the tensor's largest value.
    tol = 2e-5 if dtype == F32 else 4 * 12 ** 0.5 * 2.0 ** -8
    for name, a, b in zip(("y", "dq", "dkv", "dg", "dwq", "dwkv", "dbias"), got, (ref, *grads)):
        a, b = a.double().cpu(), b.detach()
        err, top = float((a - b).abs().max()), float(b.abs().max())
        assert err <= tol * top, f"{name}: {err:.3e} of {top:.3e}"


# ---------------------------------------------------------------------------
# serving: a captured step over a common prefix
# ---------------------------------------------------------------------------
def test_a_captured_step_over_a_common_prefix():
    """Requests that go on from one prompt: their compressed tables begin with its
    blocks.  Each step plans, normalises and rotates, writes, attends, turns back;
    the attention of every step is the oracle's over what the cache holds."""
    from _cache import check_attn
    R, H, D, W, m, bs, rot, shared = 5, 8, 64, 16, 4, 16, 32, 3
    scale, P = 1 / math.sqrt(D), shared * 16 * 4  # P tokens of the prompt
    gen = torch.Generator().manual_seed(2)
    rnd = lambda *s: torch.randn(*s, generator=gen)  # noqa: E731
    nblocks, cols_raw, cols = 64, -(-W // bs) + 1, shared + 2
    pool, scales = torch.zeros(nblocks, bs, D).to(torch.float8_e4m3fn).to(DEV), torch.ones(nblocks, device=DEV)
    free, count = i32(list(range(nblocks))), i32([nblocks])
    wq, wkv, freq = (1 + 0.2 * rnd(D)).to(DEV), (1 + 0.2 * rnd(D)).to(DEV), rnd(rot // 2).abs().to(DEV)
    bias = torch.zeros(m, device=DEV)

    # the prompt, once: its compressed entries into blocks of their own
    prompt = rnd(P, D).to(BF16).to(DEV)
    one, held0, added0 = torch.full((1, shared), -1, dtype=torch.int32, device=DEV), i32([0]), i32([P])
    _, slots, _ = hca.hca_cache_plan(held0, added0, one, free, count, nblocks, bs, P // m, m=m, free_left=count, check=True)
    _, kvp = hca.hca_cache_norm_rope(None, prompt, i32([0, P]), held0, None, wkv, freq, EPS)
    gates = rnd(P).to(DEV)
    hca.hca_cache_append(hca.hca_compress_fwd(kvp[None], gates[None], bias, None, m)[0], slots, pool, scales, check=True)
    # the requests: tables that begin with the prompt's blocks, and the prompt's last rows in rings of their own
    comp_table = torch.full((R, cols), -1, dtype=torch.int32, device=DEV)
    comp_table[:, :shared] = one
    raw_table = torch.full((R, cols_raw), -1, dtype=torch.int32, device=DEV)
    h = P - W
    held = i32([h] * R)
    for r in range(R):  # a ring's columns are all in use by then
        for c in range(cols_raw):
            raw_table[r, c] = free[int(count) - 1]
            count -= 1
    page = torch.arange(h, P, device=DEV)
    for r in range(R):
        slots = (raw_table[r][(page // bs) % cols_raw] * bs + page % bs).int()
        hca.hca_cache_append(kvp[h:], slots, pool, scales, check=True)
    held.fill_(P)

    # one step: a token each, with room for one more row than there are
    N = R + 1
    x_q, x_kv, x_g = (torch.zeros(N, H, D, dtype=BF16, device=DEV), torch.zeros(N, D, dtype=BF16, device=DEV),
                      torch.zeros(N, device=DEV))
    added, first, shared_cols = i32([1] * R), i32([0, R]), i32([shared])
    recent, gate, rows = torch.zeros(R, m, D, dtype=BF16, device=DEV), torch.zeros(R, m, device=DEV), torch.arange(R, device=DEV)
    out, lse, y = torch.zeros(N, H, D, dtype=BF16, device=DEV), torch.zeros(N, H, device=DEV), torch.zeros(N, H, D, dtype=BF16, device=DEV)
    qr, kvr = torch.zeros_like(x_q), torch.zeros_like(x_kv)
    at_held = torch.zeros_like(held)

    def step():
        start, slots, _ = hca.hca_cache_plan(held, added, raw_table, free, count, nblocks, bs, N, free_left=count)
        ent_start, ent_slots, _ = hca.hca_cache_plan(held, added, comp_table, free, count, nblocks, bs, R, m=m, free_left=count)
        hca.hca_cache_norm_rope(x_q, x_kv, start, held, wq, wkv, freq, EPS, qo=qr, kvo=kvr)
        at = (held % m).long()
        recent[rows, at], gate[rows, at] = kvr[:R], x_g[:R]
        entries = hca.hca_compress_fwd(recent, gate, bias, None, m)[:, 0]
        entries = entries[torch.searchsorted(ent_start[1:], rows.int(), right=True).clamp(max=R - 1)]
        hca.hca_cache_append(kvr, slots, pool, scales)
        hca.hca_cache_append(entries, ent_slots, pool, scales)
        hca.hca_cache_attn_shared(qr, start, held, (pool, scales, raw_table), (pool, scales, comp_table), first, shared_cols, W, m, scale,
                                  out=out, lse=lse)
        hca.hca_cache_rope(out, start, held, freq, inverse=True, y=y)
        at_held.copy_(held)
        held.add_(added)

    state = [t.clone() for t in (held, count, raw_table, comp_table, pool.view(torch.uint8), scales, recent, gate)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    hca.hca_test_inject(hca.INJECT_SHARED_PATH, 1)
    try:
        with torch.cuda.stream(side):
            step()
        torch.cuda.current_stream().wait_stream(side)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step()
    finally:
        hca.hca_test_inject(hca.INJECT_RESET)
    for t, v in zip((held, count, raw_table, comp_table, pool.view(torch.uint8), scales, recent, gate), state):
        t.copy_(v)
    start = torch.arange(R + 1, dtype=torch.int32)
    for n in range(3 * bs):  # past the ends of windows, blocks and ring columns
        x_q.copy_(rnd(N, H, D))
        x_kv.copy_(rnd(N, D))
        x_g.copy_(rnd(N))
        y[R] = 7
        graph.replay()
        torch.cuda.synchronize()
        assert bool((y[R] == 7).all()) and bool((out[R] == 0).all())
        if n % 7 and n < 3 * bs - 2:
            continue
        cache = (pool.cpu(), scales.cpu())
        hd = at_held.cpu()
        assert hd.tolist() == [P + n] * R and comp_table[:, :shared].tolist() == [one[0].tolist()] * R
        check_attn((out[:R], lse[:R]), qr[:R].cpu(), start, hd, (*cache, raw_table.cpu()), (*cache, comp_table.cpu()), W, m, scale, BF16)
        th = ON.angles(hd.numpy()[None], freq.cpu().numpy()[None])
        f64 = lambda t: t.float().cpu().double().numpy()  # noqa: E731
        for name, got, ref, tol in (
                ("q", qr[:R], ON.forward(f64(x_q[:R]), f64(wq), EPS, th[:, None], D - rot, False),
                 ON.forward_bound(f64(x_q[:R]), f64(wq), EPS, th[:, None], D - rot, False)),
                ("y", y[:R], ON.rotate(f64(out[:R]), -th[:, None], D - rot, False), ON.rotate_bound(f64(out[:R]), -th[:, None], D - rot, False))):
            assert np.all(np.abs(f64(got) - ref) <= 2.0 ** -8 * (np.abs(ref) + tol) + tol), name
