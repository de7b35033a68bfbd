"""Compressed entries of a captured decode step, from calls that are there: the rows
of each request's open window are kept, compressed every step, and the device
knows which of them are complete."""
import numpy as np
import pytest
import torch

from _cache import E4M3, check_attn, ring_cols, scale_of, values
from block_sparse_compressed_gb300 import hca
from oracle import cache as OC

pytestmark = pytest.mark.gpu
DEV = "cuda"


def i32(v):
    return torch.tensor(v, dtype=torch.int32, device=DEV)


@pytest.mark.parametrize("dtype,H,D", [(torch.bfloat16, 64, 128), (torch.float32, 4, 64)])
def test_a_captured_step_compresses_its_own_windows(dtype, H, D):
    R, W, m, bs, steps = 5, 40, 8, 16, 19
    prompt = [37, 5, 64, 15, 0]
    g = torch.Generator().manual_seed(7)
    n = [p + steps for p in prompt]
    kv = [torch.randn(k, D, generator=g).to(dtype).to(DEV) for k in n]
    gate = [torch.randn(k, generator=g).to(DEV) for k in n]
    bias = torch.randn(m, generator=g).to(DEV)
    qs = torch.randn(steps, R, H, D, generator=g).to(dtype).to(DEV)
    whole = [hca.hca_compress_fwd(kv[r][None], gate[r][None], bias, None, m)[0] for r in range(R)]

    cols, ccols = ring_cols(W, max(prompt), bs), -(-(max(n) // m) // bs)
    nblocks = R * (cols + ccols)
    pool, scale = torch.zeros(nblocks, bs, D, device=DEV).to(E4M3), torch.ones(nblocks, device=DEV)
    raw_table, comp_table = (torch.full((R, c), -1, dtype=torch.int32, device=DEV) for c in (cols, ccols))
    free, count, held = i32(list(range(nblocks))), i32([nblocks]), i32([0] * R)
    recent, gates = torch.zeros(R, m, D, dtype=dtype, device=DEV), torch.zeros(R, m, device=DEV)
    rows = torch.arange(R, device=DEV)

    def plan(added, table, nslots, m):
        return hca.hca_cache_plan(held, added, table, free, count, nblocks, bs, nslots, m=m, free_left=count)[:2]

    # the prompts, whose entries are known beforehand
    added = i32(prompt)
    start, slots = plan(added, raw_table, sum(prompt), 1)
    _, cslots = plan(added, comp_table, sum(p // m for p in prompt), m)
    hca.hca_cache_append(torch.cat([kv[r][:p] for r, p in enumerate(prompt)]), slots, pool, scale, check=True)
    hca.hca_cache_append(torch.cat([whole[r][:p // m] for r, p in enumerate(prompt)]), cslots, pool, scale, check=True)
    for r, p in enumerate(prompt):
        recent[r, :p % m], gates[r, :p % m] = kv[r][p // m * m:p], gate[r][p // m * m:p]
    held += added
    one = i32([1] * R)

    def step(x, gx, q):
        start, slots = plan(one, raw_table, R, 1)
        cstart, cslots = plan(one, comp_table, R, m)
        at = (held % m).long()
        recent[rows, at], gates[rows, at] = x, gx
        ent = hca.hca_compress_fwd(recent, gates, bias, None, m)[:, 0]
        ent = ent[torch.searchsorted(cstart[1:], rows.int(), right=True).clamp(max=R - 1)]  # those that complete a window, packed
        hca.hca_cache_append(x, slots, pool, scale)
        hca.hca_cache_append(ent, cslots, pool, scale)
        out, lse = hca.hca_cache_attn(q, start, held, (pool, scale, raw_table), (pool, scale, comp_table), W, m, scale_of(D))
        held.add_(one)
        return out, lse, ent, cslots

    def inputs(k):
        return torch.stack([kv[r][prompt[r] + k] for r in range(R)]), torch.stack([gate[r][prompt[r] + k] for r in range(R)]), qs[k]

    state = (pool.view(torch.uint8), scale, raw_table, comp_table, count, held, recent, gates)
    kept = [t.clone() for t in state]
    fixed = [t.clone() for t in inputs(0)]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step(*fixed)
    torch.cuda.current_stream().wait_stream(side)
    for t, s in zip(state, kept):
        t.copy_(s)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out, lse, ent, cslots = step(*fixed)
    for t, s in zip(state, kept):
        t.copy_(s)
    want, wscale = values(pool), scale.cpu().double().numpy()
    for k in range(steps):
        for t, v in zip(fixed, inputs(k)):
            t.copy_(v)
        graph.replay()
        h = [p + k for p in prompt]
        done = [r for r in range(R) if (h[r] + 1) % m == 0]
        live = [s for s in cslots.tolist() if s >= 0]
        assert len(live) == len(done) and cslots.tolist()[:len(done)] == live
        for i, r in enumerate(done):
            assert torch.equal(ent[i], whole[r][h[r] // m])
        raw = raw_table.cpu().numpy()
        for r in range(R):                              # rows of different blocks: one call each gives the same
            slot = int(raw[r, (h[r] // bs) % cols]) * bs + h[r] % bs
            want, wscale = OC.append(fixed[0][r:r + 1].float().cpu().double().numpy(), [slot], want, wscale)
        want, wscale = OC.append(ent[:len(done)].float().cpu().double().numpy(), live, want, wscale)
        np.testing.assert_array_equal(values(pool), want)
        np.testing.assert_array_equal(scale.cpu().double().numpy(), wscale)
        c = [(t.cpu(), scale.cpu(), tab.cpu()) for t, tab in ((pool, raw_table), (pool, comp_table))]
        check_attn((out, lse), fixed[2].cpu(), torch.arange(R + 1, dtype=torch.int32), torch.tensor(h, dtype=torch.int32), c[0], c[1], W, m,
                   scale_of(D), dtype)
