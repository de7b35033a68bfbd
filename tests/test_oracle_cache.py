"""CPU checks of the serving oracle (oracle/cache.py): against the dense HCA
oracle, against torch's own e4m3 conversion, and by hand."""
import numpy as np
import pytest
import torch

import oracle
from _cache import attn_case, oracle_cache, scale_of, values
from block_sparse_compressed_gb300 import inputs as I
from oracle import cache as OC


def test_e4m3_values_and_rounding_match_the_type():
    codes = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).float().numpy()
    np.testing.assert_array_equal(OC.e4m3_table(), codes.astype(np.float64))
    g = torch.Generator().manual_seed(3)
    x = torch.cat([(torch.rand(4000, generator=g) * 2 - 1) * s for s in (448.0, 8.0, 0.1, 0.01)])
    mids = (OC.e4m3_table()[:126] + OC.e4m3_table()[1:127]) / 2   # every tie
    x = torch.cat([x, torch.from_numpy(mids).float(), torch.from_numpy(-mids).float()])
    np.testing.assert_array_equal(OC.e4m3_round(x.double().numpy()), values(x.to(torch.float8_e4m3fn)))


@pytest.mark.parametrize("W,m,lens", [(8, 4, [40, 17]), (64, 16, [130]), (1, 7, [29, 28])])
def test_attention_over_a_full_cache_is_the_dense_attention(W, m, lens):
    # every token of a request as one step, blocks in any order: the dense
    # oracle on the same rows, one document per request
    H, D, bs = 3, 16, 16
    held = [0] * len(lens)
    q, start, held, raw, comp = attn_case(held, lens, H, D, W, m, bs, torch.float32, 5, ring=False)
    out, lse, _, _ = OC.attend(q.double().numpy(), start.numpy(), held.numpy(), oracle_cache(raw), oracle_cache(comp), W, m,
                               scale_of(D))
    for r, L in enumerate(lens):
        kv = torch.from_numpy(OC._rows(oracle_cache(raw), r, range(L)))[None]
        ck = torch.zeros(1, -(-L // m), D, dtype=torch.float64)
        ck[0, :L // m] = torch.from_numpy(OC._rows(oracle_cache(comp), r, range(L // m)))
        a, b = int(start[r]), int(start[r + 1])
        qr = q[a:b].double().permute(1, 0, 2)[None].contiguous()
        ro, rl = oracle.fwd(qr, kv, ck, None, W, m, scale_of(D))
        np.testing.assert_allclose(out[a:b], np.asarray(ro)[0].transpose(1, 0, 2), atol=1e-12)
        np.testing.assert_allclose(lse[a:b], np.asarray(rl)[0].T, atol=1e-12)


def test_append_by_hand():
    pool, scale = np.zeros((2, 16, 16)), np.array([2.0 ** -8, 2.0 ** -8])
    pool[1, 0] = 448.0          # 1.75
    x = np.zeros((3, 16))
    x[0, 0], x[1, 0], x[2, 0] = 1.75, np.inf, 3.5
    pool, scale = OC.append(x, [2 * 16 - 15, 2 * 16 - 14, 0], pool, scale)
    assert scale.tolist() == [2.0 ** -7, 2.0 ** -8]     # 3.5 = 448 / 128
    assert pool[1, 1, 0] == 448.0 and np.isnan(pool[1, 2, 0]) and pool[0, 0, 0] == 448.0
    pool, scale = OC.append(np.full((1, 16), 1.76), [16 + 3], pool, scale)
    assert scale[1] == 2.0 ** -7 and pool[1, 0, 0] == 224.0 and pool[1, 3, 0] == 224.0
    assert np.isnan(pool[1, 2, 0])


def test_plan_by_hand():
    # cols = 2, bs = 16: request 0 keeps a ring, request 1 starts, request 2 adds nothing
    table = np.array([[5, -1], [-1, -1], [7, 8]], dtype=np.int32)
    start, slots, left, table = OC.plan([15, 0, 32], [40, 3, 0], table, [1, 2, 3, 4], 4, 16, 45, 1)
    assert start == [0, 40, 43, 43] and left == 2
    assert table.tolist() == [[5, 4], [3, -1], [7, 8]]
    # entries 15..54: blocks 0..3 of the request; entries before 32 are overwritten
    assert slots[:17] == [-1] * 17 and slots[17] == 5 * 16 and slots[33] == 4 * 16 and slots[39] == 4 * 16 + 6
    assert slots[40:] == [48, 49, 50, -1, -1]
    assert OC.plan([0], [33], np.full((1, 3), -1), [1, 2], 2, 16, 40, 1) is None
    assert OC.plan([0], [33], np.full((1, 3), -1), [1, 2, 0], 3, 16, 32, 1) is None


def test_chained_steps_hold_the_same_rows_as_one():
    # a prompt in one step or in several gives the same tables and, where no
    # block's scale grows, the same rows
    rng = np.random.default_rng(0)
    x = np.clip(rng.standard_normal((50, 16)), -1.7, 1.7)
    x[::16, 0] = 1.75  # each block's largest comes first
    pools = []
    for steps in ([50], [1] * 50, [20, 13, 17]):
        table, free, left, held = np.full((1, 4), -1), [3, 1, 0, 2], 4, 0
        pool, scale = np.zeros((4, 16, 16)), np.ones(4)
        for n in steps:
            start, slots, left, table = OC.plan([held], [n], table, free, left, 16, n, 1)
            pool, scale = OC.append(x[held:held + n], slots, pool, scale)
            held += n
        pools.append(pool[:, :, :] * scale[:, None, None])
    np.testing.assert_array_equal(pools[0], pools[1])
    np.testing.assert_array_equal(pools[0], pools[2])
