"""What the attention of shared prefixes refuses, on the host before any CUDA call."""
import pytest
import torch

from block_sparse_compressed_gb300 import hca

OK, E_NULL, E_SHAPE, E_DTYPE, E_ALIGN, E_ARG, E_SEG, E_WS, E_UNSUPPORTED = range(9)
P = 1 << 20  # an aligned address; nothing is read


@pytest.fixture(scope="module")
def lib():
    from block_sparse_compressed_gb300 import build
    build.build()
    return hca.load()


def call(lib, **k):
    a = dict(q=P, start=P, held=P, rp=P, rs=P, rt=P, rb=64, rc=4, cp=P, cs=P, ct=P, cb=64, cc=8, first=P, cols=P, out=P, lse=P, N=4, R=3, H=8, D=128,
             G=2, W=128, m=4, bs=16, scale=0.1, dtype=0, ws=P, wsb=1 << 40)
    a.update(k)
    return lib.hca_cache_attn_shared(*a.values(), None)


@pytest.mark.parametrize("change,status", [
    (dict(G=-1), E_SHAPE), (dict(G=257), E_SHAPE), (dict(N=-1), E_SHAPE), (dict(R=-1), E_SHAPE), (dict(H=0), E_SHAPE), (dict(D=0), E_SHAPE),
    (dict(dtype=2), E_DTYPE), (dict(W=0), E_ARG), (dict(m=0), E_ARG), (dict(bs=24), E_ARG), (dict(scale=float("nan")), E_ARG), (dict(rc=0), E_SHAPE),
    (dict(cc=0), E_SHAPE), (dict(cb=-1), E_SHAPE), (dict(first=None), E_NULL), (dict(cols=None), E_NULL), (dict(ct=None), E_NULL),
    (dict(cp=None), E_NULL), (dict(cs=None), E_NULL), (dict(q=None), E_NULL), (dict(out=None), E_NULL), (dict(lse=None), E_NULL),
    (dict(start=None), E_NULL), (dict(held=None), E_NULL), (dict(q=P + 8), E_ALIGN), (dict(out=P + 2), E_ALIGN), (dict(ws=None), E_WS),
    (dict(wsb=4096), E_WS), (dict(ws=P + 16), E_WS)])
@pytest.mark.parametrize("dtype", [0, 1])
def test_refusals(lib, change, status, dtype):
    assert call(lib, **dict(dict(dtype=dtype), **change)) == status


def test_columns_of_the_tensor_cores(lib):
    """bf16 has 64 and 128 columns, as hca_cache_attn; fp32 multiples of 16."""
    assert call(lib, D=96) == E_UNSUPPORTED
    assert lib.hca_cache_attn_shared_workspace_size(4, 3, 8, 96, 2, 0) == 0 < lib.hca_cache_attn_shared_workspace_size(4, 3, 8, 96, 2, 1)


def test_workspace(lib):
    size = lib.hca_cache_attn_shared_workspace_size
    assert size(4, 3, 8, 128, 257, 0) == size(4, 3, 8, 128, -1, 0) == size(4, 3, 8, 128, 2, 2) == 0
    for dtype in (0, 1):
        own = lib.hca_cache_attn_workspace_size(4, 3, 8, 128, dtype)
        need = size(4, 3, 8, 128, 2, dtype)
        assert need >= own > 0
        assert call(lib, dtype=dtype, wsb=need - 1) == E_WS


def test_setting(lib):
    try:
        for v, status in [(0, OK), (1, OK), (2, OK), (3, E_ARG), (-1, E_ARG)]:
            assert lib.hca_test_inject(hca.INJECT_SHARED_PATH, v) == status
    finally:
        lib.hca_test_inject(hca.INJECT_RESET, 0)


def test_binding_refuses():
    q, start, held = torch.zeros(4, 8, 128), torch.zeros(4, dtype=torch.int32), torch.zeros(3, dtype=torch.int32)
    pages = (torch.zeros(8, 16, 128, dtype=torch.float8_e4m3fn), torch.zeros(8), torch.zeros(3, 4, dtype=torch.int32))
    first, cols = torch.zeros(3, dtype=torch.int32), torch.zeros(2, dtype=torch.int32)
    with pytest.raises(ValueError):  # CPU tensors
        hca.hca_cache_attn_shared(q, start, held, pages, pages, first, cols, 128, 4, 0.1)
