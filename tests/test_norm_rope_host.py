"""What the norm and rotation calls refuse, on the host before any CUDA call."""
import ctypes

import pytest
import torch

from block_sparse_compressed_gb300 import hca

OK, E_NULL, E_SHAPE, E_DTYPE, E_ALIGN, E_ARG, E_SEG, E_WS = range(8)
P = 1 << 20  # an aligned address; nothing is read


@pytest.fixture(scope="module")
def lib():
    from block_sparse_compressed_gb300 import build
    build.build()
    return hca.load()


def strides(*v):
    return (ctypes.c_int64 * len(v))(*v)


def fwd(lib, **k):
    a = dict(q=P, qs=None, wq=P, qo=P, kv=P, kvs=None, wkv=P, kvo=P, pos=P, freq=P, start=None, held=None, B=2, H=4, S=8, D=64, R=0, axes=1,
             first=32, rot=32, halves=0, eps=1e-6, dtype=0)
    a.update(k)
    return lib.hca_norm_rope_fwd(*a.values(), None)


def bwd(lib, **k):
    a = dict(q=P, qs=None, wq=P, dqo=P, dq=P, dqs=None, dwq=P, kv=P, kvs=None, wkv=P, dkvo=P, dkv=P, dkvs=None, dwkv=P, pos=P, freq=P,
             B=2, H=4, S=8, D=64, axes=1, first=32, rot=32, halves=0, eps=1e-6, dtype=0, ws=P, wsb=1 << 30)
    a.update(k)
    return lib.hca_norm_rope_bwd(*a.values(), None)


def rope(lib, **k):
    a = dict(x=P, xs=None, y=P, ys=None, pos=P, freq=P, start=None, held=None, B=2, H=4, S=8, D=64, R=0, axes=1, first=0, rot=64, halves=0,
             inverse=0, dtype=0)
    a.update(k)
    return lib.hca_rope(*a.values(), None)


COMMON = [(dict(dtype=2), E_DTYPE), (dict(B=-1), E_SHAPE), (dict(S=-1), E_SHAPE), (dict(H=-1), E_SHAPE), (dict(D=0), E_SHAPE),
          (dict(D=520), E_SHAPE), (dict(D=60), E_ALIGN), (dict(axes=0), E_ARG), (dict(axes=5), E_ARG), (dict(rot=-8), E_ARG),
          (dict(first=-8), E_ARG), (dict(first=40), E_ARG), (dict(first=4, rot=8), E_ARG), (dict(first=0, rot=12), E_ARG),
          (dict(first=0, rot=24, halves=1), E_ARG), (dict(freq=None), E_NULL), (dict(axes=2, pos=None), E_NULL)]


@pytest.mark.parametrize("call", [fwd, bwd, rope])
@pytest.mark.parametrize("change,status", COMMON)
def test_sizes_and_rotation(lib, call, change, status):
    if call is rope and "first" in change and change["first"] == 40:
        change = dict(change, rot=32)
    assert call(lib, **change) == status


@pytest.mark.parametrize("call", [fwd, bwd])
@pytest.mark.parametrize("change,status", [
    (dict(eps=-1.0), E_ARG), (dict(eps=float("nan")), E_ARG), (dict(eps=float("inf")), E_ARG), (dict(q=None), E_NULL),
    (dict(kv=None), E_NULL), (dict(q=P + 2), E_ALIGN), (dict(kv=P + 8), E_ALIGN), (dict(qs=strides(2048, 511, 64)), E_ALIGN),
    (dict(qs=strides(-2048, 512, 64)), E_ALIGN), (dict(kvs=strides(512, 60)), E_ALIGN)])
def test_rows(lib, call, change, status):
    assert call(lib, **change) == status


@pytest.mark.parametrize("call,change,status", [
    (fwd, dict(qo=None), E_NULL), (fwd, dict(kvo=None), E_NULL), (fwd, dict(start=P, held=P, R=1), E_SHAPE),
    (fwd, dict(start=P, held=None, pos=None, R=1, B=1), E_NULL), (fwd, dict(held=P), E_NULL), (fwd, dict(R=-1), E_SHAPE),
    (bwd, dict(dqo=None), E_NULL), (bwd, dict(dkv=None), E_NULL), (bwd, dict(wq=None), E_NULL), (bwd, dict(ws=None), E_WS),
    (bwd, dict(wsb=1000), E_WS), (bwd, dict(ws=P + 16), E_WS), (bwd, dict(dqs=strides(0, 512, 64)), E_ARG),
    (bwd, dict(dqs=strides(2048, 64, 64)), E_ARG), (bwd, dict(dkvs=strides(448, 64)), E_ARG),
    (rope, dict(x=None), E_NULL), (rope, dict(y=None), E_NULL), (rope, dict(ys=strides(2048, 256, 64)), E_ARG),
    (rope, dict(y=P + 4), E_ALIGN)])
def test_results(lib, call, change, status):
    assert call(lib, **change) == status


def test_nothing_to_do(lib):
    assert fwd(lib, S=0) == OK and rope(lib, B=0) == OK and rope(lib, H=0) == OK
    assert fwd(lib, q=None, qo=None, kv=None, kvo=None) == OK
    assert fwd(lib, B=1, start=P, held=P, R=0) == OK
    assert lib.hca_norm_rope_workspace_size(128) > 0 == lib.hca_norm_rope_workspace_size(0) == lib.hca_norm_rope_workspace_size(513)


def test_binding_refuses():
    q, kv, f = torch.zeros(1, 2, 4, 64), torch.zeros(1, 4, 64), torch.zeros(16)
    start, held = torch.zeros(2, dtype=torch.int32), torch.zeros(1, dtype=torch.int32)
    with pytest.raises(ValueError):  # CPU tensors
        hca.hca_norm_rope_fwd(q, kv, None, None, None, f, 1e-6)
    with pytest.raises(ValueError):
        hca.hca_rope(q, None, f)
    with pytest.raises(ValueError):
        hca.hca_norm_rope_fwd(None, None, None, None, None, f, 1e-6)
    with pytest.raises(ValueError):
        hca.hca_norm_rope_bwd(q[0], kv, None, None, None, f, 1e-6, q, kv)
    with pytest.raises(ValueError):
        hca.hca_cache_norm_rope(q[0], kv[0], start, None, None, None, f, 1e-6)
    with pytest.raises(ValueError):
        hca.hca_cache_rope(q, start, held, f)
    with pytest.raises(ValueError):
        hca.hca_cache_rope(q[0], start, held, f)
