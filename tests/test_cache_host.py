"""Host-side checks of the serving calls: argument errors are found before any
CUDA call, so fake addresses are fine and no GPU is needed."""
import ctypes

import pytest
import torch

from block_sparse_compressed_gb300 import hca

OK, E_NULL, E_SHAPE, E_DTYPE, E_ALIGN, E_ARG, E_SEG, E_WS, E_UNSUP, E_CUDA, E_TIME, E_CAP, E_CACHE = range(13)
P = lambda v: None if v is None else ctypes.c_void_p(v)  # noqa: E731


@pytest.fixture(scope="module")
def lib():
    from block_sparse_compressed_gb300 import build
    build.build()
    return hca.load()


def test_status_strings(lib):
    for s in (E_CAP, E_CACHE):
        assert hca.hca_status_string(s).startswith("HCA_ERR_CA")


def _plan(lib, **kw):
    a = dict(held=16, added=16, table=16, free=16, fin=16, fout=16, start=16, slots=16, R=4, cols=2, bs=16, m=1, nblocks=8,
             nfree=8, nslots=10, ws=256, wsb=512)
    a.update(kw)
    return lib.hca_cache_plan(*[P(a[k]) for k in ("held", "added", "table", "free", "fin", "fout", "start", "slots")],
                              a["R"], a["cols"], a["bs"], a["m"], a["nblocks"], a["nfree"], a["nslots"], P(a["ws"]),
                              a["wsb"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(R=-1), E_SHAPE), (dict(cols=0), E_SHAPE), (dict(nslots=-1), E_SHAPE), (dict(nfree=-1), E_SHAPE),
    (dict(nblocks=1 << 28), E_SHAPE), (dict(bs=24), E_ARG), (dict(bs=256), E_ARG), (dict(m=0), E_ARG),
    (dict(held=None), E_NULL), (dict(added=None), E_NULL), (dict(table=None), E_NULL), (dict(free=None), E_NULL),
    (dict(fin=None), E_NULL), (dict(fout=None), E_NULL), (dict(start=None), E_NULL), (dict(slots=None), E_NULL),
    (dict(ws=None), E_WS), (dict(ws=128), E_WS), (dict(wsb=256), E_WS),
])
def test_plan_refusals(lib, kw, want):
    assert _plan(lib, **kw) == want


def _append(lib, **kw):
    a = dict(x=16, slots=16, pool=16, scale=16, N=4, D=128, bs=64, nblocks=8, dt=0, ws=256, wsb=1 << 20)
    a.update(kw)
    return lib.hca_cache_append(P(a["x"]), P(a["slots"]), P(a["pool"]), P(a["scale"]), a["N"], a["D"], a["bs"],
                                a["nblocks"], a["dt"], P(a["ws"]), a["wsb"], None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=2), E_DTYPE), (dict(N=-1), E_SHAPE), (dict(D=0), E_SHAPE), (dict(D=272), E_SHAPE), (dict(D=24), E_ALIGN),
    (dict(nblocks=-1), E_SHAPE), (dict(nblocks=1 << 25), E_SHAPE), (dict(bs=48), E_ARG), (dict(x=None), E_NULL),
    (dict(slots=None), E_NULL), (dict(pool=None), E_NULL), (dict(scale=None), E_NULL), (dict(x=24), E_ALIGN),
    (dict(pool=8), E_ALIGN), (dict(ws=None), E_WS), (dict(wsb=256), E_WS),
])
def test_append_refusals(lib, kw, want):
    assert _append(lib, **kw) == want


def _attn(lib, **kw):
    a = dict(q=16, start=16, held=16, rp=16, rs=16, rt=16, rb=8, rc=4, cp=16, cs=16, ct=16, cb=8, cc=4, out=16, lse=16, N=4,
             R=4, H=64, D=128, W=128, m=128, bs=64, scale=0.1, dt=0, ws=256, wsb=1 << 30)
    a.update(kw)
    return lib.hca_cache_attn(P(a["q"]), P(a["start"]), P(a["held"]), P(a["rp"]), P(a["rs"]), P(a["rt"]), a["rb"], a["rc"],
                              P(a["cp"]), P(a["cs"]), P(a["ct"]), a["cb"], a["cc"], P(a["out"]), P(a["lse"]), a["N"],
                              a["R"], a["H"], a["D"], a["W"], a["m"], a["bs"], a["scale"], a["dt"], P(a["ws"]), a["wsb"],
                              None)


@pytest.mark.parametrize("kw,want", [
    (dict(dt=3), E_DTYPE), (dict(N=-1), E_SHAPE), (dict(R=-1), E_SHAPE), (dict(H=0), E_SHAPE), (dict(H=1 << 15), E_SHAPE),
    (dict(D=512), E_SHAPE), (dict(D=40), E_ALIGN), (dict(D=96), E_UNSUP), (dict(D=256), E_UNSUP), (dict(W=0), E_ARG),
    (dict(m=0), E_ARG), (dict(bs=8), E_ARG), (dict(scale=float("nan")), E_ARG), (dict(scale=float("inf")), E_ARG),
    (dict(rb=-1), E_SHAPE), (dict(rc=0), E_SHAPE), (dict(cb=-1), E_SHAPE), (dict(cc=0), E_SHAPE),
    (dict(rb=1 << 25), E_SHAPE), (dict(cb=1 << 25), E_SHAPE), (dict(q=None), E_NULL), (dict(start=None), E_NULL),
    (dict(held=None), E_NULL), (dict(rp=None), E_NULL), (dict(rs=None), E_NULL), (dict(rt=None), E_NULL),
    (dict(cp=None), E_NULL), (dict(cs=None), E_NULL), (dict(out=None), E_NULL), (dict(lse=None), E_NULL),
    (dict(q=20), E_ALIGN), (dict(out=20), E_ALIGN), (dict(rp=20), E_ALIGN), (dict(cp=20), E_ALIGN), (dict(ws=None), E_WS),
    (dict(wsb=4096), E_WS), (dict(ct=None, cp=None, cs=None, cb=0, cc=0, wsb=4096), E_WS), (dict(D=96, dt=1, wsb=4096), E_WS),
])
def test_attn_refusals(lib, kw, want):
    assert _attn(lib, **kw) == want


def test_workspace_sizes(lib):
    f = lib.hca_cache_attn_workspace_size
    assert f(64, 64, 64, 128, 0) > 0 and f(64, 64, 64, 96, 0) == 0 and f(64, 64, 64, 96, 1) > 0
    assert f(64, 64, 0, 128, 0) == 0 and f(64, 64, 64, 128, 5) == 0 and f(-1, 64, 64, 128, 0) == 0
    # grows with the tokens, not with the cache
    assert f(65536, 4, 64, 128, 0) < f(256, 4, 64, 128, 0) + 65536 * 128
    assert lib.hca_cache_append_workspace_size(1000) >= 4000 and lib.hca_cache_append_workspace_size(-1) == 0
    assert lib.hca_cache_plan_workspace_size(1000) >= 4000 and lib.hca_cache_plan_workspace_size(-1) == 0


def test_binding_checks_tensors():
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    pool, scale = torch.zeros(4, 16, 64).to(torch.float8_e4m3fn), torch.ones(4)
    with pytest.raises(TypeError):
        hca.hca_cache_append(torch.zeros(3, 64, dtype=torch.float16), i32(3), pool, scale)
    with pytest.raises(ValueError):
        hca.hca_cache_append(torch.zeros(3, 32), i32(3), pool, scale)
    with pytest.raises(ValueError):
        hca.hca_cache_append(torch.zeros(64, 3).T, i32(3), pool, scale)   # strided rows
    with pytest.raises(TypeError):
        hca.hca_cache_append(torch.zeros(3, 64), i32(3).long(), pool, scale)
    with pytest.raises(TypeError):
        hca.hca_cache_append(torch.zeros(3, 64), i32(3), pool.view(torch.uint8), scale)
    with pytest.raises(ValueError):
        hca.hca_cache_plan(i32(3), i32(4), i32(3, 2), i32(5), i32(1), 8, 16, 4)
    q = torch.zeros(2, 4, 64)
    with pytest.raises(ValueError):
        hca.hca_cache_attn(q, i32(2), i32(2), (pool, scale, i32(2, 3)), None, 8, 4, 0.1)
    with pytest.raises(ValueError):
        hca.hca_cache_attn(q, i32(3), i32(2), (pool, scale, i32(1, 3)), None, 8, 4, 0.1)
    other = torch.zeros(4, 32, 64).to(torch.float8_e4m3fn)
    with pytest.raises(ValueError):
        hca.hca_cache_attn(q, i32(3), i32(2), (pool, scale, i32(2, 3)), (other, scale, i32(2, 3)), 8, 4, 0.1)


def test_the_short_way_declines_what_is_not_ordinary():
    # tensors of the CPU, of other types and shapes, no tensors at all: None, and nothing done
    hca.load()
    if hca._py is None:
        pytest.skip("built without the headers of Python or torch")
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    pool, scale, x = torch.zeros(4, 16, 64).to(torch.float8_e4m3fn), torch.ones(4), torch.zeros(3, 64)
    for a in ((x, i32(3), pool, scale, None, False), (None, i32(3), pool, scale, None, False), (x, 3, pool, scale, None, False), (x,),
              (x[0], i32(3), pool, scale, None, False), (x, i32(3), pool[0], scale, None, False), (x.half(), i32(3), pool, scale, None, False)):
        assert hca._py.cache_append(*a) is None
    assert hca._py.cache_plan(i32(3), i32(3), i32(3, 2), i32(5), i32(1), 8, 16, 4, 1, None, None, None, None, False) is None
    assert hca._py.cache_plan(i32(3), i32(3), i32(3, 2), i32(5), i32(1), 8.0, 16, 4, 1, None, None, None, None, False) is None
    c = (pool, scale, i32(2, 3))
    for raw, comp in ((c, None), (c, c), (list(c), None), (c[:2], None), (None, c)):
        assert hca._py.cache_attn(torch.zeros(2, 4, 64), i32(3), i32(2), raw, comp, 8, 4, 0.1, None, None, None, False) is None
    assert hca._py.cache_attn(torch.zeros(2, 4, 64), i32(3), i32(2), c, None, 1 << 40, 4, 0.1, None, None, None, False) is None


def test_the_binding_refuses_other_devices_and_workspaces():
    # nothing of a CPU tensor or a foreign workspace reaches the device
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    pool, scale, x = torch.zeros(4, 16, 64).to(torch.float8_e4m3fn), torch.ones(4), torch.zeros(3, 64)
    ws = torch.zeros(1 << 20, dtype=torch.uint8)
    c = (pool, scale, i32(2, 3))
    calls = (lambda **k: hca.hca_cache_append(x, i32(3), pool, scale, **k),
             lambda **k: hca.hca_cache_plan(i32(3), i32(3), i32(3, 2), i32(5), i32(1), 8, 16, 4, **k),
             lambda **k: hca.hca_cache_attn(torch.zeros(2, 4, 64), i32(3), i32(2), c, None, 8, 4, 0.1, **k))
    for call in calls:
        with pytest.raises(ValueError, match="CUDA"):
            call(ws=ws)
        with pytest.raises(ValueError, match="ws is on"):
            call(ws=torch.empty(1 << 20, dtype=torch.uint8, device="meta"))
        with pytest.raises(TypeError):
            call(ws=ws.float())
        with pytest.raises(ValueError, match="contiguous"):
            call(ws=ws[::2])


@pytest.mark.parametrize("kw,status", [(dict(nblocks=(1 << 32) + 8), E_SHAPE), (dict(bs=(1 << 32) + 16), E_ARG), (dict(m=1 - (1 << 32)), E_ARG),
                                       (dict(nblocks=8 - (1 << 32)), E_SHAPE)])
def test_plan_refuses_numbers_beyond_32_bits(kw, status, monkeypatch):
    # each is an ordinary number in its lower 32 bits
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    monkeypatch.setattr(hca, "_enqueue", lambda dev, f, *a: f(*a, None))   # refused in front of any CUDA call
    a = dict(dict(nblocks=8, bs=16, m=1), **kw)
    with pytest.raises(hca.HCAError) as e:
        hca.hca_cache_plan(i32(3), i32(3), i32(3, 2), i32(5), i32(1), a["nblocks"], a["bs"], 4, m=a["m"])
    assert e.value.status == status


@pytest.mark.parametrize("W,m", [(5 - (1 << 32), 4), (5, 4 - (1 << 32)), (-(1 << 40), 4), (5, -(1 << 31) - 1)])
def test_attention_refuses_numbers_beyond_32_bits(W, m, monkeypatch):
    i32 = lambda *s: torch.zeros(*s, dtype=torch.int32)  # noqa: E731
    monkeypatch.setattr(hca, "_enqueue", lambda dev, f, *a: f(*a, None))
    c = (torch.zeros(4, 16, 64).to(torch.float8_e4m3fn), torch.ones(4), i32(2, 3))
    with pytest.raises(hca.HCAError) as e:
        hca.hca_cache_attn(torch.zeros(2, 4, 64), i32(3), i32(2), c, c, W, m, 0.1)
    assert e.value.status == E_ARG
