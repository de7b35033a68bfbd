"""Thin Python binding of libhca (the C ABI declared in include/hca.h).

Argument marshalling only: every entry point checks tensor dtypes/shapes,
allocates outputs and workspace through PyTorch (device memory is torch's),
passes raw pointers, sizes and torch's current CUDA stream to the C function
of the same name, and turns a non-zero status into an exception.  All of the
computation runs in libhca's CUDA kernels; there is no fallback of any kind,
and a missing library is an error.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import os
import threading
from typing import Optional, Tuple

import torch

_HERE = os.path.dirname(os.path.abspath(__file__))
LIB_PATH = os.path.join(_HERE, "libhca.so")

HCA_BF16, HCA_F32 = 0, 1
_DTYPES = {torch.bfloat16: HCA_BF16, torch.float32: HCA_F32}

_lock = threading.Lock()
_lib = None
_py = None  # the serving calls' short way (csrc/hca_py.cpp)

EXPORTS = ("hca_status_string", "hca_version", "hca_workspace_size", "hca_query_tile_positions", "hca_attn_fwd",
           "hca_attn_bwd", "hca_visible_pairs", "hca_tile_map", "hca_workspace_status", "hca_profile_enable",
           "hca_profile_read", "hca_num_kernels", "hca_kernel_name", "hca_attn_fwd_noalloc",
           "hca_local_workspace_size", "hca_local_attn_fwd", "hca_local_attn_bwd", "hca_test_inject",
           "hca_compress_fwd", "hca_compress_workspace_size", "hca_compress_bwd", "hca_indexer_workspace_size",
           "hca_indexer_topk", "hca_csa_workspace_size", "hca_csa_attn_fwd", "hca_csa_attn_bwd",
           "hca_cache_plan_workspace_size", "hca_cache_plan", "hca_cache_append_workspace_size", "hca_cache_append",
           "hca_cache_attn_workspace_size", "hca_cache_attn", "hca_norm_rope_fwd", "hca_norm_rope_workspace_size",
           "hca_norm_rope_bwd", "hca_rope", "hca_cache_attn_shared_workspace_size", "hca_cache_attn_shared")

# failure-path test hooks (hca_test_inject)
INJECT_RESET, INJECT_LAUNCH_FAILURE, INJECT_STALL, INJECT_WAIT_LIMIT_NS, INJECT_CSA_UNION, INJECT_SHARED_PATH = 0, 1, 2, 3, 4, 5


class HCAError(RuntimeError):
    def __init__(self, status: int, where: str):
        self.status = status
        super().__init__(f"{where}: {hca_status_string(status)}")


def _extension():
    """The extension module, or None: not built (no host compiler, no headers of
    Python or torch), or built with another torch."""
    try:
        from . import _hca_py as py
    except ImportError:
        return None
    return py if getattr(py, "torch_version", None) == torch.__version__ else None


def load(path: str = LIB_PATH):
    """Load libhca.so and declare the C signatures (no CUDA call is made)."""
    global _lib, _py
    with _lock:
        if _lib is None:
            if not os.path.exists(path):
                raise RuntimeError(f"libhca.so is not built ({path}); run "
                                   "`python -m block_sparse_compressed_gb300.build`")
            lib = ctypes.CDLL(path)
            P, I, F, Z = ctypes.c_void_p, ctypes.c_int, ctypes.c_float, ctypes.c_size_t
            lib.hca_status_string.argtypes = [I]
            lib.hca_status_string.restype = ctypes.c_char_p
            lib.hca_version.argtypes = []
            lib.hca_version.restype = I
            lib.hca_workspace_size.argtypes = [I, I, I, I, I, I, I, I]
            lib.hca_workspace_size.restype = Z
            lib.hca_query_tile_positions.argtypes = [I, I, I]
            lib.hca_query_tile_positions.restype = I
            lib.hca_attn_fwd.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, F, I, P, Z, P]
            lib.hca_attn_fwd.restype = I
            lib.hca_attn_bwd.argtypes = [P, P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, F, I, P, Z, P]
            lib.hca_attn_bwd.restype = I
            lib.hca_visible_pairs.argtypes = [P, I, I, I, I, P, P, P, Z, P]
            lib.hca_visible_pairs.restype = I
            lib.hca_tile_map.argtypes = [P, I, I, I, I, I, P, P, Z, P]
            lib.hca_tile_map.restype = I
            lib.hca_workspace_status.argtypes = [P, P]
            lib.hca_workspace_status.restype = I
            lib.hca_profile_enable.argtypes = [I]
            lib.hca_profile_enable.restype = I
            lib.hca_profile_read.argtypes = [I, ctypes.POINTER(ctypes.c_longlong), ctypes.POINTER(ctypes.c_double)]
            lib.hca_profile_read.restype = I
            lib.hca_num_kernels.argtypes = []
            lib.hca_num_kernels.restype = I
            lib.hca_kernel_name.argtypes = [I]
            lib.hca_kernel_name.restype = ctypes.c_char_p
            lib.hca_attn_fwd_noalloc.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, F, I, P]
            lib.hca_attn_fwd_noalloc.restype = I
            lib.hca_local_workspace_size.argtypes = [I, I, I, I, I, I, I]
            lib.hca_local_workspace_size.restype = Z
            lib.hca_local_attn_fwd.argtypes = [P, P, P, P, P, I, I, I, I, I, F, I, P, Z, P]
            lib.hca_local_attn_fwd.restype = I
            lib.hca_local_attn_bwd.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, F, I, P, Z, P]
            lib.hca_local_attn_bwd.restype = I
            lib.hca_test_inject.argtypes = [I, ctypes.c_longlong]
            lib.hca_test_inject.restype = I
            lib.hca_compress_fwd.argtypes = [P, P, P, P, P, I, I, I, I, I, P]
            lib.hca_compress_fwd.restype = I
            lib.hca_compress_workspace_size.argtypes = [I, I, I]
            lib.hca_compress_workspace_size.restype = Z
            lib.hca_compress_bwd.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, P, Z, P]
            lib.hca_compress_bwd.restype = I
            lib.hca_indexer_workspace_size.argtypes = [I, I, I]
            lib.hca_indexer_workspace_size.restype = Z
            lib.hca_indexer_topk.argtypes = [P, P, P, P, P, P, I, I, I, I, I, I, P, Z, P]
            lib.hca_indexer_topk.restype = I
            lib.hca_csa_workspace_size.argtypes = [I, I, I, I, I, I, I, I, I]
            lib.hca_csa_workspace_size.restype = Z
            lib.hca_csa_attn_fwd.argtypes = [P, P, P, P, P, P, P, I, I, I, I, I, I, I, F, I, P, Z, P]
            lib.hca_csa_attn_fwd.restype = I
            lib.hca_csa_attn_bwd.argtypes = [P, P, P, P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, F, I, P, Z, P]
            lib.hca_csa_attn_bwd.restype = I
            lib.hca_cache_plan_workspace_size.argtypes = [I]
            lib.hca_cache_plan_workspace_size.restype = Z
            lib.hca_cache_plan.argtypes = [P, P, P, P, P, P, P, P, I, I, I, I, I, I, I, P, Z, P]
            lib.hca_cache_plan.restype = I
            lib.hca_cache_append_workspace_size.argtypes = [I]
            lib.hca_cache_append_workspace_size.restype = Z
            lib.hca_cache_append.argtypes = [P, P, P, P, I, I, I, I, I, P, Z, P]
            lib.hca_cache_append.restype = I
            lib.hca_cache_attn_workspace_size.argtypes = [I, I, I, I, I]
            lib.hca_cache_attn_workspace_size.restype = Z
            lib.hca_cache_attn.argtypes = [P, P, P, P, P, P, I, I, P, P, P, I, I, P, P, I, I, I, I, I, I, I, F, I, P, Z, P]
            lib.hca_cache_attn.restype = I
            lib.hca_norm_rope_fwd.argtypes = [P] * 12 + [I] * 9 + [F, I, P]
            lib.hca_norm_rope_fwd.restype = I
            lib.hca_norm_rope_workspace_size.argtypes = [I]
            lib.hca_norm_rope_workspace_size.restype = Z
            lib.hca_norm_rope_bwd.argtypes = [P] * 16 + [I] * 8 + [F, I, P, Z, P]
            lib.hca_norm_rope_bwd.restype = I
            lib.hca_rope.argtypes = [P] * 8 + [I] * 11 + [P]
            lib.hca_rope.restype = I
            lib.hca_cache_attn_shared_workspace_size.argtypes = [I, I, I, I, I, I]
            lib.hca_cache_attn_shared_workspace_size.restype = Z
            lib.hca_cache_attn_shared.argtypes = [P, P, P, P, P, P, I, I, P, P, P, I, I, P, P, P, P, I, I, I, I, I, I, I, I, F, I, P, Z, P]
            lib.hca_cache_attn_shared.restype = I
            py = _extension()
            if py is not None:
                py.bind(*(ctypes.cast(getattr(lib, f), P).value for f in (
                    "hca_cache_plan_workspace_size", "hca_cache_plan", "hca_cache_append_workspace_size",
                    "hca_cache_append", "hca_cache_attn_workspace_size", "hca_cache_attn", "hca_cache_attn_shared_workspace_size",
                    "hca_cache_attn_shared", "hca_norm_rope_fwd", "hca_norm_rope_workspace_size", "hca_norm_rope_bwd", "hca_rope")))
                _py = py
            _lib = lib
    return _lib


def hca_status_string(status: int) -> str:
    return load().hca_status_string(int(status)).decode()


def hca_version() -> int:
    return load().hca_version()


def _dtype_code(t: torch.Tensor) -> int:
    if t.dtype not in _DTYPES:
        raise TypeError(f"unsupported dtype {t.dtype}; use bfloat16 or float32")
    return _DTYPES[t.dtype]


def _ptr(t: Optional[torch.Tensor]):
    return None if t is None else ctypes.c_void_p(t.data_ptr())


def _stream(device) -> ctypes.c_void_p:
    return ctypes.c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _on(device):
    """Make `device` the current CUDA device for the C call: the library
    resolves per-device state (kernel attributes, the built-in scratch of the
    no-allocation entry point) on the current device."""
    device = torch.device(device)
    return torch.cuda.device(device) if device.type == "cuda" else contextlib.nullcontext()


def _check(rc: int, where: str):
    if rc != 0:
        raise HCAError(rc, where)


def _need(t: torch.Tensor, name: str, shape, dtype, device):
    if t is None:
        raise ValueError(f"{name} is required")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")


def hca_workspace_size(B: int, H: int, S: int, D: int, W: int, m: int, dtype: torch.dtype,
                       for_backward: bool) -> int:
    return load().hca_workspace_size(B, H, S, D, W, m, _DTYPES[dtype], int(for_backward))


def hca_query_tile_positions(H: int, D: int, dtype: torch.dtype) -> int:
    return load().hca_query_tile_positions(H, D, _DTYPES[dtype])


def workspace(B, H, S, D, W, m, dtype, for_backward, device) -> torch.Tensor:
    n = hca_workspace_size(B, H, S, D, W, m, dtype, for_backward)
    if n == 0:
        raise ValueError("invalid sizes for hca_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def hca_workspace_status(ws: torch.Tensor) -> int:
    """Synchronise the current stream and return the device-recorded status."""
    with _on(ws.device):
        return load().hca_workspace_status(_ptr(ws), _stream(ws.device))


def hca_test_inject(what: int, value: int = 0) -> None:
    """Failure-path test hook (include/hca.h, hca_test_inject)."""
    _check(load().hca_test_inject(int(what), int(value)), "hca_test_inject")


def _shapes(q, kv, ckv, seg, m):
    if q.dim() != 4:
        raise ValueError("q must be [B,H,S,D]")
    B, H, S, D = q.shape
    Sc = -(-S // m)
    dev = q.device
    _need(kv, "kv", (B, S, D), q.dtype, dev)
    _need(ckv, "ckv", (B, Sc, D), q.dtype, dev)
    if seg is not None:
        _need(seg, "seg", (B, S), torch.int32, dev)
    return B, H, S, D, Sc


def hca_attn_fwd(q: torch.Tensor, kv: torch.Tensor, ckv: torch.Tensor, seg: Optional[torch.Tensor], W: int,
                 m: int, scale: float, out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                 ws: Optional[torch.Tensor] = None, check: bool = False) -> Tuple[torch.Tensor, torch.Tensor]:
    """HCA forward: returns (out[B,H,S,D], lse[B,H,S] fp32)."""
    lib = load()
    if m < 1:
        raise ValueError("m must be >= 1")
    B, H, S, D, Sc = _shapes(q, kv, ckv, seg, m)
    _need(q, "q", q.shape, q.dtype, q.device)
    dt = _dtype_code(q)
    if out is None:
        out = torch.empty_like(q)
    if lse is None:
        lse = torch.empty(B, H, S, dtype=torch.float32, device=q.device)
    _need(out, "out", q.shape, q.dtype, q.device)
    _need(lse, "lse", (B, H, S), torch.float32, q.device)
    if ws is None:
        ws = workspace(B, H, S, D, W, m, q.dtype, False, q.device)
    with _on(q.device):
        rc = lib.hca_attn_fwd(_ptr(q), _ptr(kv), _ptr(ckv), _ptr(seg), _ptr(out), _ptr(lse), B, H, S, D, W, m,
                              float(scale), dt, _ptr(ws), ws.numel(), _stream(q.device))
    _check(rc, "hca_attn_fwd")
    if check:
        _check(hca_workspace_status(ws), "hca_attn_fwd (device)")
    return out, lse


def hca_attn_bwd(q, kv, ckv, seg, out, lse, dout, W: int, m: int, scale: float, dq=None, dkv=None, dckv=None,
                 ws=None, check: bool = False):
    """HCA backward: returns (dq[B,H,S,D], dkv[B,S,D], dckv[B,Sc,D])."""
    lib = load()
    if m < 1:
        raise ValueError("m must be >= 1")
    B, H, S, D, Sc = _shapes(q, kv, ckv, seg, m)
    _need(q, "q", q.shape, q.dtype, q.device)
    _need(out, "out", q.shape, q.dtype, q.device)
    _need(dout, "dout", q.shape, q.dtype, q.device)
    _need(lse, "lse", (B, H, S), torch.float32, q.device)
    dt = _dtype_code(q)
    dq = torch.empty_like(q) if dq is None else dq
    dkv = torch.empty_like(kv) if dkv is None else dkv
    dckv = torch.empty_like(ckv) if dckv is None else dckv
    _need(dq, "dq", q.shape, q.dtype, q.device)
    _need(dkv, "dkv", kv.shape, q.dtype, q.device)
    _need(dckv, "dckv", ckv.shape, q.dtype, q.device)
    if ws is None:
        ws = workspace(B, H, S, D, W, m, q.dtype, True, q.device)
    with _on(q.device):
        rc = lib.hca_attn_bwd(_ptr(q), _ptr(kv), _ptr(ckv), _ptr(seg), _ptr(out), _ptr(lse), _ptr(dout), _ptr(dq),
                              _ptr(dkv), _ptr(dckv), B, H, S, D, W, m, float(scale), dt, _ptr(ws), ws.numel(),
                              _stream(q.device))
    _check(rc, "hca_attn_bwd")
    if check:
        _check(hca_workspace_status(ws), "hca_attn_bwd (device)")
    return dq, dkv, dckv


def hca_local_workspace_size(B: int, H: int, S: int, D: int, W: int, dtype: torch.dtype, for_backward: bool) -> int:
    return load().hca_local_workspace_size(B, H, S, D, W, _DTYPES[dtype], int(for_backward))


def local_workspace(B, H, S, D, W, dtype, for_backward, device) -> torch.Tensor:
    n = hca_local_workspace_size(B, H, S, D, W, dtype, for_backward)
    if n == 0:
        raise ValueError("invalid sizes for hca_local_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def _local_shapes(q, kv, seg):
    if q.dim() != 4:
        raise ValueError("q must be [B,H,S,D]")
    B, H, S, D = q.shape
    _need(kv, "kv", (B, S, D), q.dtype, q.device)
    if seg is not None:
        _need(seg, "seg", (B, S), torch.int32, q.device)
    return B, H, S, D


def hca_local_attn_fwd(q, kv, seg, W: int, scale: float, out=None, lse=None, ws=None, check: bool = False):
    """Local sliding-window attention forward: returns (out, lse)."""
    lib = load()
    B, H, S, D = _local_shapes(q, kv, seg)
    dt = _dtype_code(q)
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty(B, H, S, dtype=torch.float32, device=q.device) if lse is None else lse
    _need(out, "out", q.shape, q.dtype, q.device)
    _need(lse, "lse", (B, H, S), torch.float32, q.device)
    if ws is None:
        ws = local_workspace(B, H, S, D, W, q.dtype, False, q.device)
    with _on(q.device):
        rc = lib.hca_local_attn_fwd(_ptr(q), _ptr(kv), _ptr(seg), _ptr(out), _ptr(lse), B, H, S, D, W, float(scale), dt,
                                    _ptr(ws), ws.numel(), _stream(q.device))
    _check(rc, "hca_local_attn_fwd")
    if check:
        _check(hca_workspace_status(ws), "hca_local_attn_fwd (device)")
    return out, lse


def hca_local_attn_bwd(q, kv, seg, out, lse, dout, W: int, scale: float, dq=None, dkv=None, ws=None,
                       check: bool = False):
    """Local sliding-window attention backward: returns (dq, dkv)."""
    lib = load()
    B, H, S, D = _local_shapes(q, kv, seg)
    _need(out, "out", q.shape, q.dtype, q.device)
    _need(dout, "dout", q.shape, q.dtype, q.device)
    _need(lse, "lse", (B, H, S), torch.float32, q.device)
    dt = _dtype_code(q)
    dq = torch.empty_like(q) if dq is None else dq
    dkv = torch.empty_like(kv) if dkv is None else dkv
    _need(dq, "dq", q.shape, q.dtype, q.device)
    _need(dkv, "dkv", kv.shape, q.dtype, q.device)
    if ws is None:
        ws = local_workspace(B, H, S, D, W, q.dtype, True, q.device)
    with _on(q.device):
        rc = lib.hca_local_attn_bwd(_ptr(q), _ptr(kv), _ptr(seg), _ptr(out), _ptr(lse), _ptr(dout), _ptr(dq), _ptr(dkv),
                                    B, H, S, D, W, float(scale), dt, _ptr(ws), ws.numel(), _stream(q.device))
    _check(rc, "hca_local_attn_bwd")
    if check:
        _check(hca_workspace_status(ws), "hca_local_attn_bwd (device)")
    return dq, dkv


def hca_visible_pairs(seg: Optional[torch.Tensor], B: int, S: int, W: int, m: int, device=None):
    """(raw_pairs[B], comp_pairs[B]) int64 device tensors."""
    lib = load()
    device = seg.device if seg is not None else torch.device(device or "cuda")
    raw = torch.empty(B, dtype=torch.int64, device=device)
    comp = torch.empty(B, dtype=torch.int64, device=device)
    ws = workspace(B, 1, S, 16, W, m, torch.float32, False, device)
    with _on(device):
        rc = lib.hca_visible_pairs(_ptr(seg), B, S, W, m, _ptr(raw), _ptr(comp), _ptr(ws), ws.numel(), _stream(device))
    _check(rc, "hca_visible_pairs")
    return raw, comp


def hca_tile_map(seg: Optional[torch.Tensor], B: int, S: int, W: int, m: int, Pq: int, device=None):
    """int32 [B, ceil(S/Pq), 4] device tensor of per-tile key ranges."""
    lib = load()
    device = seg.device if seg is not None else torch.device(device or "cuda")
    nt = -(-S // Pq)
    out = torch.empty(B, nt, 4, dtype=torch.int32, device=device)
    ws = workspace(B, 1, S, 16, W, m, torch.float32, False, device)
    with _on(device):
        rc = lib.hca_tile_map(_ptr(seg), B, S, W, m, Pq, _ptr(out), _ptr(ws), ws.numel(), _stream(device))
    _check(rc, "hca_tile_map")
    return out


def hca_profile_enable(on: bool = True) -> None:
    _check(load().hca_profile_enable(int(on)), "hca_profile_enable")


def hca_profile_read() -> dict:
    """{kernel name: (launches, total_ms)} since the last enable (syncs)."""
    lib = load()
    res = {}
    for k in range(lib.hca_num_kernels()):
        n, ms = ctypes.c_longlong(0), ctypes.c_double(0.0)
        _check(lib.hca_profile_read(k, ctypes.byref(n), ctypes.byref(ms)), "hca_profile_read")
        res[lib.hca_kernel_name(k).decode()] = (int(n.value), float(ms.value))
    return res


NOALLOC_MAX_POSITIONS = 1 << 20


def hca_attn_fwd_noalloc(q, kv, ckv, seg, W: int, m: int, scale: float, out=None, lse=None):
    """Forward through the entry point that uses the library's built-in
    scratch instead of a workspace (for callers that cannot allocate device
    memory; B*S <= NOALLOC_MAX_POSITIONS).  Returns (out, lse)."""
    lib = load()
    if m < 1:
        raise ValueError("m must be >= 1")
    B, H, S, D, Sc = _shapes(q, kv, ckv, seg, m)
    _need(q, "q", q.shape, q.dtype, q.device)
    dt = _dtype_code(q)
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty(B, H, S, dtype=torch.float32, device=q.device) if lse is None else lse
    _need(out, "out", q.shape, q.dtype, q.device)
    _need(lse, "lse", (B, H, S), torch.float32, q.device)
    with _on(q.device):
        rc = lib.hca_attn_fwd_noalloc(_ptr(q), _ptr(kv), _ptr(ckv), _ptr(seg), _ptr(out), _ptr(lse), B, H, S, D, W, m,
                                      float(scale), dt, _stream(q.device))
    _check(rc, "hca_attn_fwd_noalloc")
    return out, lse


def hca_compress_fwd(x: torch.Tensor, g: torch.Tensor, bias: torch.Tensor, seg: Optional[torch.Tensor], m: int,
                     ckv: Optional[torch.Tensor] = None) -> torch.Tensor:
    """HCA compressor: ckv[B, ceil(S/m), D] from x[B,S,D], gates g[B,S] fp32,
    block bias[m] fp32 (include/hca.h, hca_compress_fwd)."""
    lib = load()
    B, S, D = x.shape
    Sc = -(-S // m)
    dev = x.device
    _need(x, "x", (B, S, D), x.dtype, dev)
    _need(g, "g", (B, S), torch.float32, dev)
    _need(bias, "bias", (m,), torch.float32, dev)
    if seg is not None:
        _need(seg, "seg", (B, S), torch.int32, dev)
    ckv = torch.empty(B, Sc, D, dtype=x.dtype, device=dev) if ckv is None else ckv
    _need(ckv, "ckv", (B, Sc, D), x.dtype, dev)
    with _on(dev):
        rc = lib.hca_compress_fwd(_ptr(x), _ptr(g), _ptr(bias), _ptr(seg), _ptr(ckv), B, S, D, m, _dtype_code(x),
                                  _stream(dev))
    _check(rc, "hca_compress_fwd")
    return ckv


def hca_compress_bwd(x, g, bias, seg, m: int, dckv, dx=None, dg=None, dbias=None, ws=None):
    """Backward of the compressor: (dx[B,S,D], dg[B,S] fp32, dbias[m] fp32)."""
    lib = load()
    B, S, D = x.shape
    Sc = -(-S // m)
    dev = x.device
    _need(dckv, "dckv", (B, Sc, D), x.dtype, dev)
    dx = torch.empty_like(x) if dx is None else dx
    dg = torch.empty(B, S, dtype=torch.float32, device=dev) if dg is None else dg
    dbias = torch.empty(m, dtype=torch.float32, device=dev) if dbias is None else dbias
    if ws is None:
        ws = torch.empty(lib.hca_compress_workspace_size(B, S, m), dtype=torch.uint8, device=dev)
    with _on(dev):
        rc = lib.hca_compress_bwd(_ptr(x), _ptr(g), _ptr(bias), _ptr(seg), _ptr(dckv), _ptr(dx), _ptr(dg),
                                  _ptr(dbias), B, S, D, m, _dtype_code(x), _ptr(ws), ws.numel(), _stream(dev))
    _check(rc, "hca_compress_bwd")
    return dx, dg, dbias


def hca_indexer_topk(qi: torch.Tensor, ki: torch.Tensor, w: torch.Tensor, seg: Optional[torch.Tensor], m: int,
                     k: int, with_scores: bool = False, ws: Optional[torch.Tensor] = None, check: bool = False):
    """Lightning Indexer top-k: (sel[B,S,k] int32, scores[B,S,Sc] fp32 or
    None) from qi[B,S,Hi,128], ki[B,ceil(S/m),128] (bf16), w[B,S,Hi] fp32."""
    lib = load()
    B, S, Hi, Di = qi.shape
    Sc = -(-S // m)
    dev = qi.device
    _need(qi, "qi", (B, S, Hi, Di), torch.bfloat16, dev)
    _need(ki, "ki", (B, Sc, Di), torch.bfloat16, dev)
    _need(w, "w", (B, S, Hi), torch.float32, dev)
    if seg is not None:
        _need(seg, "seg", (B, S), torch.int32, dev)
    sel = torch.empty(B, S, k, dtype=torch.int32, device=dev)
    scores = torch.empty(B, S, Sc, dtype=torch.float32, device=dev) if with_scores else None
    if ws is None:
        ws = torch.empty(lib.hca_indexer_workspace_size(B, S, m), dtype=torch.uint8, device=dev)
    with _on(dev):
        rc = lib.hca_indexer_topk(_ptr(qi), _ptr(ki), _ptr(w), _ptr(seg), _ptr(sel), _ptr(scores), B, S, Hi, Di, m, k,
                                  _ptr(ws), ws.numel(), _stream(dev))
    _check(rc, "hca_indexer_topk")
    if check:
        _check(hca_workspace_status(ws), "hca_indexer_topk (device)")
    return sel, scores


def csa_workspace(B, H, S, D, W, m, k, dtype, for_backward, device) -> torch.Tensor:
    n = load().hca_csa_workspace_size(B, H, S, D, W, m, k, _DTYPES[dtype], int(for_backward))
    if n == 0:
        raise HCAError(8, "hca_csa_workspace_size")
    return torch.empty(n, dtype=torch.uint8, device=device)


def hca_csa_attn_fwd(q, kv, ckv, seg, sel, W: int, m: int, scale: float, out=None, lse=None, ws=None,
                     check: bool = False):
    """CSA forward: (out, lse); sel[B,S,k] int32 selected compressed entries."""
    lib = load()
    B, H, S, D, Sc = _shapes(q, kv, ckv, seg, m)
    k = sel.shape[-1]
    _need(sel, "sel", (B, S, k), torch.int32, q.device)
    dt = _dtype_code(q)
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty(B, H, S, dtype=torch.float32, device=q.device) if lse is None else lse
    ws = csa_workspace(B, H, S, D, W, m, k, q.dtype, False, q.device) if ws is None else ws
    with _on(q.device):
        rc = lib.hca_csa_attn_fwd(_ptr(q), _ptr(kv), _ptr(ckv), _ptr(seg), _ptr(sel), _ptr(out), _ptr(lse), B, H, S,
                                  D, W, m, k, float(scale), dt, _ptr(ws), ws.numel(), _stream(q.device))
    _check(rc, "hca_csa_attn_fwd")
    if check:
        _check(hca_workspace_status(ws), "hca_csa_attn_fwd (device)")
    return out, lse


def hca_csa_attn_bwd(q, kv, ckv, seg, sel, out, lse, dout, W: int, m: int, scale: float, dq=None, dkv=None,
                     dckv=None, ws=None, check: bool = False):
    """CSA backward: (dq, dkv, dckv)."""
    lib = load()
    B, H, S, D, Sc = _shapes(q, kv, ckv, seg, m)
    k = sel.shape[-1]
    _need(sel, "sel", (B, S, k), torch.int32, q.device)
    dt = _dtype_code(q)
    dq = torch.empty_like(q) if dq is None else dq
    dkv = torch.empty_like(kv) if dkv is None else dkv
    dckv = torch.empty_like(ckv) if dckv is None else dckv
    ws = csa_workspace(B, H, S, D, W, m, k, q.dtype, True, q.device) if ws is None else ws
    with _on(q.device):
        rc = lib.hca_csa_attn_bwd(_ptr(q), _ptr(kv), _ptr(ckv), _ptr(seg), _ptr(sel), _ptr(out), _ptr(lse),
                                  _ptr(dout), _ptr(dq), _ptr(dkv), _ptr(dckv), B, H, S, D, W, m, k, float(scale), dt,
                                  _ptr(ws), ws.numel(), _stream(q.device))
    _check(rc, "hca_csa_attn_bwd")
    if check:
        _check(hca_workspace_status(ws), "hca_csa_attn_bwd (device)")
    return dq, dkv, dckv


# ---------------------------------------------------------------------------
# norms and positions
# ---------------------------------------------------------------------------
def _rows(t: torch.Tensor, name: str, shape, dtype, device):
    """Pointer and strides (elements; NULL where contiguous) of a tensor whose
    rows' columns are adjacent."""
    if t is None:
        raise ValueError(f"{name} is required")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} has shape {tuple(t.shape)}, expected {tuple(shape)}")
    if t.dtype != dtype:
        raise TypeError(f"{name} has dtype {t.dtype}, expected {dtype}")
    if t.device != device:
        raise ValueError(f"{name} is on {t.device}, expected {device}")
    if t.is_contiguous():
        return t.data_ptr(), None
    if t.stride(-1) != 1:
        raise ValueError(f"{name}'s last dimension must be contiguous")
    st = t.stride()[:-1]
    return t.data_ptr(), (ctypes.c_int64 * len(st))(*st)


def _angles(pos, freq, lead, dev):
    """(pos pointer, freq pointer, axes, rot) for tokens of shape `lead`: pos
    [*lead] or [axes, *lead] int32 or None, freq [rot/2] or [axes, rot/2] fp32."""
    if freq is None:
        raise ValueError("freq is required")
    if freq.dim() not in (1, 2):
        raise ValueError("freq must be [rot/2] or [axes,rot/2]")
    axes = freq.shape[0] if freq.dim() == 2 else 1
    _need(freq, "freq", freq.shape, torch.float32, dev)
    if pos is not None:
        _need(pos, "pos", lead if axes == 1 and pos.dim() == len(lead) else (axes, *lead), torch.int32, dev)
    elif axes > 1:
        raise ValueError("pos is required for more than one axis")
    return _pp(pos), freq.data_ptr(), axes, 2 * freq.shape[-1]


def _pp(t: Optional[torch.Tensor]):
    return None if t is None else t.data_ptr()


def _weight(w, name: str, D: int, dev):
    if w is not None:
        _need(w, name, (D,), torch.float32, dev)
    return _pp(w)


def _norm_rope_sizes(q, kv):
    """(B, H, S, D, dtype, device) of q[B,H,S,D] and kv[B,S,D], either of which may be None."""
    t = q if q is not None else kv
    if t is None:
        raise ValueError("q or kv is required")
    if (q is not None and q.dim() != 4) or (kv is not None and kv.dim() != 3):
        raise ValueError("q must be [B,H,S,D] and kv [B,S,D]")
    B, S, D = t.shape[0], t.shape[-2], t.shape[-1]
    if t.device.type != "cuda":
        raise ValueError(f"the calls work on CUDA tensors, not on {t.device}")
    return B, (q.shape[1] if q is not None else 0), S, D, t.dtype, t.device


def hca_norm_rope_fwd(q: Optional[torch.Tensor], kv: Optional[torch.Tensor], wq: Optional[torch.Tensor],
                      wkv: Optional[torch.Tensor], pos: Optional[torch.Tensor], freq: torch.Tensor, eps: float,
                      first: Optional[int] = None, halves: bool = False, qo: Optional[torch.Tensor] = None,
                      kvo: Optional[torch.Tensor] = None):
    """Norms of each head of q[B,H,S,D] and of kv[B,S,D] (bf16 or fp32; any
    strides with adjacent columns, such as a projection's [B,S,H,D] seen as
    [B,H,S,D]) and the rotation of columns [first, first + rot) (the last ones
    by default): (qo[B,H,S,D], kvo[B,S,D]), contiguous.  wq, wkv [D] fp32 or
    None; pos [B,S] or [axes,B,S] int32 (None: 0 .. S - 1); freq [rot/2] or
    [axes,rot/2] fp32 (include/hca.h, hca_norm_rope_fwd).  q or kv may be None."""
    lib = _lib or load()
    r = _py and _py.norm_rope_fwd(q, kv, None, None, wq, wkv, pos, freq, eps, first, halves, qo, kvo)
    if r is not None:
        return _made(r, "hca_norm_rope_fwd", False)
    B, H, S, D, dt, dev = _norm_rope_sizes(q, kv)
    pp, fp, axes, rot = _angles(pos, freq, (B, S), dev)
    args = []
    for x, w, y, name, shape in ((q, wq, qo, "q", (B, H, S, D)), (kv, wkv, kvo, "kv", (B, S, D))):
        if x is None:
            args += [None, None, None, None]
            continue
        y = torch.empty(shape, dtype=dt, device=dev) if y is None else y
        _need(y, name + "o", shape, dt, dev)
        args += [*_rows(x, name, shape, dt, dev), _weight(w, "w" + name, D, dev), y.data_ptr()]
        if name == "q":
            qo = y
        else:
            kvo = y
    with _on(dev):
        rc = lib.hca_norm_rope_fwd(*args, pp, fp, None, None, B, H, S, D, 0, axes, _int(D - rot if first is None else first), rot, int(halves),
                                   eps, _dtype_code(q if q is not None else kv), _stream(dev))
    _check(rc, "hca_norm_rope_fwd")
    return (qo if q is not None else None), (kvo if kv is not None else None)


def hca_norm_rope_bwd(q, kv, wq, wkv, pos, freq, eps: float, dqo, dkvo, first: Optional[int] = None, halves: bool = False, dq=None,
                      dkv=None, dwq=None, dwkv=None, ws: Optional[torch.Tensor] = None):
    """Backward of hca_norm_rope_fwd for the cotangents dqo[B,H,S,D] and
    dkvo[B,S,D] (contiguous): (dq, dkv, dwq, dwkv), dq and dkv laid out as q and
    kv are, None where there is no q, kv or weight."""
    lib = _lib or load()
    r = _py and _py.norm_rope_bwd(q, kv, wq, wkv, pos, freq, eps, dqo, dkvo, first, halves, dq, dkv, dwq, dwkv, ws)
    if r is not None:
        return _made(r, "hca_norm_rope_bwd", False)
    B, H, S, D, dt, dev = _norm_rope_sizes(q, kv)
    pp, fp, axes, rot = _angles(pos, freq, (B, S), dev)
    args, res = [], []
    for x, w, g, dx, dw, name, shape in ((q, wq, dqo, dq, dwq, "q", (B, H, S, D)), (kv, wkv, dkvo, dkv, dwkv, "kv", (B, S, D))):
        if x is None:
            args += [None] * 7
            res.append((None, None))
            continue
        _need(g, f"d{name}o", shape, dt, dev)
        px = _rows(x, name, shape, dt, dev)
        if dx is None:
            dx = torch.empty_like(x) if 0 not in x.stride() else torch.empty(shape, dtype=dt, device=dev)
        if w is None and dw is not None:
            raise ValueError(f"dw{name} is the gradient of w{name}, which is None")
        dw = torch.empty(D, dtype=torch.float32, device=dev) if dw is None and w is not None else dw
        args += [*px, _weight(w, "w" + name, D, dev), g.data_ptr(), *_rows(dx, "d" + name, shape, dt, dev),
                 _weight(dw, "dw" + name, D, dev)]
        res.append((dx, dw))
    if ws is None:
        ws = torch.empty(lib.hca_norm_rope_workspace_size(D), dtype=torch.uint8, device=dev)
    with _on(dev):
        rc = lib.hca_norm_rope_bwd(*args, pp, fp, B, H, S, D, axes, _int(D - rot if first is None else first), rot, int(halves), eps,
                                   _dtype_code(q if q is not None else kv), *_scratch(ws, dev), _stream(dev))
    _check(rc, "hca_norm_rope_bwd")
    return res[0][0], res[1][0], res[0][1], res[1][1]


def hca_rope(x: torch.Tensor, pos: Optional[torch.Tensor], freq: torch.Tensor, inverse: bool = False,
             first: Optional[int] = None, halves: bool = False, y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The rotation alone of x[B,H,S,D]: y[B,H,S,D] (any strides with adjacent
    columns for both; y may be x).  ``inverse`` turns back, as the attention's
    output has to be before the output projection; it is also the gradient of
    the call without it, and the other way round."""
    lib = _lib or load()
    r = _py and _py.rope(x, None, None, pos, freq, inverse, first, halves, y)
    if r is not None:
        return _made(r, "hca_rope", False)[0]
    if x.dim() != 4:
        raise ValueError("x must be [B,H,S,D]")
    B, H, S, D = x.shape
    dev = x.device
    if dev.type != "cuda":
        raise ValueError(f"the calls work on CUDA tensors, not on {dev}")
    pp, fp, axes, rot = _angles(pos, freq, (B, S), dev)
    y = torch.empty(x.shape, dtype=x.dtype, device=dev) if y is None else y
    with _on(dev):
        rc = lib.hca_rope(*_rows(x, "x", x.shape, x.dtype, dev), *_rows(y, "y", x.shape, x.dtype, dev), pp, fp, None, None, B, H, S, D,
                          0, axes, _int(D - rot if first is None else first), rot, int(halves), int(inverse), _dtype_code(x), _stream(dev))
    _check(rc, "hca_rope")
    return y


# ---------------------------------------------------------------------------
# serving: plan, append and attend over a paged 8-bit cache
#
# A decode step's kernels take a few microseconds each, so what these calls do
# in Python counts.  An ordinary one goes through _hca_py (its tensors fit and
# are on the current device); what that declines is checked, refused or done
# here.
# ---------------------------------------------------------------------------
_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None)


def _enqueue(dev: torch.device, f, *args) -> int:
    """f(*args, stream) on the device's current stream."""
    if dev.type != "cuda":
        raise ValueError(f"the cache calls work on CUDA tensors, not on {dev}")
    if _raw_stream is not None and dev.index == torch.cuda.current_device():
        return f(*args, _raw_stream(dev.index))
    with _on(dev):
        return f(*args, _stream(dev))


def _made(r, name: str, check: bool):
    """The answer of a call that _hca_py has made: its results and workspace, or the status."""
    if type(r) is int:
        _check(r, name)
    elif check:
        _check(hca_workspace_status(r[-1]), name + " (device)")
    return r


def _fits(t: torch.Tensor, name: str, shape, dtype, device) -> int:
    """The pointer of a tensor that is as it has to be (as _need)."""
    if t.shape != shape or t.dtype is not dtype or t.device != device or not t.is_contiguous():
        _need(t, name, shape, dtype, device)
    return t.data_ptr()


def _scratch(ws: torch.Tensor, dev: torch.device) -> Tuple[int, int]:
    """Pointer and bytes of a caller's workspace (what it holds is for the C function to check)."""
    if ws.dtype is not torch.uint8:
        raise TypeError(f"ws has dtype {ws.dtype}, expected {torch.uint8}")
    if ws.device != dev:
        raise ValueError(f"ws is on {ws.device}, expected {dev}")
    if not ws.is_contiguous():
        raise ValueError("ws must be contiguous")
    return ws.data_ptr(), ws.numel()


_I32, _F32, _E4M3 = torch.int32, torch.float32, torch.float8_e4m3fn


def _int(v: int) -> int:
    """v as an int32 (ctypes would drop its upper bits).  No window and no ratio
    reaches beyond the largest; every other number out of range stays one that
    the C function refuses."""
    return max(min(v, (1 << 31) - 1), -(1 << 31))


@functools.lru_cache(maxsize=4096)
def _plan_ws_bytes(R: int) -> int:
    return load().hca_cache_plan_workspace_size(R)


@functools.lru_cache(maxsize=4096)
def _append_ws_bytes(nblocks: int) -> int:
    return load().hca_cache_append_workspace_size(nblocks)


@functools.lru_cache(maxsize=4096)
def _attn_ws_bytes(N: int, R: int, H: int, D: int, dt: int) -> int:
    n = load().hca_cache_attn_workspace_size(N, R, H, D, dt)
    if n == 0:
        raise HCAError(8, "hca_cache_attn_workspace_size")
    return n


def hca_cache_plan(held: torch.Tensor, added: torch.Tensor, table: torch.Tensor, free_blocks: torch.Tensor,
                   free_count: torch.Tensor, nblocks: int, bs: int, nslots: int, m: int = 1,
                   start: Optional[torch.Tensor] = None, slots: Optional[torch.Tensor] = None,
                   free_left: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None, check: bool = False):
    """Block tables and slot maps of a serving step (include/hca.h,
    hca_cache_plan): held[R], added[R], table[R,cols] (updated in place),
    free_blocks[nfree], free_count[1], all int32.  Returns (start[R+1],
    slots[nslots], free_left[1]); free_left may be free_count itself."""
    lib = _lib or load()
    r = _py and _py.cache_plan(held, added, table, free_blocks, free_count, nblocks, bs, nslots, m, start, slots,
                               free_left, ws, check)
    if r is not None:
        return _made(r, "hca_cache_plan", check)[:3]
    dev = held.device
    if held.dim() != 1 or table.dim() != 2 or free_blocks.dim() != 1:
        raise ValueError("held must be [R], table [R,cols] and free_blocks [nfree]")
    R, cols = table.shape
    nfree = free_blocks.shape[0]
    start = torch.empty(R + 1, dtype=_I32, device=dev) if start is None else start
    slots = torch.empty(nslots, dtype=_I32, device=dev) if slots is None else slots
    free_left = torch.empty(1, dtype=_I32, device=dev) if free_left is None else free_left
    ws = torch.empty(_plan_ws_bytes(R), dtype=torch.uint8, device=dev) if ws is None else ws
    rc = _enqueue(dev, lib.hca_cache_plan, _fits(held, "held", (R,), _I32, dev), _fits(added, "added", (R,), _I32, dev),
                  _fits(table, "table", (R, cols), _I32, dev), _fits(free_blocks, "free_blocks", (nfree,), _I32, dev),
                  _fits(free_count, "free_count", (1,), _I32, dev), _fits(free_left, "free_left", (1,), _I32, dev),
                  _fits(start, "start", (R + 1,), _I32, dev), _fits(slots, "slots", (nslots,), _I32, dev), R, cols, _int(bs),
                  _int(m), _int(nblocks), nfree, _int(nslots), *_scratch(ws, dev))
    if rc != 0:
        _check(rc, "hca_cache_plan")
    if check:
        _check(hca_workspace_status(ws), "hca_cache_plan (device)")
    return start, slots, free_left


def hca_cache_append(x: torch.Tensor, slots: torch.Tensor, pool: torch.Tensor, scale: torch.Tensor,
                     ws: Optional[torch.Tensor] = None, check: bool = False) -> None:
    """Rows x[N,D] (bf16 or fp32) into slots[N] (int32, -1: nowhere) of the
    cache pool[nblocks,bs,D] (float8_e4m3fn) with scale[nblocks] (fp32), both
    updated in place (include/hca.h, hca_cache_append)."""
    lib = _lib or load()
    r = _py and _py.cache_append(x, slots, pool, scale, ws, check)
    if r is not None:
        _made(r, "hca_cache_append", check)
        return
    dev = x.device
    if x.dim() != 2 or pool.dim() != 3:
        raise ValueError("x must be [N,D] and pool [nblocks,bs,D]")
    dt = _dtype_code(x)
    nblocks, bs, D = pool.shape
    N = x.shape[0]
    ws = torch.empty(_append_ws_bytes(nblocks), dtype=torch.uint8, device=dev) if ws is None else ws
    rc = _enqueue(dev, lib.hca_cache_append, _fits(x, "x", (N, D), x.dtype, dev), _fits(slots, "slots", (N,), _I32, dev),
                  _fits(pool, "pool", (nblocks, bs, D), _E4M3, dev), _fits(scale, "scale", (nblocks,), _F32, dev), N, D,
                  bs, nblocks, dt, *_scratch(ws, dev))
    if rc != 0:
        _check(rc, "hca_cache_append")
    if check:
        _check(hca_workspace_status(ws), "hca_cache_append (device)")


def _cache_args(name: str, cache, R: int, bs: int, D: int, dev):
    if cache is None:
        return None, None, None, 0, 0
    pool, scale, table = cache
    if pool.dim() != 3 or table.dim() != 2:
        raise ValueError(f"{name} must be (pool[nblocks,bs,D], scale[nblocks], table[R,cols])")
    nblocks, cols = pool.shape[0], table.shape[1]
    return (_fits(pool, f"{name} pool", (nblocks, bs, D), _E4M3, dev), _fits(scale, f"{name} scale", (nblocks,), _F32, dev),
            _fits(table, f"{name} table", (R, cols), _I32, dev), nblocks, cols)


def hca_cache_attn(q: torch.Tensor, start: torch.Tensor, held: torch.Tensor, raw, comp, W: int, m: int, scale: float,
                   out: Optional[torch.Tensor] = None, lse: Optional[torch.Tensor] = None,
                   ws: Optional[torch.Tensor] = None, check: bool = False) -> Tuple[torch.Tensor, torch.Tensor]:
    """HCA attention of packed query tokens q[N,H,D] over the cache
    (include/hca.h, hca_cache_attn): request r's tokens are rows
    start[r]..start[r+1]-1 at positions held[r]...  raw and comp are
    (pool, scale, table[R,cols]); comp may be None.  Returns (out[N,H,D],
    lse[N,H] fp32)."""
    lib = _lib or load()
    r = _py and _py.cache_attn(q, start, held, raw, comp, W, m, scale, out, lse, ws, check)
    if r is not None:
        return _made(r, "hca_cache_attn", check)[:2]
    dev = q.device
    if q.dim() != 3 or held.dim() != 1 or raw[0].dim() != 3:
        raise ValueError("q must be [N,H,D], held [R] and the raw pool [nblocks,bs,D]")
    N, H, D = q.shape
    R, bs = held.shape[0], raw[0].shape[1]
    dt = _dtype_code(q)
    args = (*_cache_args("raw", raw, R, bs, D, dev), *_cache_args("comp", comp, R, bs, D, dev))
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty((N, H), dtype=_F32, device=dev) if lse is None else lse
    ws = torch.empty(_attn_ws_bytes(N, R, H, D, dt), dtype=torch.uint8, device=dev) if ws is None else ws
    rc = _enqueue(dev, lib.hca_cache_attn, _fits(q, "q", (N, H, D), q.dtype, dev), _fits(start, "start", (R + 1,), _I32, dev),
                  _fits(held, "held", (R,), _I32, dev), *args, _fits(out, "out", (N, H, D), q.dtype, dev),
                  _fits(lse, "lse", (N, H), _F32, dev), N, R, H, D, _int(W), _int(m), bs, scale, dt,
                  *_scratch(ws, dev))
    if rc != 0:
        _check(rc, "hca_cache_attn")
    if check:
        _check(hca_workspace_status(ws), "hca_cache_attn (device)")
    return out, lse


@functools.lru_cache(maxsize=4096)
def _attn_shared_ws_bytes(N: int, R: int, H: int, D: int, G: int, dt: int) -> int:
    n = load().hca_cache_attn_shared_workspace_size(N, R, H, D, G, dt)
    if n == 0:
        raise HCAError(8, "hca_cache_attn_shared_workspace_size")
    return n


def hca_cache_attn_shared(q: torch.Tensor, start: torch.Tensor, held: torch.Tensor, raw, comp, first: torch.Tensor,
                          shared_cols: torch.Tensor, W: int, m: int, scale: float, out: Optional[torch.Tensor] = None,
                          lse: Optional[torch.Tensor] = None, ws: Optional[torch.Tensor] = None,
                          check: bool = False) -> Tuple[torch.Tensor, torch.Tensor]:
    """hca_cache_attn for requests that begin with the same blocks of compressed
    entries, which are attended once for all of them (include/hca.h,
    hca_cache_attn_shared): requests first[g] .. first[g+1] - 1 have the first
    shared_cols[g] columns of their compressed tables in common; first[G+1] and
    shared_cols[G] are int32 tensors.  Results as hca_cache_attn's."""
    lib = _lib or load()
    r = _py and _py.cache_attn_shared(q, start, held, raw, comp, first, shared_cols, W, m, scale, out, lse, ws, check)
    if r is not None:
        return _made(r, "hca_cache_attn_shared", check)[:2]
    dev = q.device
    if q.dim() != 3 or held.dim() != 1 or raw[0].dim() != 3:
        raise ValueError("q must be [N,H,D], held [R] and the raw pool [nblocks,bs,D]")
    if comp is None or shared_cols.dim() != 1:
        raise ValueError("comp is required, and shared_cols must be [G]")
    N, H, D = q.shape
    R, bs, G = held.shape[0], raw[0].shape[1], shared_cols.shape[0]
    dt = _dtype_code(q)
    args = (*_cache_args("raw", raw, R, bs, D, dev), *_cache_args("comp", comp, R, bs, D, dev),
            _fits(first, "first", (G + 1,), _I32, dev), _fits(shared_cols, "shared_cols", (G,), _I32, dev))
    out = torch.empty_like(q) if out is None else out
    lse = torch.empty((N, H), dtype=_F32, device=dev) if lse is None else lse
    ws = torch.empty(_attn_shared_ws_bytes(N, R, H, D, G, dt), dtype=torch.uint8, device=dev) if ws is None else ws
    rc = _enqueue(dev, lib.hca_cache_attn_shared, _fits(q, "q", (N, H, D), q.dtype, dev), _fits(start, "start", (R + 1,), _I32, dev),
                  _fits(held, "held", (R,), _I32, dev), *args, _fits(out, "out", (N, H, D), q.dtype, dev),
                  _fits(lse, "lse", (N, H), _F32, dev), N, R, H, D, G, _int(W), _int(m), bs, scale, dt, *_scratch(ws, dev))
    if rc != 0:
        _check(rc, "hca_cache_attn_shared")
    if check:
        _check(hca_workspace_status(ws), "hca_cache_attn_shared (device)")
    return out, lse


def _packed(t: torch.Tensor, name: str, shape, dtype, dev):
    """Pointer and strides of packed rows [N,H,D] or [N,D] as the C functions take them."""
    p, st = _rows(t, name, shape, dtype, dev)
    if st is None:
        return p, None
    return p, (ctypes.c_int64 * 3)(0, st[1], st[0]) if len(shape) == 3 else (ctypes.c_int64 * 2)(0, st[0])


def _packed_requests(start, held, pos, dev):
    if start is None or start.dim() != 1 or start.shape[0] < 1:
        raise ValueError("start must be [R+1]")
    R = start.shape[0] - 1
    if held is None and pos is None:
        raise ValueError("held or pos is required")
    return _fits(start, "start", (R + 1,), _I32, dev), None if held is None else _fits(held, "held", (R,), _I32, dev), R


def hca_cache_norm_rope(q: Optional[torch.Tensor], kv: Optional[torch.Tensor], start: torch.Tensor, held: Optional[torch.Tensor],
                        wq: Optional[torch.Tensor], wkv: Optional[torch.Tensor], freq: torch.Tensor, eps: float,
                        first: Optional[int] = None, halves: bool = False, pos: Optional[torch.Tensor] = None,
                        qo: Optional[torch.Tensor] = None, kvo: Optional[torch.Tensor] = None):
    """hca_norm_rope_fwd for a serving step's packed tokens: q[N,H,D] and kv[N,D]
    of the requests that hca_cache_attn takes by start[R+1] and held[R]; pos
    [N] or [axes,N] int32 replaces the positions held[r], held[r] + 1, ...  Rows
    of the results from start[R] on are left as they are.  Returns (qo, kvo)."""
    lib = _lib or load()
    r = _py and start is not None and _py.norm_rope_fwd(q, kv, start, held, wq, wkv, pos, freq, eps, first, halves, qo, kvo)
    if r:
        return _made(r, "hca_cache_norm_rope", False)
    t = q if q is not None else kv
    if t is None:
        raise ValueError("q or kv is required")
    if (q is not None and q.dim() != 3) or (kv is not None and kv.dim() != 2):
        raise ValueError("q must be [N,H,D] and kv [N,D]")
    N, D, dev, dt = t.shape[0], t.shape[-1], t.device, t.dtype
    H = q.shape[1] if q is not None else 0
    ps, ph, R = _packed_requests(start, held, pos, dev)
    pp, fp, axes, rot = _angles(pos, freq, (N,), dev)
    args = []
    for x, w, y, name, shape in ((q, wq, qo, "q", (N, H, D)), (kv, wkv, kvo, "kv", (N, D))):
        if x is None:
            args += [None, None, None, None]
            continue
        y = torch.empty(shape, dtype=dt, device=dev) if y is None else y
        args += [*_packed(x, name, shape, dt, dev), _weight(w, "w" + name, D, dev), _fits(y, name + "o", shape, dt, dev)]
        if name == "q":
            qo = y
        else:
            kvo = y
    rc = _enqueue(dev, lib.hca_norm_rope_fwd, *args, pp, fp, ps, ph, 1, H, N, D, R, axes, _int(D - rot if first is None else first), rot,
                  int(halves), eps, _dtype_code(t))
    if rc != 0:
        _check(rc, "hca_cache_norm_rope")
    return (qo if q is not None else None), (kvo if kv is not None else None)


def hca_cache_rope(x: torch.Tensor, start: torch.Tensor, held: Optional[torch.Tensor], freq: torch.Tensor, inverse: bool = False,
                   first: Optional[int] = None, halves: bool = False, pos: Optional[torch.Tensor] = None,
                   y: Optional[torch.Tensor] = None) -> torch.Tensor:
    """hca_rope for a serving step's packed tokens x[N,H,D] (arguments as
    hca_cache_norm_rope); y may be x."""
    lib = _lib or load()
    r = _py and start is not None and _py.rope(x, start, held, pos, freq, inverse, first, halves, y)
    if r:
        return _made(r, "hca_cache_rope", False)[0]
    if x.dim() != 3:
        raise ValueError("x must be [N,H,D]")
    N, H, D = x.shape
    dev = x.device
    ps, ph, R = _packed_requests(start, held, pos, dev)
    pp, fp, axes, rot = _angles(pos, freq, (N,), dev)
    y = torch.empty(x.shape, dtype=x.dtype, device=dev) if y is None else y
    rc = _enqueue(dev, lib.hca_rope, *_packed(x, "x", x.shape, x.dtype, dev), *_packed(y, "y", x.shape, x.dtype, dev), pp, fp, ps, ph, 1, H,
                  N, D, R, axes, _int(D - rot if first is None else first), rot, int(halves), int(inverse), _dtype_code(x))
    if rc != 0:
        _check(rc, "hca_cache_rope")
    return y
