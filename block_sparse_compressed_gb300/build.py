"""Build libhca.so (the C-ABI CUDA library) in-tree with nvcc for sm_103a.

Each ``csrc/*.cu`` translation unit is compiled to an object in parallel,
then linked into ``block_sparse_compressed_gb300/libhca.so`` with the CUDA
runtime linked statically (the driver API is reached at run time through
``cudaGetDriverEntryPoint``, so the library loads on a machine without a
GPU).  ``csrc/hca_py.cpp``, the serving calls without their Python, becomes an
extension module with the host compiler and torch's headers; its file name says
which Python it is for and the module itself which torch.  Usage: ``python -m
block_sparse_compressed_gb300.build [--force]`` (without torch: ``python
block_sparse_compressed_gb300/build.py``).
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libhca.so")
PY_LIB = os.path.join(HERE, "_hca_py" + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-Xcompiler", "-fvisibility=hidden"]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libhca")


def _sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _deps():
    hdrs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))]
    hdrs.append(os.path.join(os.path.dirname(HERE), "include", "hca.h"))
    return hdrs


def _stale(target, inputs) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(p) > t for p in inputs)


def _torch():
    """torch, or None: libhca.so needs nothing of it."""
    try:
        import torch
        return torch
    except ImportError:
        return None


def _py_command(torch, target: str):
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    inc = [os.path.join(root, "include"), os.path.join(root, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    return [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
            f'-DHCA_TORCH="{torch.__version__}"', f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(a for i in inc for a in ("-isystem", i)),
            os.path.join(CSRC, "hca_py.cpp"), "-o", target, "-L" + os.path.join(root, "lib"), "-ltorch_python",
            "-ltorch_cpu", "-lc10_cuda", "-lc10"]


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    srcs = _sources()
    deps = _deps()
    objs = []
    jobs = []
    for s in srcs:
        o = os.path.join(BUILD, os.path.basename(s)[:-3] + ".o")
        objs.append(o)
        if force or _stale(o, [s] + deps):
            cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra_flags, "-c", s, "-o", o]
            jobs.append(cmd)

    # the module belongs to the Python, the torch and the command that it was compiled with
    torch = _torch()
    stamp = os.path.join(BUILD, "hca_py.command")
    known = open(stamp).read() if os.path.exists(stamp) else ""
    made_with = "\n".join([sys.version, *_py_command(torch, PY_LIB)]) if torch is not None else ""
    py_src = [os.path.join(CSRC, "hca_py.cpp"), os.path.join(os.path.dirname(HERE), "include", "hca.h")]
    py_tmp = PY_LIB + f".tmp{os.getpid()}"
    py_stale = force or torch is None or known != made_with or _stale(PY_LIB, py_src)
    kernels = len(jobs)
    py_cmd = _py_command(torch, py_tmp) if torch is not None and py_stale else None
    if py_cmd:
        jobs.insert(0, py_cmd)

    def run(cmd):
        try:
            r = subprocess.run(cmd, capture_output=True, text=True)
        except OSError as e:  # no such compiler
            r = subprocess.CompletedProcess(cmd, 127, "", str(e))
        return cmd, r

    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs), os.cpu_count() or 4))) as ex:
        for cmd, r in ex.map(run, jobs):
            if verbose or r.returncode != 0:
                sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
            if r.returncode != 0 and cmd is not py_cmd:
                raise RuntimeError(f"nvcc failed on {cmd[-3]}")
    if py_stale and not os.path.exists(py_tmp):
        # no torch, no headers of it or of Python, no host compiler: the calls work
        # without the module, through ctypes
        sys.stderr.write(f"{os.path.basename(PY_LIB)} was not built: the serving calls cost 10 to 20 us more each\n")
    if py_stale and os.path.exists(py_tmp):
        os.replace(py_tmp, PY_LIB)
        with open(stamp, "w") as f:
            f.write(made_with)
    elif py_stale and os.path.exists(PY_LIB):
        os.remove(PY_LIB)  # of another Python, torch or source
    plain = os.path.join(HERE, "_hca_py.so")  # any Python would take that one
    if plain != PY_LIB and os.path.exists(plain):
        os.remove(plain)
    if force or kernels or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-Xcompiler", "-fPIC"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
            raise RuntimeError("linking libhca.so failed")
        os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose="-v" in sys.argv)
    print(LIB)
