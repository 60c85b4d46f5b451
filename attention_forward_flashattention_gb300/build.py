"""Builds the CUDA libraries in-tree with nvcc for sm_103a.

  _build/libfa_sm103.so    the product: C ABI of include/fa.h and fa_cache.h
  _build/libfa_selftest.so GPU unit tests of the PTX building blocks
  _build/_fa_cache_torch.so  the block cache's calls on torch tensors (host
                           code, g++, linked against libfa_sm103.so); left out
                           where there is no PyTorch, which the libraries do
                           not need

Translation units are compiled in parallel (one nvcc process each), then
linked. ptxas resource usage (registers, spills, shared memory) of every
kernel is kept in _build/ptxas_<unit>.log.
"""
from __future__ import annotations

import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT = os.path.join(PKG, "_build")
INCLUDE = os.path.join(ROOT, "include")

LIB_NAME = "libfa_sm103.so"
SELFTEST_NAME = "libfa_selftest.so"
LIB_UNITS = ["fa_host.cu", "fa_fwd_d64.cu", "fa_fwd_d128.cu", "fa_fwd_fp8.cu", "fa_fwd_pair.cu",
             "fa_bwd_d64.cu", "fa_bwd_d128.cu", "fa_noalloc.cu", "fa_pipeline.cu",
             "fa_cache_host.cu", "fa_cache_plan.cu", "fa_cache_append.cu", "fa_cache_attn.cu"]
SELFTEST_UNITS = ["selftest.cu"]
TORCH_NAME = "_fa_cache_torch.so"
TORCH_UNIT = "fa_cache_torch.cpp"
HEADERS = ["ptx.cuh", "fa_common.cuh", "fa_kernel.cuh", "fa_launch.cuh", "fa_pair.cuh", "fa_bwd.cuh",
           "fa_bwd_launch.cuh", "fa_dispatch.h", "fa_cache.cuh", "fa_cache_step.cuh", "fa_cache_chunk.cuh"]
PUBLIC_HEADERS = ["fa.h", "fa_cache.h"]

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found (set NVCC or put the CUDA toolkit on PATH)")


def _cuda_home(nvcc: str) -> str:
    return os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))


def _flags() -> list[str]:
    return ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                   "-Xptxas", "-v", "-I", INCLUDE, "-I", CSRC]


def lib_path() -> str:
    return os.path.join(OUT, LIB_NAME)


def selftest_path() -> str:
    return os.path.join(OUT, SELFTEST_NAME)


def torch_path() -> str:
    return os.path.join(OUT, TORCH_NAME)


def _torch_dir() -> str | None:
    """PyTorch's folder, None where it is not installed."""
    spec = importlib.util.find_spec("torch")
    if spec is None or not spec.submodule_search_locations:
        return None
    return list(spec.submodule_search_locations)[0]


def _torch_stamp() -> str:
    """What the torch module is built against: it is bound to that PyTorch and
    this interpreter."""
    with open(os.path.join(_torch_dir(), "version.py")) as f:
        return f"{sys.version}\n{_torch_dir()}\n{f.read()}"


def _torch_stale() -> bool:
    if _stale(torch_path(), [TORCH_UNIT]):
        return True
    try:
        with open(torch_path() + ".stamp") as f:
            return f.read() != _torch_stamp()
    except OSError:
        return True


def _torch_compile(nvcc: str, obj: str) -> list[str]:
    inc = [os.path.join(_torch_dir(), "include"), os.path.join(_cuda_home(nvcc), "include"),
           sysconfig.get_paths()["include"], INCLUDE]
    # (system headers: their warnings are not ours)
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall"] + [x for i in inc for x in ("-isystem", i)] + [
        "-c", os.path.join(CSRC, TORCH_UNIT), "-o", obj]


def _torch_link(obj: str, out: str) -> list[str]:
    lib = os.path.join(_torch_dir(), "lib")
    return ["g++", "-shared", "-o", out, obj, "-L" + OUT, "-l:" + LIB_NAME, "-L" + lib,
            "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-ltorch", "-lc10_cuda", "-lc10",
            "-Wl,-rpath,$ORIGIN", "-Wl,-rpath," + lib]


def _stale(target: str, sources: list[str]) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    deps = [os.path.join(CSRC, s) for s in sources + HEADERS] + [os.path.join(INCLUDE, h) for h in PUBLIC_HEADERS]
    return any(os.path.getmtime(d) > t for d in deps)


def _start(cmd: list[str], unit: str):
    """Starts a compiler; what it prints goes to the unit's log."""
    with open(_log_path(unit), "w") as log:
        return subprocess.Popen(cmd, stdout=log, stderr=subprocess.STDOUT)


def _log_path(unit: str) -> str:
    return os.path.join(OUT, f"ptxas_{os.path.splitext(unit)[0]}.log")


def _raise_failed(units: list[str]) -> None:
    msgs = []
    for u in units:
        with open(_log_path(u)) as f:
            msgs.append(f"--- {u}\n" + f.read()[-6000:])
    raise RuntimeError("compilation failed:\n" + "\n".join(msgs))


def build(force: bool = False, verbose: bool = False) -> tuple[str, str]:
    """Compiles the libraries and the torch module if any source is newer (the
    module also if PyTorch is another one); returns the libraries' paths. The
    libraries are complete before anything about the module can fail."""
    nvcc = nvcc_path()
    os.makedirs(OUT, exist_ok=True)
    jobs = []
    for units, name in ((LIB_UNITS, LIB_NAME), (SELFTEST_UNITS, SELFTEST_NAME)):
        if force or _stale(os.path.join(OUT, name), units):
            jobs.append((units, name))
    torch_job = _torch_dir() is not None and (force or bool(jobs) or _torch_stale())
    if not jobs and not torch_job:
        return lib_path(), selftest_path()
    procs, torch_proc, torch_error = [], None, None
    torch_obj = os.path.join(OUT, "fa_cache_torch.o")
    if torch_job:
        try:
            torch_proc = _start(_torch_compile(nvcc, torch_obj), TORCH_UNIT)
        except OSError as e:
            torch_error = e
    for units, _ in jobs:
        for u in units:
            obj = os.path.join(OUT, u.replace(".cu", ".o"))
            cmd = [nvcc] + _flags() + ["-c", os.path.join(CSRC, u), "-o", obj]
            if verbose:
                print(" ".join(cmd), file=sys.stderr)
            procs.append((u, _start(cmd, u)))
    failed = [u for u, p in procs if p.wait() != 0]
    torch_failed = torch_proc is not None and torch_proc.wait() != 0
    if failed:
        _raise_failed(failed)
    libdir = os.path.join(_cuda_home(nvcc), "lib64")
    for units, name in jobs:
        objs = [os.path.join(OUT, u.replace(".cu", ".o")) for u in units]
        tmp = os.path.join(OUT, name + f".tmp{os.getpid()}")
        cmd = [nvcc] + ARCH + ["-shared", "-cudart", "shared", "-o", tmp] + objs + [
            "-Xlinker", "-rpath", "-Xlinker", libdir]
        subprocess.run(cmd, check=True)
        os.replace(tmp, os.path.join(OUT, name))
    if torch_error is not None:
        raise RuntimeError(f"{TORCH_UNIT} not compiled: {torch_error}")
    if torch_failed:
        _raise_failed([TORCH_UNIT])
    if torch_job:
        tmp = torch_path() + f".tmp{os.getpid()}"
        subprocess.run(_torch_link(torch_obj, tmp), check=True)
        os.replace(tmp, torch_path())
        with open(tmp, "w") as f:
            f.write(_torch_stamp())
        os.replace(tmp, torch_path() + ".stamp")
    return lib_path(), selftest_path()


if __name__ == "__main__":
    paths = build(force="--force" in sys.argv, verbose=True)
    print("\n".join(paths))
