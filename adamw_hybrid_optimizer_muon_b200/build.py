"""Build the MuonAdamW CUDA library in-tree for sm_100a.

    python -m adamw_hybrid_optimizer_muon_b200.build [--verbose] [--force]

Compiles every ``csrc/*.cu`` with nvcc (``-gencode arch=compute_100a,code=sm_100a``)
into ``lib/libmuonadamw.so``, and once more with ``-DMA_DEBUG`` into
``lib/libmuonadamw_debug.so``: the debug build checks every hand-computed device
index against the extent of its buffer (a failed check records MA_ERR_BOUNDS
and skips the access) and otherwise computes the same bits. Each object is
rebuilt only when a source or header is newer than it; the objects compile in
parallel. nvcc cross-compiles, so no GPU is needed. ``csrc/marshal.cpp`` becomes
a Python extension module built against the installed torch (its name in ``lib/``
has the versions of Python and torch); the libraries do not need it, and where it cannot be built there is a warning.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
if not __package__:  # run as a script
    sys.path.insert(0, ROOT)

from adamw_hybrid_optimizer_muon_b200 import _marshal_path  # noqa: E402

CSRC = os.path.join(HERE, "csrc")
OBJ = os.path.join(HERE, "_build")
LIB_DIR = os.path.join(HERE, "lib")
LIB = os.path.join(LIB_DIR, "libmuonadamw.so")
LIB_DEBUG = os.path.join(LIB_DIR, "libmuonadamw_debug.so")
VARIANTS = (("release", LIB, []), ("debug", LIB_DEBUG, ["-DMA_DEBUG"]))

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O3",
         "--expt-relaxed-constexpr", "-I" + os.path.join(ROOT, "include")]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _headers():
    return glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h"))


def _build_marshal(verbose: bool, force: bool) -> None:
    """The extension module that reads lists of tensors. The binding does without it, more slowly: what goes wrong
    here is reported and not raised."""
    src = os.path.join(CSRC, "marshal.cpp")
    try:
        import torch
    except ImportError:
        sys.stderr.write("marshal.cpp not built: torch cannot be imported\n")
        return
    out = _marshal_path(torch)
    if not force and os.path.exists(out) and os.path.getmtime(out) >= os.path.getmtime(src):
        return
    base = os.path.dirname(torch.__file__)
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-w",
           "-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(base, "include"),
           "-I" + os.path.join(base, "include", "torch", "csrc", "api", "include"), src, "-o", out,
           "-L" + os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10"]
    try:
        res = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        sys.stderr.write(f"marshal.cpp not built: {e}\n")
        return
    if verbose or res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
    if res.returncode != 0:
        sys.stderr.write(f"marshal.cpp not built: {cmd[0]} failed\n")


def build(verbose: bool = False, force: bool = False) -> str:
    """Build both libraries, and the extension module where that works; returns the release library's path."""
    os.makedirs(LIB_DIR, exist_ok=True)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    hdr_mtime = max([os.path.getmtime(h) for h in _headers()] + [0.0])
    jobs = []  # (source, object, extra flags)
    objs = {}
    for name, _, extra in VARIANTS:
        odir = os.path.join(OBJ, name)
        os.makedirs(odir, exist_ok=True)
        objs[name] = []
        for src in srcs:
            obj = os.path.join(odir, os.path.basename(src)[:-3] + ".o")
            objs[name].append(obj)
            if force or not os.path.exists(obj) or os.path.getmtime(obj) < max(os.path.getmtime(src), hdr_mtime):
                jobs.append((src, obj, extra))

    def compile_one(job):
        src, obj, extra = job
        cmd = [nvcc()] + ARCH + FLAGS + extra + (["-Xptxas", "-v"] if verbose else []) + ["-c", src, "-o", obj]
        return job, subprocess.run(cmd, capture_output=True, text=True)

    workers = max(1, min(len(jobs), os.cpu_count() or 1))
    failed = []
    with concurrent.futures.ThreadPoolExecutor(max_workers=workers) as pool:
        for (src, obj, extra), res in pool.map(compile_one, jobs):
            if verbose or res.returncode != 0:
                sys.stderr.write(res.stdout + res.stderr)
            if res.returncode != 0:
                failed.append(os.path.basename(src) + (" (debug)" if extra else ""))
    if failed:
        raise RuntimeError("nvcc failed on " + ", ".join(failed))
    for name, lib_path, _ in VARIANTS:
        o = objs[name]
        if force or not os.path.exists(lib_path) or os.path.getmtime(lib_path) < max(os.path.getmtime(x) for x in o):
            cmd = [nvcc()] + ARCH + ["-shared", "-Xcompiler", "-fPIC", "-o", lib_path] + o
            res = subprocess.run(cmd, capture_output=True, text=True)
            if res.returncode != 0:
                sys.stderr.write(res.stdout + res.stderr)
                raise RuntimeError(f"link failed ({name})")
    _build_marshal(verbose, force)
    return LIB


if __name__ == "__main__":
    print(build(verbose="--verbose" in sys.argv, force="--force" in sys.argv))
