"""Build libmoe.so in-tree with nvcc for sm_103a.

Each .cu translation unit under csrc/ is compiled in parallel, then linked
into moe_expert_mlp_gb300/libmoe.so.  No cmake, no torch extension machinery:
the library is a plain C-ABI shared object.  csrc/moe_binding.c, the Python
binding of the smallest calls, is compiled beside it for the Python that runs
(its headers and a C compiler are needed for this part alone).
"""
from __future__ import annotations

import concurrent.futures as cf
import contextlib
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmoe.so")
BINDING = os.path.join(PKG, "_binding" + sysconfig.get_config_var("EXT_SUFFIX"))

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + [
    "-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
    "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include"),
]


def _nvcc():
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def _stale(out, deps):
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def _binding_job(nvcc, header, force):
    """Command that compiles the Python binding, up to its output; None where
    the one that is there is fresh."""
    src = os.path.join(CSRC, "moe_binding.c")
    if not force and not _stale(BINDING, [src, header]):
        return None
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "include")
    return [os.environ.get("CC", "gcc"), "-O2", "-std=gnu11", "-shared", "-fPIC", "-Wall", "-Wextra",
            "-I", sysconfig.get_paths()["include"], "-I", cuda, "-I", os.path.join(ROOT, "include"),
            src, "-o"]


def _build_binding(cmd, verbose):
    """The library stands without the binding: a failure is reported here, and
    the calls that go through it raise.  An outdated binding does not stay."""
    if cmd is None:
        return
    part = f"{BINDING}.{os.getpid()}"
    try:
        r = subprocess.run(cmd + [part], capture_output=True, text=True)
        said, ok = r.stdout + r.stderr, r.returncode == 0
    except OSError as e:
        said, ok = f"{e}\n", False
    if verbose or not ok:
        sys.stderr.write(" ".join(cmd + [part]) + "\n" + said)
    if ok:
        os.replace(part, BINDING)
    else:
        with contextlib.suppress(FileNotFoundError):
            os.remove(BINDING)
        sys.stderr.write("the Python binding is not built: calls of the residual block's norms, of "
                         "gradient lists, of the router's losses and of updates will raise\n")


def build_library(verbose: bool = False, ptxas_info: bool = False, force: bool = False) -> str:
    """Compile (if needed) and return the path of libmoe.so; the Python binding
    too, where it can be."""
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    headers = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    headers.append(os.path.join(ROOT, "include", "moe.h"))
    objs, jobs = [], []
    for src in sources():
        obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
        objs.append(obj)
        if force or _stale(obj, [src] + headers):
            cmd = [nvcc] + NVCC_FLAGS + (["-Xptxas", "-v"] if ptxas_info else []) + ["-c", src, "-o", obj]
            jobs.append(cmd)
    binding = _binding_job(nvcc, headers[-1], force)

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs) + 1, os.cpu_count() or 4))) as ex:
        beside = ex.submit(_build_binding, binding, verbose)
        for cmd, r in ex.map(run, jobs):
            if verbose or ptxas_info or r.returncode != 0:
                sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
            if r.returncode != 0:
                raise RuntimeError("compilation failed for " + cmd[-3])
        beside.result()
    if force or jobs or _stale(LIB, objs):
        cmd = [nvcc] + ARCH + ["-shared", "-o", LIB] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if verbose or r.returncode != 0:
            sys.stderr.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError("link of libmoe.so failed")
    return LIB


if __name__ == "__main__":
    build_library(verbose=True, ptxas_info="--ptxas" in sys.argv, force="--force" in sys.argv)
    print(LIB)
