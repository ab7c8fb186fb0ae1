"""Build libpkd.so in-tree with nvcc for sm_103a.

Each translation unit compiles in its own nvcc process (in parallel); the
objects are linked into ``paged_kv_decode_host_gb300/libpkd.so``.  No CMake.
Beside it, when the Python headers are installed, the host C compiler builds
``_pkd_plan``: the binding's argument-marshalling fast path for the per-step
plan calls (the binding falls back to ctypes without it), and the host C++
compiler ``_pkd_step``, which takes the calls of a step with drafts on torch's
tensors directly (likewise).  What either was built from (its source, Python,
torch) is kept beside the objects, with the outcome: one that cannot be built is
tried again only when something of that changes, and no old one stays.
"""
from __future__ import annotations

import contextlib
import hashlib
import importlib.metadata
import importlib.util
import os
import platform
import shutil
import subprocess
import sys
import sysconfig
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libpkd.so")
SOURCES = ["planner.cpp", "api.cu", "decode_kernel.cu", "prefix_tc_kernel.cu",
           "merge_kernels.cu", "static_scratch.cu", "append_kernel.cu", "selftest.cu",
           "latent_kernel.cu", "weights_kernel.cu", "evict_kernel.cu", "plan_tree.cpp",
           "tree_kernel.cu", "rotate_kernel.cu", "accept_kernel.cu", "api_step.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
_SUFFIX = sysconfig.get_config_var("EXT_SUFFIX") or ".so"
PYPLAN = os.path.join(HERE, "_pkd_plan" + _SUFFIX)
PYSTEP = os.path.join(HERE, "_pkd_step" + _SUFFIX)


def _python_include():
    inc = sysconfig.get_paths().get("include")
    return inc if inc and os.path.exists(os.path.join(inc, "Python.h")) else None


def _torch_dir():
    spec = importlib.util.find_spec("torch")
    d = spec.submodule_search_locations[0] if spec and spec.submodule_search_locations else None
    return d if d and os.path.exists(os.path.join(d, "include", "ATen")) else None


def _torch_version():
    try:
        return importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        return ""


def _plan_command():
    """The C compiler's command for _pkd_plan; None without it or the Python headers."""
    inc, cc = _python_include(), shutil.which("cc") or shutil.which("gcc")
    if inc is None or cc is None:
        return None
    return [cc, "-O2", "-shared", "-fPIC", f"-I{inc}", os.path.join(CSRC, "pyplan.c")]


def _step_command():
    """The C++ compiler's command for _pkd_step; None without it, the CUDA toolkit, torch or the
    Python headers."""
    inc, torch_dir = _python_include(), _torch_dir()
    cxx = shutil.which("c++") or shutil.which("g++")
    try:
        cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    except RuntimeError:
        return None
    if inc is None or torch_dir is None or cxx is None:
        return None
    dirs = [INCLUDE, inc, os.path.join(torch_dir, "include"), cuda]
    return [cxx, "-O2", "-std=c++17", "-shared", "-fPIC", *[f"-I{d}" for d in dirs],
            f'-DPKD_TORCH="{_torch_version().split("+")[0]}"', os.path.join(CSRC, "pystep.cpp"),
            "-L" + os.path.join(torch_dir, "lib"), "-lc10", "-ltorch_cpu", "-ltorch_python",
            "-lc10_cuda"]


def _optional():
    """(module, its command, the file that keeps what it was built from, that) of those that
    can be built here; what is there of others stays."""
    for path, command in ((PYPLAN, _plan_command()), (PYSTEP, _step_command())):
        if command is None:
            continue
        # (not where compilers and headers lie: another shell's PATH is no reason to build anew)
        h = hashlib.sha256("\0".join([sys.version, platform.machine(), _torch_version()]).encode())
        for f in ("csrc/pyplan.c", "csrc/pystep.cpp", "../include/pkd.h"):
            with open(os.path.join(HERE, f), "rb") as src:
                h.update(src.read())
        yield path, command, os.path.join(BUILD, os.path.basename(path) + ".key"), h.hexdigest()


def _optional_stale(path, command, kept, key):
    try:
        with open(kept) as f:
            was, outcome = f.read().rsplit(" ", 1)
    except (OSError, ValueError):
        return True
    return was != key or os.path.exists(path) != (outcome == "built")


def _build_optional(path, command, kept, key):
    for old in (kept, path):   # (an old module must not be loaded beside a new libpkd)
        with contextlib.suppress(FileNotFoundError):
            os.remove(old)
    tmp = path + f".tmp{os.getpid()}"
    r = subprocess.run([*command, "-o", tmp], capture_output=True, text=True)
    built = r.returncode == 0
    if built:
        os.replace(tmp, path)
    else:
        sys.stderr.write(f"{os.path.basename(path)} not built (general path used):\n"
                         f"{r.stderr[-2000:]}\n")
    with open(kept, "w") as f:
        f.write(f"{key} {'built' if built else 'failed'}")


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _flags():
    return ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
            "-Xcompiler", "-fno-strict-aliasing", f"-I{INCLUDE}", f"-I{CSRC}"] + ARCH


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "pkd.h")]
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    modules, stale = [m for m in _optional() if force or _optional_stale(*m)], force or _stale()
    if modules or stale:
        os.makedirs(BUILD, exist_ok=True)
    if not stale:
        for m in modules:
            _build_optional(*m)
        return LIB
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, src + ".o")
        lang = ["-x", "cu"] if src.endswith(".cu") else []
        cmd = [nvcc, "-c", *lang, os.path.join(CSRC, src), "-o", obj, *_flags(), *extra_flags]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose and (r.stdout or r.stderr):
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 2) as ex:
        others = [ex.submit(_build_optional, *m) for m in modules]
        objs = list(ex.map(compile_one, SOURCES))
        for m in others:
            m.result()
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, "-shared", "-o", tmp, *objs, *ARCH, "-Xcompiler", "-fPIC", "-lpthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                extra_flags=["-Xptxas", "-v"] if "--ptxas-v" in sys.argv else ()))
