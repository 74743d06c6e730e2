"""Build ``libkda.so`` (the C-ABI library) in-tree with nvcc for sm_103a.

Each ``csrc/*.cu`` file is compiled to an object in parallel, then linked
into ``kda_chunked_prefill_gb300/libkda.so``. No CMake, no torch extension
machinery: the library has a plain C ABI (``include/kda.h``). Beside it, g++
compiles ``csrc/kda_binding.cpp`` into ``_native.so``, the plain calls of the
binding as native code; it depends on the installed torch, and the binding works
without it (slower on the host).
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import hashlib
import os
import re
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_PATH = os.path.join(PKG, "libkda.so")
NATIVE_SOURCE = os.path.join(CSRC, "kda_binding.cpp")
NATIVE_PATH = os.path.join(PKG, "_native.so")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
              "-Xptxas", "-warn-spills"]


def nvcc() -> str:
    home = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    path = os.path.join(home, "bin", "nvcc")
    return path if os.path.exists(path) else (shutil.which("nvcc") or "nvcc")


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stamp() -> str:
    h = hashlib.sha256()
    for f in _sources() + sorted(glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))) + \
            sorted(glob.glob(os.path.join(INCLUDE, "*.h"))) + [__file__]:
        h.update(os.path.relpath(f, ROOT).encode())
        with open(f, "rb") as fh:
            h.update(fh.read())
    h.update(" ".join(ARCH + NVCC_FLAGS).encode())
    return h.hexdigest()


def _local_includes(path: str, seen: set) -> None:
    """Add `path` and, transitively, the csrc headers it includes with quotes."""
    if path in seen:
        return
    seen.add(path)
    with open(path, encoding="utf-8") as fh:
        for line in fh:
            m = re.match(r'\s*#\s*include\s+"([^"]+)"', line)
            if m:
                dep = os.path.join(CSRC, m.group(1))
                if os.path.exists(dep):
                    _local_includes(dep, seen)


def kernel_stamp(source: str) -> str:
    """Hash of one kernel's translation unit: its .cu file, the csrc headers it
    includes (transitively), and the compile flags. A change elsewhere (another
    kernel, the host API and its documentation in include/, a header this file
    does not include) leaves it unchanged."""
    files: set = set()
    _local_includes(os.path.join(CSRC, source), files)
    h = hashlib.sha256()
    for f in sorted(files):
        h.update(os.path.relpath(f, ROOT).encode())
        with open(f, "rb") as fh:
            h.update(fh.read())
    h.update(" ".join(ARCH + NVCC_FLAGS).encode())
    return h.hexdigest()


def build_native(force: bool = False) -> bool:
    """Compile ``_native.so`` against the installed torch; skipped when nothing has
    changed. False, with a note on stderr, where that does not work."""
    import importlib.util
    import sysconfig

    os.makedirs(BUILD_DIR, exist_ok=True)
    spec = importlib.util.find_spec("torch")  # (found, not imported: an unchanged build does not pay for that)
    if spec is not None and spec.origin:
        where = os.path.dirname(spec.origin)
        cuda = os.environ.get("CUDA_HOME", "/usr/local/cuda")
        tmp = NATIVE_PATH + f".tmp{os.getpid()}"
        cmd = ["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-I", INCLUDE,
               *(f for d in ("include", "include/torch/csrc/api/include") for f in ("-isystem", os.path.join(where, d))),
               "-isystem", os.path.join(cuda, "include"), "-isystem", sysconfig.get_paths()["include"], NATIVE_SOURCE,
               "-L" + os.path.join(where, "lib"), "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-ltorch_python"]
        h = hashlib.sha256((sys.version + " ".join(cmd)).encode())
        for f in (NATIVE_SOURCE, os.path.join(INCLUDE, "kda.h"), os.path.join(where, "version.py")):
            if os.path.exists(f):
                with open(f, "rb") as fh:
                    h.update(fh.read())
        stamp_file = os.path.join(BUILD_DIR, "native_stamp")
        if not force and os.path.exists(NATIVE_PATH) and os.path.exists(stamp_file) and open(stamp_file).read() == h.hexdigest():
            return True
        try:
            import torch
            abi = f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"
            version = f'-DKDA_TORCH_VERSION="{torch.__version__}"'  # (the binding uses it with no other)
            r = subprocess.run([*cmd, abi, version, "-o", tmp], capture_output=True, text=True)
            failed = r.stderr if r.returncode != 0 else None
        except (OSError, ImportError) as e:
            failed = str(e)
    else:
        failed = "torch is not installed"
    if failed is not None:
        if os.path.exists(NATIVE_PATH):
            os.remove(NATIVE_PATH)
        sys.stderr.write(f"_native.so is left out:\n{failed}\n")
        return False
    os.replace(tmp, NATIVE_PATH)
    with open(stamp_file, "w") as fh:
        fh.write(h.hexdigest())
    return True


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile and link; skipped when the sources are unchanged since the last build."""
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        native = ex.submit(build_native, force)
        path = _build_library(force, verbose)
        native.result()
    return path


def _build_library(force: bool, verbose: bool) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    stamp_file = os.path.join(BUILD_DIR, "stamp")
    stamp = _stamp()
    if not force and os.path.exists(LIB_PATH) and os.path.exists(stamp_file):
        if open(stamp_file).read() == stamp:
            return LIB_PATH
    extra = ["-Xptxas", "-v"] if verbose else []

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [nvcc(), *ARCH, *NVCC_FLAGS, *extra, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
        results = list(ex.map(compile_one, _sources()))
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc(), *ARCH, "-shared", "-o", tmp, *[o for o, _ in results], "-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB_PATH)
    with open(stamp_file, "w") as fh:
        fh.write(stamp)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
