"""The build of the native calls: optional, and free where nothing has changed (no GPU, no compiler: the compiler is a stand-in)."""
import os
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

SCRIPT = """
import importlib.util, os, sys
spec = importlib.util.spec_from_file_location("standalone_build", {path!r})
b = importlib.util.module_from_spec(spec)
spec.loader.exec_module(b)
b.BUILD_DIR, b.NATIVE_PATH = {tmp!r}, os.path.join({tmp!r}, "_native.so")
b._build_library = lambda force, verbose: "the library"

class Done:
    returncode, stderr, stdout = 0, "", ""

def compiler(cmd, **kw):
    open(cmd[cmd.index("-o") + 1], "w").write("compiled")
    return Done

b.subprocess.run = compiler
{before}
print(b.build(), b.build_native(), "torch" in sys.modules and sys.modules["torch"] is not None, os.path.exists(b.NATIVE_PATH))
"""


def run(tmp, before=""):
    path = os.path.join(ROOT, "kda_chunked_prefill_gb300", "build.py")
    r = subprocess.run([sys.executable, "-c", SCRIPT.format(path=path, tmp=str(tmp), before=before)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return r.stdout.split("\n")[0], r.stderr


def test_without_torch_the_library_is_built_and_the_native_calls_left_out(tmp_path):
    out, err = run(tmp_path, 'sys.modules["torch"] = None  # (not installed)')
    assert out == "the library False False False" and "_native.so is left out" in err


def test_an_unchanged_build_does_not_import_torch(tmp_path):
    assert run(tmp_path)[0] == "the library True True True"
    assert run(tmp_path)[0] == "the library True False True"


def test_a_compiler_that_fails_leaves_the_native_calls_out(tmp_path):
    assert run(tmp_path)[0].startswith("the library True")
    out, err = run(tmp_path, 'Done.returncode, Done.stderr = 1, "no such header"\nopen(os.path.join(b.BUILD_DIR, "native_stamp"), "w").close()')
    assert out == "the library False True False" and "no such header" in err


def test_native_calls_of_another_torch_are_not_used():
    """What was compiled against one torch reads tensors by that one's layout: beside another the general calls are taken."""
    script = """
import sys, types, torch
import kda_chunked_prefill_gb300 as kda
from kda_chunked_prefill_gb300 import _lib
used = []
native = types.ModuleType("kda_chunked_prefill_gb300._native")
native.set_entry = lambda *a: used.append(len(a))
{version}
sys.modules["kda_chunked_prefill_gb300._native"] = kda._native = native
_lib.load_library(build_if_missing=True)
print(used, _lib._native is native)
"""
    for version, want in (("native.torch_version = torch.__version__", "[5] True"), ("native.torch_version = '1.0.0'", "[] False"),
                          ("", "[] False")):
        r = subprocess.run([sys.executable, "-c", script.format(version=version)], capture_output=True, text=True, cwd=ROOT)
        assert r.returncode == 0 and r.stdout.strip() == want, (version, r.stdout, r.stderr)


def test_native_calls_name_their_torch():
    import pytest
    import torch

    from kda_chunked_prefill_gb300 import _lib
    _lib.load_library(build_if_missing=True)
    if _lib._native is None:
        pytest.skip("the native calls are not built")
    assert _lib._native.torch_version == torch.__version__
