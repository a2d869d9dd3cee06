"""The build's own checks: kernels are one body of code, without calls."""
import os
import re
import subprocess
from concurrent.futures import ThreadPoolExecutor

import pytest

from selective_state_space_06_amd import build as b


def compiled(src, out, *extra):
    subprocess.run([b.hipcc(), *b.compile_flags(), *extra, "-o", str(out), str(src)], check=True, capture_output=True)
    return str(out)


def test_calls_are_counted(tmp_path):
    text = """#include <hip/hip_runtime.h>
    __device__ float OTHER f(float v) { return v * v + 1.0f; }
    __global__ void k(float* p) { p[threadIdx.x] = f(p[threadIdx.x]); }
    """
    for how, calls in (("__attribute__((noinline))", 1), ("__attribute__((always_inline))", 0)):
        src = tmp_path / f"k{calls}.hip"
        src.write_text(text.replace("OTHER", how))
        assert b.calls_in(compiled(src, tmp_path / f"k{calls}.o", "-c")) == calls
    host = tmp_path / "h.hip"
    host.write_text("int h() { return 1; }\n")
    assert b.calls_in(compiled(host, tmp_path / "h.o", "-c")) == 0


def test_without_the_tools_nothing_is_said(tmp_path, monkeypatch):
    there = os.path.exists
    monkeypatch.setattr(os.path, "exists", lambda p: "llvm" not in str(p) and there(p))
    assert b.calls_in(str(tmp_path / "any.o")) is None


def test_tools_that_refuse_end_no_build(tmp_path, monkeypatch):
    src = tmp_path / "k.hip"
    src.write_text("#include <hip/hip_runtime.h>\n__global__ void k(float* p) { p[0] = 1.0f; }\n")
    obj = compiled(src, tmp_path / "k.o", "-c")
    monkeypatch.setattr(b, "ARCH", "gfx90a")  # no such code in the object
    assert b.calls_in(obj) is None


def test_the_library_builds_without_pythons_headers(tmp_path, monkeypatch, capsys):
    """A user of the C library has no use for them; other errors of the module's build still end it."""
    import sysconfig
    paths, made = dict(sysconfig.get_paths(), include=str(tmp_path / "none")), []
    monkeypatch.setattr(b, "SOURCES", ["abi.hip"])  # one small source stands for all; nothing in the tree is replaced
    for name in ("PKG_DIR", "LIB_PATH", "NATIVE_LIB"):
        monkeypatch.setattr(b, name, str(tmp_path / os.path.basename(getattr(b, name)) if name != "PKG_DIR" else tmp_path))
    monkeypatch.setattr(b, "build_example", lambda verbose=False: made.append("example"))
    monkeypatch.setattr(sysconfig, "get_paths", lambda *a, **k: paths)
    native = b.LIB_PATH.replace(b.LIB_NAME, "_native.so")
    assert b.build() == b.LIB_PATH and os.path.exists(b.LIB_PATH)
    assert made == ["example"] and not os.path.exists(native)
    assert "headers are missing" in capsys.readouterr().err
    (tmp_path / "none").mkdir()
    (tmp_path / "none" / "Python.h").write_text("#error no such thing\n")
    with pytest.raises(RuntimeError, match="native_calls"):
        b.build()


def test_built_objects_have_none():
    objs = [os.path.join(b.PKG_DIR, "_build", os.path.splitext(s)[0] + ".o") for s in b.SOURCES]
    if not all(map(os.path.exists, objs)):
        pytest.skip("not built here")
    assert b.calls_in(objs[0]) is not None
    assert [b.calls_in(o) for o in objs] == [0] * len(objs)


def test_lambdas_with_lane_moves_are_inlined_whatever_the_compiler_thinks(tmp_path):
    """Compiled with the compiler's own inlining off, only the two forms of the backward walks' inner lambdas
    (for whole tiles and others) are functions of their own."""
    def lambdas(name):
        out = compiled(os.path.join(b.CSRC, name + ".hip"), tmp_path / (name + ".s"), "-S", "--offload-device-only",
                       "-fno-inline-functions")
        with open(out) as f:
            return {m for m in re.findall(r"^\s*\.type\s+(\S+),@function", f.read(), re.M) if re.search(r"clE|clI", m)}

    with ThreadPoolExecutor(3) as ex:
        gated, conv, beam = ex.map(lambdas, ("gated_scan", "conv1d_bwd", "beam"))
    assert not beam
    for found, kernel in ((gated, "gated_bwd_kernel"), (conv, "conv_bwd_kernel")):
        for m in found:
            assert kernel in m and re.search(r"clINS_(True|False|4TrueE|5FalseE)", m), m
