"""Build libmamba_scan.so (gfx950) in-tree with hipcc.

    python -m selective_state_space_06_amd.build

Every HIP source is compiled for gfx950 only, with packed-fp32 instruction selection
turned off (-Xclang -target-feature -Xclang -packed-fp32-ops): plain fp32 VALU code.
The host pass warns that it does not know that feature; the warning is harmless.
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys

PKG_DIR = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG_DIR)
CSRC = os.path.join(PKG_DIR, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB_NAME = "libmamba_scan.so"
LIB_PATH = os.path.join(PKG_DIR, LIB_NAME)
SOURCES = ["abi.hip", "scan_fwd.hip", "scan_fast.hip", "scan_bwd.hip", "state_update.hip", "conv1d.hip",
           "ssd_scan.hip", "gated_scan.hip", "conv1d_bwd.hip", "beam.hip", "abi_recurrent.hip",
           "rms_norm.hip", "linear_attention.hip", "token_logprobs.hip", "abi_layers.hip"]
ARCH = "gfx950"


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found (set HIPCC or install ROCm under /opt/rocm)")


def compile_flags() -> list[str]:
    return ["-O3", "-std=c++17", f"--offload-arch={ARCH}", "-fPIC",
            "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
            "-Wno-unused-command-line-argument", "-I", INCLUDE, "-I", CSRC]


EXAMPLE_SRC = os.path.join(PKG_DIR, "examples", "scan_from_c.c")
EXAMPLE_BIN = os.path.join(PKG_DIR, "examples", "scan_from_c")


def build_example(verbose: bool = False) -> str:
    """Compile the plain-C example against the built library (host code only: gcc and the HIP
    runtime's C API). Returns the executable's path."""
    rocm = os.environ.get("ROCM_PATH", "/opt/rocm")
    cmd = [os.environ.get("CC", "gcc"), "-std=c11", "-O2", "-Wall", "-Wextra", "-D__HIP_PLATFORM_AMD__",
           "-I", os.path.join(rocm, "include"), "-I", INCLUDE, EXAMPLE_SRC, "-L", PKG_DIR, "-lmamba_scan",
           "-L", os.path.join(rocm, "lib"), "-lamdhip64", "-Wl,-rpath,$ORIGIN/..",
           "-Wl,-rpath," + os.path.join(rocm, "lib"), "-o", EXAMPLE_BIN]
    if verbose:
        print(" ".join(cmd), flush=True)
    proc = subprocess.run(cmd, capture_output=True, text=True)
    if proc.returncode != 0:
        sys.stderr.write(proc.stdout + proc.stderr)
        raise RuntimeError(f"compiling the C example failed with exit code {proc.returncode}")
    return EXAMPLE_BIN


NATIVE_SRC = os.path.join(CSRC, "native_calls.c")
NATIVE_LIB = os.path.join(PKG_DIR, "_native.so")


def have_python_headers() -> bool:
    import sysconfig
    return os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h"))


def build_native(verbose: bool = False) -> str:
    """Compile the CPython module `_native` (host code only) against the built library, which it finds
    beside itself. Returns its path."""
    import sysconfig
    tmp = NATIVE_LIB + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CC", "gcc"), "-std=c11", "-O2", "-Wall", "-Wextra", "-fPIC", "-shared", "-I", INCLUDE,
           "-I", sysconfig.get_paths()["include"], NATIVE_SRC, "-L", PKG_DIR, "-lmamba_scan", "-Wl,-rpath,$ORIGIN",
           "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    proc = subprocess.run(cmd, capture_output=True, text=True)
    if proc.returncode != 0:
        sys.stderr.write(proc.stdout + proc.stderr)
        raise RuntimeError(f"compiling native_calls.c failed with exit code {proc.returncode}")
    os.replace(tmp, NATIVE_LIB)
    return NATIVE_LIB


def calls_in(obj: str) -> int | None:
    """The call instructions in an object file's gfx950 code (None: the compiler came without the tools
    that tell, or with others)."""
    import tempfile
    roots = (os.environ.get("ROCM_PATH"), os.path.dirname(os.path.dirname(hipcc())), "/opt/rocm")
    dirs = [os.path.join(r, "llvm", "bin") for r in roots if r]
    need = ("llvm-objdump", "llvm-objcopy", "clang-offload-bundler")
    tools = next((d for d in dirs if all(os.path.exists(os.path.join(d, t)) for t in need)), None)
    if tools is None:
        return None

    def run(tool, *args):
        return subprocess.run([os.path.join(tools, tool), *args], capture_output=True, text=True, check=True).stdout

    with tempfile.TemporaryDirectory() as d:
        fat, code = os.path.join(d, "fat"), os.path.join(d, "code")
        if ".hip_fatbin" not in run("llvm-objdump", "-h", obj):
            return 0
        try:
            run("llvm-objcopy", f"--dump-section=.hip_fatbin={fat}", obj, os.path.join(d, "rest"))
            run("clang-offload-bundler", "--unbundle", "--type=o", f"--targets=hipv4-amdgcn-amd-amdhsa--{ARCH}",
                f"--input={fat}", f"--output={code}")
            asm = run("llvm-objdump", "-d", "--no-show-raw-insn", code)
        except subprocess.CalledProcessError:
            return None
    return sum("s_swappc_b64" in line or "s_call_b64" in line for line in asm.splitlines())


def build(verbose: bool = False, extra: list[str] | None = None) -> str:
    """Compile every source (in parallel, one object each) and link them into LIB_PATH
    (atomically replaced), then the C example and, where Python's headers are, the `_native` module
    against it. Returns the library's path."""
    from concurrent.futures import ThreadPoolExecutor

    objdir = os.path.join(PKG_DIR, "_build")
    os.makedirs(objdir, exist_ok=True)

    def compile_one(src: str) -> str:
        obj = os.path.join(objdir, os.path.splitext(src)[0] + ".o")
        cmd = [hipcc(), *compile_flags(), *(extra or []), "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        proc = subprocess.run(cmd, capture_output=True, text=True)
        if proc.returncode != 0:
            sys.stderr.write(proc.stdout + proc.stderr)
            raise RuntimeError(f"hipcc failed on {src} with exit code {proc.returncode}")
        calls = calls_in(obj)
        if calls:  # moves between lanes and barriers are written for one body of code
            raise RuntimeError(f"{src}: the compiler left {calls} calls in its kernels; mark the functions MSS_INLINED")
        return obj

    jobs = max(1, min(len(SOURCES), os.cpu_count() or 1, 16))
    with ThreadPoolExecutor(max_workers=jobs) as ex:
        objs = list(ex.map(compile_one, SOURCES))
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [hipcc(), f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    proc = subprocess.run(cmd, capture_output=True, text=True)
    if proc.returncode != 0:
        sys.stderr.write(proc.stdout + proc.stderr)
        raise RuntimeError(f"linking failed with exit code {proc.returncode}")
    os.replace(tmp, LIB_PATH)
    build_example(verbose)
    if have_python_headers():
        build_native(verbose)
    else:  # the library is whole without it; its absence is reported where it is used
        sys.stderr.write("Python's headers are missing: _native, which the torch front end of the gated scan, the conv's "
                         "gradients, beam search, norms, linear attention and log probabilities needs, is not built\n")
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose=True))
