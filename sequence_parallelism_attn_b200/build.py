"""Build libra_b200.so in-tree from csrc/*.cu with nvcc for sm_100a.

Every translation unit is compiled with
  nvcc -gencode arch=compute_100a,code=sm_100a -lineinfo -O3 -std=c++17 -Xcompiler -fPIC
and linked with the static CUDA runtime into one shared library whose only exported
symbols are the ra_* entry points of include/ra.h (a linker version script hides the
static runtime, so it can never bind to another copy loaded in the same process).  Beside
it _ra_torch.so, the native Python binding of the operators that run once per token
(csrc/binding.cpp, g++ against torch's headers).
"""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
LIB = os.path.join(HERE, "libra_b200.so")
NATIVE = os.path.join(HERE, "_ra_torch.so")
BINDING = "binding.cpp"
BUILD_DIR = os.path.join(HERE, "_build")
SOURCES = ["api.cu", "attn_sm100.cu", "attn_bwd_sm100.cu", "bwd_static.cu", "attn_fp32.cu",
           "lse_merge.cu", "permute.cu", "api_kv.cu", "paged_append.cu", "kv_rows.cu",
           "cross_bwd.cu", "kv_tiles_sm100.cu", "kv_cluster.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler",
              "-fvisibility=hidden", f"-I{INCLUDE}", f"-I{CSRC}"]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.sep not in cand or os.path.exists(cand)):
            return cand
    return "nvcc"


def _mtime(*files: str) -> float:
    return max(os.path.getmtime(f) for f in (*files, os.path.abspath(__file__)))


def _deps_mtime() -> float:
    return _mtime(*(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f != BINDING),
                  os.path.join(INCLUDE, "ra.h"))


def _run(cmd, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), file=sys.stderr)
    subprocess.run(cmd, check=True)


def build_native(force: bool = False, verbose: bool = False) -> str:
    """The native Python module over the library (csrc/binding.cpp), linked to it by a path
    relative to itself."""
    import sysconfig

    import torch
    src = os.path.join(CSRC, BINDING)
    # it holds torch's and Python's ABI, so it is out of date too when one of them has changed
    stamp = os.path.join(BUILD_DIR, "native.stamp")
    built_for = f"torch {torch.__version__}, Python {sys.version}"
    if not force and os.path.exists(NATIVE) and os.path.exists(stamp) and \
            os.path.getmtime(NATIVE) >= _mtime(src, os.path.join(INCLUDE, "ra.h")):
        with open(stamp) as f:
            if f.read() == built_for:
                return NATIVE
    root = os.path.dirname(os.path.abspath(torch.__file__))
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    tmp = NATIVE + ".tmp"
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-shared",
          f"-I{root}/include", f"-I{root}/include/torch/csrc/api/include", f"-I{cuda}/include",
          f"-I{sysconfig.get_paths()['include']}", src, "-o", tmp, f"-L{root}/lib", "-ltorch",
          "-ltorch_cpu", "-ltorch_python", "-lc10", "-lc10_cuda", f"-L{HERE}",
          f"-l:{os.path.basename(LIB)}", "-Wl,-rpath,$ORIGIN"], verbose)
    os.replace(tmp, NATIVE)
    os.makedirs(BUILD_DIR, exist_ok=True)
    with open(stamp, "w") as f:
        f.write(built_for)
    return NATIVE


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Build what is out of date (the library, then the native module); returns the library."""
    if force or not os.path.exists(LIB) or os.path.getmtime(LIB) < _deps_mtime():
        os.makedirs(BUILD_DIR, exist_ok=True)
        nvcc = _nvcc()
        cmds, objs = [], []
        for src in SOURCES:
            obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
            cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
            if ptxas_info:
                cmd.insert(1, "-Xptxas=-v")
            cmds.append(cmd)
            objs.append(obj)
        with ThreadPoolExecutor(max_workers=os.cpu_count() or 1) as pool:
            list(pool.map(lambda cmd: _run(cmd, verbose), cmds))
        vscript = os.path.join(BUILD_DIR, "exports.map")
        with open(vscript, "w") as f:
            f.write("{ global: ra_*; local: *; };\n")
        tmp = LIB + ".tmp"
        _run([nvcc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs,
              "-Xlinker", f"--version-script={vscript}", "-Xlinker", "--exclude-libs,ALL"],
             verbose)
        os.replace(tmp, LIB)
    build_native(force, verbose)
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas-info" in sys.argv)
    print(LIB)
