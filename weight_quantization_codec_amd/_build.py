"""Build libqamw.so in-tree with hipcc for gfx950."""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libqamw.so")
HOST = os.path.join(PKG, "_w8_host.so")
BUILD_DIR = os.path.join(ROOT, "_build", "qamw")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC",
    # distances and butterflies are specified as separately rounded IEEE operations
    "-ffp-contract=off",
    # no packed fp32 instructions (v_pk_add_f32 / v_pk_mul_f32 / v_pk_fma_f32)
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wno-unused-command-line-argument",
]


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.hip")))


def _compile(src: str) -> str:
    obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
    cmd = [HIPCC] + FLAGS + ["-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("hipcc failed for %s:\n%s\n%s" % (src, " ".join(cmd), r.stderr[-6000:]))
    return obj


def build(jobs: int = 8) -> str:
    """Compile every HIP source for gfx950 and link libqamw.so (always rebuilds)."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        objs = list(ex.map(_compile, sources()))
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [HIPCC, "--offload-arch=gfx950", "-shared", "-fPIC", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s" % r.stderr[-4000:])
    os.replace(tmp, LIB)
    return LIB


def build_host() -> str:
    """Compile the binding's host module (csrc/w8_host.cpp, mx4_host.cpp) against the installed torch.  Where that fails
    no older module stays: w8.py and mx4.py do without one."""
    import sysconfig

    from torch.utils import cpp_extension
    tmp = HOST + ".tmp%d" % os.getpid()
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1", "-I", INCLUDE, "-I", CSRC, "-I", sysconfig.get_paths()["include"]]
    for d in cpp_extension.include_paths("cuda"):
        cmd += ["-isystem", d]
    cmd += [os.path.join(CSRC, "w8_host.cpp"), os.path.join(CSRC, "mx4_host.cpp"), "-o", tmp]
    for d in cpp_extension.library_paths():
        cmd += ["-L", d]
    cmd += ["-ltorch_python", "-ltorch_cpu", "-ltorch_hip", "-lc10", "-lc10_hip"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        failure = r.stderr[-4000:] if r.returncode else None
    except OSError as e:   # no such compiler
        failure = str(e)
    if failure is not None:
        if os.path.exists(HOST):
            os.remove(HOST)
        raise RuntimeError("g++ failed for w8_host.cpp, mx4_host.cpp:\n%s\n%s" % (" ".join(cmd), failure))
    os.replace(tmp, HOST)
    return HOST


if __name__ == "__main__":
    print(build())
    print(build_host())
