"""Build libmlora.so in-tree with hipcc for gfx950 (CDNA4), and the Python module _marshal beside it.

Every .hip and .cpp file of csrc/ is compiled to an object in parallel, then linked into
lora_serving_amd/libmlora.so.  All device code is built with the packed-FP32 feature switched
off (the host pass warns that it does not know the feature; that is harmless).
"""
from __future__ import annotations

import concurrent.futures
import glob
import importlib.util
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libmlora.so")
MARSHAL = os.path.join(PKG, "_marshal.so")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

FLAGS = [f"--offload-arch={ARCH}", "-O3", "-std=c++17", "-fPIC", "-Wall", "-Wno-unused-function",
         "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops", "-I", INCLUDE, "-I", CSRC]


def sources():
    return (sorted(glob.glob(os.path.join(CSRC, "*.hip"))) +
            sorted(glob.glob(os.path.join(CSRC, "*.cpp"))))


def _compile(src: str) -> str:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    lang = ["-x", "hip"] if src.endswith(".hip") else []
    cmd = [HIPCC, *FLAGS, *lang, "-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    out = "\n".join(l for l in (r.stdout + r.stderr).splitlines()
                    if "packed-fp32-ops" not in l)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on {src}:\n{out}")
    if out.strip():
        print(out, file=sys.stderr)
    return obj


def build(jobs: int = 8) -> str:
    os.makedirs(BUILD, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=jobs) as ex:
        objs = list(ex.map(_compile, sources()))
    tmp = LIB + f".tmp{os.getpid()}"
    subprocess.run([HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp],
                   check=True)
    os.replace(tmp, LIB)
    build_marshal()
    return LIB


def build_marshal() -> str | None:
    """The binding's marshalling (csrc/python/marshal.cpp): host code over torch's tensor API.  None, and no
    module, where torch is not installed: the C library stands without it."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        if os.path.exists(MARSHAL):
            os.remove(MARSHAL)
        print("torch is not installed: libmlora.so without its Python binding", file=sys.stderr)
        return None
    torch = os.path.dirname(spec.origin)
    tmp = MARSHAL + f".tmp{os.getpid()}"
    cmd = [HIPCC, "-x", "c++", "-O2", "-std=c++17", "-fPIC", "-shared", "-no-hip-rt",
           "-D__HIP_PLATFORM_AMD__", "-I", INCLUDE, "-isystem", "/opt/rocm/include", "-isystem",
           os.path.join(torch, "include"), "-isystem",
           os.path.join(torch, "include", "torch", "csrc", "api", "include"), "-isystem",
           sysconfig.get_paths()["include"], os.path.join(CSRC, "python", "marshal.cpp"), "-o", tmp,
           "-L", PKG, "-lmlora", "-Wl,-rpath,$ORIGIN", "-L", os.path.join(torch, "lib"), "-lc10",
           "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed on marshal.cpp:\n{r.stdout + r.stderr}")
    os.replace(tmp, MARSHAL)
    return MARSHAL


if __name__ == "__main__":
    print(build())
