"""Build libnvfp4moe.so (the C-ABI library) from csrc/*.cu for sm_103a, and
_tensor_calls.so (binding.py's short calls, against the installed torch) from
csrc/tensor_calls.cpp.

One compiler per translation unit, run in parallel, then one link each. The
library links the CUDA runtime statically and reaches the driver's tensor-map
encoder through the runtime's entry-point query, so it needs no -lcuda.
"""
import concurrent.futures as cf
import importlib.util
import os
import subprocess
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libnvfp4moe.so")
CALLS = os.path.join(PKG, "_tensor_calls.so")
SOURCES = ["quantize.cu", "routing.cu", "front.cu", "gemm.cu", "api.cu", "layout.cu", "sorted.cu",
           "fp8_quantize.cu", "fp8_gemm.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I" + INCLUDE, "-I" + CSRC]


def _nvcc():
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".cpp"))]
    files.append(os.path.join(INCLUDE, "nvfp4moe.h"))
    return files


def stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(CALLS):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(CALLS))
    return any(os.path.getmtime(f) > t for f in _inputs())


def _torch_dir():
    return os.path.dirname(importlib.util.find_spec("torch").origin)


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("%s failed:\n%s%s" % (what, r.stdout, r.stderr))
    return r.stdout + r.stderr


def _compile_calls():
    torch = _torch_dir()
    obj = os.path.join(BUILD, "tensor_calls.o")
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())) or "/usr/local/cuda", "include")
    dirs = [INCLUDE, os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
            cuda, sysconfig.get_paths()["include"]]
    log = _run(["g++", "-O2", "-std=c++17", "-fPIC", *("-I" + d for d in dirs), "-c",
                os.path.join(CSRC, "tensor_calls.cpp"), "-o", obj], "g++ for tensor_calls.cpp")
    return obj, log


def _link_calls(obj):
    lib = os.path.join(_torch_dir(), "lib")
    tmp = CALLS + ".tmp%d" % os.getpid()
    _run(["g++", "-shared", "-o", tmp, obj, "-L" + PKG, "-lnvfp4moe", "-Wl,-rpath,$ORIGIN", "-L" + lib,
          "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda", "-Wl,-rpath," + lib], "link of _tensor_calls.so")
    os.replace(tmp, CALLS)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [nvcc, *ARCH, *FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        return obj, _run(cmd, "nvcc for " + src)

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        calls = ex.submit(_compile_calls)
        results = list(ex.map(compile_one, SOURCES))
        calls_obj, _ = calls.result()
    if verbose:
        for _, log in results:
            print(log)
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp] + [o for o, _ in results]
    _run(cmd, "link of libnvfp4moe.so")
    os.replace(tmp, LIB)
    _link_calls(calls_obj)
    return LIB


if __name__ == "__main__":
    print(build(force=True, verbose=True))
