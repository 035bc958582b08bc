"""Build libdq.so in-tree with nvcc for sm_100a, and _dq_torch.*.so (argument marshalling) with the
host compiler.

    python -m calibration_free_weight_dualquant_b200.build
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
import sysconfig
import warnings
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "lib")
LIB = os.path.join(OUT_DIR, "libdq.so")
MARSHAL_SOURCE = os.path.join(CSRC, "dq_torch.cpp")
SOURCES = ["dq_capi.cu", "dq_solver.cu", "dq_static.cu", "dq_act.cu", "dq_norm.cu", "dq_matmul.cu"]
HEADERS = ["dq_device.cuh", "dq_fast.cuh", "dq_init.cuh", "dq_internal.h", "dq_iter.cuh", "dq_launch.h",
           "dq_tc.cuh"]

ARCH_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2", "--expt-relaxed-constexpr",
              "-Xptxas", "-v"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _stale() -> bool:
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    deps = [os.path.join(CSRC, f) for f in SOURCES + HEADERS] + [os.path.join(INCLUDE, "dq.h")]
    return any(os.path.getmtime(d) > t for d in deps)


def _run(cmd, what: str) -> str:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        sys.stderr.write(r.stdout + r.stderr)
        raise RuntimeError("%s failed" % what)
    return r.stdout + r.stderr


def marshal_path() -> str:
    """Where the compiled marshalling for this interpreter and this torch belongs: its name holds their binary
    interfaces, so a module built against others is neither kept nor loaded."""
    import torch
    name = "_dq_torch.%s-torch%s-abi%d.so" % (sysconfig.get_config_var("SOABI"), torch.__version__,
                                              torch._C._GLIBCXX_USE_CXX11_ABI)
    return os.path.join(OUT_DIR, name)


def build_marshal(force: bool = False) -> str:
    """The CPython module of csrc/dq_torch.cpp, against torch's headers and libdq.so."""
    import torch
    path = marshal_path()
    deps = [MARSHAL_SOURCE, os.path.join(INCLUDE, "dq.h")]
    if not force and os.path.exists(path) and all(os.path.getmtime(d) <= os.path.getmtime(path) for d in deps):
        return path
    t = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(nvcc())), "include")
    includes = [sysconfig.get_paths()["include"], os.path.join(t, "include"),
                os.path.join(t, "include", "torch", "csrc", "api", "include"), cuda, INCLUDE]
    tmp = path + ".tmp%d" % os.getpid()
    cmd = [shutil.which("g++") or "c++", "-O2", "-std=c++17", "-shared", "-fPIC"]
    cmd += [a for d in includes for a in ("-I", d)]
    cmd += ["-D_GLIBCXX_USE_CXX11_ABI=%d" % torch._C._GLIBCXX_USE_CXX11_ABI, MARSHAL_SOURCE, "-o", tmp, "-L", OUT_DIR,
            "-l:libdq.so", "-Wl,-rpath,$ORIGIN", "-L", os.path.join(t, "lib"), "-lc10", "-ltorch_cpu", "-ltorch_cuda",
            "-ltorch_python"]
    _run(cmd, "g++ on dq_torch.cpp")
    os.replace(tmp, path)
    return path


def build(force: bool = False, verbose: bool = False) -> str:
    """Build what is stale; returns libdq.so.  The solver and dq_act_quant need nothing else, so a marshalling module
    that cannot be built (no Python or torch headers) is a warning here; the linear layer's calls raise without it."""
    if force or _stale():
        os.makedirs(OUT_DIR, exist_ok=True)

        def compile_one(src):
            obj = os.path.join(OUT_DIR, src.replace(".cu", ".o"))
            return obj, _run([nvcc()] + ARCH_FLAGS + NVCC_FLAGS + ["-I", INCLUDE, "-I", CSRC, "-dc", "-o", obj,
                                                                  os.path.join(CSRC, src)], "nvcc on %s" % src)

        with ThreadPoolExecutor(max(1, min(len(SOURCES), os.cpu_count() or 1))) as pool:
            done = list(pool.map(compile_one, SOURCES))
        tmp = LIB + ".tmp%d" % os.getpid()
        _run([nvcc()] + ARCH_FLAGS + ["-shared", "-Xcompiler", "-fPIC", "-o", tmp] + [obj for obj, _ in done], "nvcc link")
        os.replace(tmp, LIB)
        log = "\n".join(text for _, text in done)
        with open(os.path.join(OUT_DIR, "ptxas.log"), "w") as f:
            f.write(log)
        if verbose:
            print(log)
    try:
        build_marshal(force)
    except (ImportError, OSError, RuntimeError) as e:
        warnings.warn("the linear layer's calls will not work from Python: %s" % e)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
