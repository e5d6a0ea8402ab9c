"""Build libtpmlp.so in-tree with nvcc for sm_103a.

Each CUDA translation unit is compiled in parallel, then linked into
``tensor_transformer_mlp_tcgen05_gb300/libtpmlp.so`` (the CUDA runtime is
linked statically; the driver API is reached through the runtime's entry-point
lookup, so the library does not link libcuda).  Object files go to
``_build/`` at the repository root.  A rebuild is skipped when the library is
newer than every source and header.  The library needs the CUDA toolkit only.

Next to it goes ``_pycall``, a Python module (host C++, built against the
installed torch, whose C++ layouts it holds: the versions of Python and torch are
in its file's name) with the tensor calls of ``rotary.py``, ``clip.py`` and
``fp4.py``.  Where torch is not installed it is left out; where it does not compile, build() says
so once the library is linked.

``build(checks=True)`` makes the debug variant ``libtpmlp_checks.so`` (objects
in ``_build/checks``) with ``-DTPMLP_CHECKS``: device-side checks of TMA
coordinates and store indices that report ``TPMLP_ERR_CHECK`` instead of
letting a bad access happen.  Load it by setting ``TPMLP_LIB`` to its path
before the binding is imported.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(ROOT, "_build")
LIB_PATH = os.path.join(PKG, "libtpmlp.so")
CHECKS_LIB_PATH = os.path.join(PKG, "libtpmlp_checks.so")

SOURCES = ["gemm_tc2.cu", "rowops.cu", "simt.cu",
           "tp_mlp_host.cu", "noalloc.cu", "attn_fwd.cu", "attn_bwd.cu",
           "attn_host.cu", "fp8.cu", "probe.cu",
           "qk_rows.cu", "qk_rows_bf16.cu", "qk_rows_fp32.cu", "rope_host.cu",
           "grad_clip.cu", "fp4_quant.cu", "fp4_gemm.cu", "fp4_split.cu",
           "fp4_plain.cu", "fp4_host.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC",
          "--expt-relaxed-constexpr", "-I" + INCLUDE, "-I" + CSRC]


def nvcc_path() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA 13 toolkit is required")


HEADERS = [os.path.join(INCLUDE, f) for f in ("tp_mlp.h", "tp_attn.h",
                                              "tp_rope.h", "tp_grad.h",
                                              "tp_fp4.h")]


def _inputs():
    """What the library is made of."""
    return [os.path.join(CSRC, f) for f in os.listdir(CSRC)
            if f.endswith((".cu", ".cuh", ".h"))] + HEADERS + \
        [os.path.abspath(__file__)]


def _pycall_inputs():
    return [os.path.join(CSRC, "pycall.cpp"), *HEADERS,
            os.path.abspath(__file__)]


def up_to_date(lib_path: str = LIB_PATH, inputs=None) -> bool:
    if not os.path.exists(lib_path):
        return False
    t = os.path.getmtime(lib_path)
    return all(os.path.getmtime(f) <= t for f in inputs or _inputs())


def has_torch() -> bool:
    return importlib.util.find_spec("torch") is not None


def pycall_path() -> str:
    """The file of the module for this Python and this torch."""
    import torch
    return os.path.join(PKG, f"_pycall-{sys.implementation.cache_tag}"
                             f"-torch-{torch.__version__}.so")


def build_pycall(force: bool = False) -> str:
    """Compile the Python module with the host compiler; returns its path."""
    path = pycall_path()
    if not force and up_to_date(path, _pycall_inputs()):
        return path
    import torch
    from torch.utils import cpp_extension
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        raise RuntimeError("g++ not found")
    nvcc_inc = os.path.join(os.path.dirname(os.path.dirname(nvcc_path())),
                            "include")
    inc = [*cpp_extension.include_paths(), nvcc_inc,
           sysconfig.get_paths()["include"], INCLUDE]
    tmp = path + ".tmp"
    cmd = [cxx, "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           os.path.join(CSRC, "pycall.cpp"), "-o", tmp,
           *["-I" + i for i in inc],
           "-L" + os.path.join(os.path.dirname(torch.__file__), "lib"),
           "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10",
           "-lc10_cuda"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for pycall.cpp:\n{r.stderr}")
    os.replace(tmp, path)
    return path


def build(force: bool = False, verbose: bool = False,
          ptxas_info: bool = False, checks: bool = False) -> str:
    """Compile and link; returns the library path.  Raises on failure.
    checks=True builds the debug variant (see the module docstring)."""
    lib_path = CHECKS_LIB_PATH if checks else LIB_PATH
    if not force and up_to_date(lib_path):
        if has_torch():
            build_pycall()
        return lib_path
    nvcc = nvcc_path()
    obj_dir = os.path.join(BUILD_DIR, "checks") if checks else BUILD_DIR
    os.makedirs(obj_dir, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_info else []
    if checks:
        extra.append("-DTPMLP_CHECKS")

    def compile_one(src):
        obj = os.path.join(obj_dir, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc, *ARCH, *CFLAGS, *extra, "-c", os.path.join(CSRC, src),
               "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stderr}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        pycall = ex.submit(build_pycall, force) if has_torch() else None
        results = list(ex.map(compile_one, SOURCES))
    if verbose or ptxas_info:
        for obj, log in results:
            if log.strip():
                print(f"--- {os.path.basename(obj)}\n{log}", file=sys.stderr)
    tmp = lib_path + ".tmp"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, lib_path)
    if pycall is not None:
        pycall.result()   # (its error, where there is one)
    return lib_path


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True,
                ptxas_info="--ptxas-info" in sys.argv,
                checks="--checks" in sys.argv))
