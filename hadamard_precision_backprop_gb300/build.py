"""Build libhlq.so (the CUDA kernels + C ABI) in-tree for sm_103a with nvcc,
and the binding's extension module (host code against torch's headers).

Run ``python -m hadamard_precision_backprop_gb300.build`` or call
``build()``.  Translation units compile in parallel; the shared libraries are
written to ``hadamard_precision_backprop_gb300/_build/``.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(OUT_DIR, "libhlq.so")

SOURCES = ["hlq_api.cu", "hlq_quant.cu", "hlq_gemm_simple.cu", "hlq_gemm_tc.cu",
           "hlq_step_api.cu", "hlq_norm.cu", "hlq_norm_ring_bf16.cu",
           "hlq_norm_ring_f32.cu", "hlq_norm_elem.cu", "hlq_loss.cu", "hlq_clip.cu",
           "hlq_noalloc.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: libhlq cannot be built")
    return cand


def _flags():
    return ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                   "-Xcompiler", "-Wall", "-I", INCLUDE, "-I", CSRC,
                   "--expt-relaxed-constexpr"]


def ext_path() -> str:
    """The binding's extension for this interpreter and this torch: it reads
    torch's C++ objects, so each torch has a module of its own."""
    import sysconfig
    import torch
    return os.path.join(OUT_DIR, f"_hlq_torch-{torch.__version__}"
                                 f"{sysconfig.get_config_var('EXT_SUFFIX') or '.so'}")


def can_bind() -> bool:
    """Whether there is a torch to bind to: one with CUDA.  The library alone is
    built where there is none."""
    try:
        import torch
    except ImportError:
        return False
    return torch.version.cuda is not None


def is_current(with_ext: bool) -> bool:
    """Whether the built files are there and no older than their sources."""
    return all(os.path.exists(f) and os.path.getmtime(f) >= _deps_mtime()
               for f in ([LIB, ext_path()] if with_ext else [LIB]))


def _build_ext(link_after) -> None:
    """Compile the extension module; it is linked against libhlq.so (found
    beside it) once `link_after` has returned."""
    import sysconfig
    import torch
    top = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    cxx = shutil.which("g++") or "g++"
    ext = ext_path()
    obj, tmp = os.path.join(OUT_DIR, "hlq_torch.o"), ext + f".tmp{os.getpid()}"
    inc = [os.path.join(top, "include"), sysconfig.get_paths()["include"],
           os.path.join(cuda, "include"), INCLUDE]
    _run([cxx, "-O2", "-std=c++17", "-fPIC", "-Wall",
          f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
          *[a for d in inc for a in ("-isystem", d)],
          "-c", os.path.join(CSRC, "hlq_torch.cpp"), "-o", obj], "g++")
    link_after()
    libs = os.path.join(top, "lib")
    _run([cxx, "-shared", "-o", tmp, obj, "-L", OUT_DIR, "-lhlq", "-Wl,-rpath,$ORIGIN",
          "-L", libs, f"-Wl,-rpath,{libs}", "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu",
          "-ltorch", "-lc10_cuda", "-lc10"], "link of the extension")
    os.replace(tmp, ext)


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _deps_mtime() -> float:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "hlq.h"))
    return max(os.path.getmtime(f) for f in files)


def build(force: bool = False, verbose: bool = False) -> str:
    with_ext = can_bind()
    if not force and is_current(with_ext):
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    nvcc = _nvcc()

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc] + _flags() + ["-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        _run(cmd, f"nvcc on {src}")
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        objs = [ex.submit(compile_one, src) for src in SOURCES]
        linked = cf.Future()
        ext = ex.submit(_build_ext, linked.result) if with_ext else None
        try:
            tmp = LIB + f".tmp{os.getpid()}"
            _run([nvcc] + ARCH + ["-shared", "-o", tmp] + [o.result() for o in objs], "link")
            os.replace(tmp, LIB)
        except BaseException as e:
            linked.set_exception(e)
            raise
        linked.set_result(None)
        if ext is not None:
            ext.result()
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True))
