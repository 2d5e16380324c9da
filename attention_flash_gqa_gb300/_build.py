"""Compile the CUDA sources of this package into ``libattn_gb300.so`` (in-tree), and the native part of
the Python binding into ``_ops.so``.

The library: nvcc only, one ``-gencode`` for sm_103a, translation units compiled in parallel and
linked with ``nvcc -shared``. The binding: one C++ file against torch's headers, by g++ beside them; it
belongs to the torch it was built with. The library does not need it: it is linked where the binding
cannot be built, and where torch is not installed there is no binding to build.
Used by ``__graft_entry__.build()`` and the tests.
"""
from __future__ import annotations

import concurrent.futures as cf
import importlib.util
import os
import shutil
import subprocess

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libattn_gb300.so")
OPS = os.path.join(HERE, "_ops.so")
OPS_SOURCE = os.path.join(CSRC, "py_ops.cpp")
BUILD_DIR = os.path.join(HERE, "_build_tmp")
OPS_TAG = os.path.join(BUILD_DIR, "ops_built_for.txt")  # what _ops.so was built for
SOURCES = ["api.cu", "attn_fwd.cu", "attn_bwd.cu", "attn_bwd_small.cu", "attn_bwd_sink.cu", "decode_paged.cu", "decode_paged_noalloc.cu",
           "decode_kv4.cu", "kv4_pages.cu", "merge_lse.cu", "paged_plan.cu", "qk_norm_rope.cu", "tree_paged.cu"]
GENCODE = "-gencode=arch=compute_103a,code=sm_103a"


def nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build the attention library")


def _inputs():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cu", ".cuh", ".h"))]
    files.append(os.path.join(os.path.dirname(HERE), "include", "attn.h"))
    return files


def torch_tag() -> str | None:
    """The torch and Python that a binding built now would belong to; None without torch."""
    if importlib.util.find_spec("torch") is None:
        return None
    import sysconfig

    import torch

    return f"torch {torch.__version__} {sysconfig.get_config_var('SOABI')} abi {int(torch._C._GLIBCXX_USE_CXX11_ABI)}"


def ops_tag() -> str | None:
    """What the present _ops.so was built for; None if that is not known."""
    try:
        with open(OPS_TAG) as f:
            return f.read()
    except OSError:
        return None


def _newer(target, sources) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(f) <= os.path.getmtime(target) for f in sources)


def lib_up_to_date() -> bool:
    return _newer(LIB, _inputs())


def ops_up_to_date() -> bool:
    """Newer than its sources and built for this torch (or there is no torch to build it for)."""
    tag = torch_tag()
    header = os.path.join(os.path.dirname(HERE), "include", "attn.h")
    return tag is None or (_newer(OPS, (OPS_SOURCE, header)) and ops_tag() == tag)


def up_to_date() -> bool:
    return lib_up_to_date() and ops_up_to_date()


def _build_ops() -> None:
    """Compile the native part of the Python binding against the torch of this machine."""
    import sysconfig

    import torch

    base = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(nvcc()))
    tmp = OPS + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-shared", OPS_SOURCE, "-o", tmp,
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I", sysconfig.get_paths()["include"],
           "-I", os.path.join(base, "include"), "-I", os.path.join(base, "include", "torch", "csrc", "api", "include"),
           "-I", os.path.join(cuda, "include"), "-L", os.path.join(base, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10",
           "-lc10_cuda"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        raise RuntimeError(f"py_ops.cpp needs g++: {e}") from e
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for py_ops.cpp:\n{r.stdout}\n{r.stderr}")
    if os.path.exists(OPS_TAG):
        os.remove(OPS_TAG)
    os.replace(tmp, OPS)
    with open(OPS_TAG, "w") as f:
        f.write(torch_tag())


def build(force: bool = False, verbose: bool = False) -> str:
    """Builds what is missing or stale. Raises where the binding cannot be built, with the library linked all the same."""
    do_lib, do_ops = force or not lib_up_to_date(), torch_tag() is not None and (force or not ops_up_to_date())
    os.makedirs(BUILD_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        ops = ex.submit(_build_ops) if do_ops else None
        if do_lib:
            _build_lib(verbose)
        if ops is not None:
            try:
                ops.result()
            except Exception as e:
                raise RuntimeError(f"{LIB} is built, but the native part of the Python binding is not: the calls that go "
                                   f"through it are missing\n{e}") from e
    return LIB


def _build_lib(verbose: bool) -> None:
    cc = nvcc()
    flags = [GENCODE, "-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
             "--expt-relaxed-constexpr", "-I", os.path.join(os.path.dirname(HERE), "include")]
    if verbose:
        flags += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, src.replace(".cu", ".o"))
        cmd = [cc, *flags, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    if verbose:
        for _, err in results:
            print(err)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, GENCODE, "-shared", "-o", tmp, *[o for o, _ in results], "-lcudart"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    import sys

    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
