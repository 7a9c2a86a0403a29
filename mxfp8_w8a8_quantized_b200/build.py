"""Build libmxfp8.so in-tree with nvcc for sm_100a, and the Python binding of
its per-token operators, _native.so, with the host compiler.

    python -m mxfp8_w8a8_quantized_b200.build [--force] [--verbose]

Cross-compiles without a GPU.  The library links the CUDA runtime
statically and needs only the driver at run time; the binding links the
library (found beside it) and PyTorch, and is left out where PyTorch is not
installed (a program that calls the C-ABI needs neither).
"""
import hashlib
import importlib.metadata
import importlib.util
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libmxfp8.so")
NATIVE = os.path.join(PKG, "_native.so")
NATIVE_SOURCE = os.path.join(CSRC, "torch_binding.cpp")

PUBLIC_HEADERS = ["mxfp8.h", "fp8_rowwise.h", "nvfp4.h", "mxfp4.h"]
SOURCES = ["mxfp8_quant.cu", "mxfp8_gemm.cu", "mxfp8_capi.cu", "mxfp8_noalloc.cu", "fp8_rowwise.cu", "nvfp4.cu",
           "mxfp4_quant.cu", "mxfp4_skinny.cu", "norm_quant.cu", "gated_quant.cu", "fused_capi.cu"]
HEADERS = ["ptx.cuh", "mx_element.cuh", "fp4_element.cuh", "rw_element.cuh", "quant_out.cuh", "fused_quant.cuh",
           "tmap_host.cuh", "capi_util.cuh", "async_copy.cuh"]
# The files each profiled kernel is compiled from: a profile summary names
# the hash of its kernel's files, so that it goes stale only when they change.
KERNEL_FILES = {
    "mxfp8_gemm": ["mxfp8_gemm.cu", "ptx.cuh", "mx_element.cuh", "tmap_host.cuh"],
}

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if c and (os.path.sep not in c or os.path.exists(c)):
            return c
    return "nvcc"


def _inputs():
    return ([os.path.join(CSRC, s) for s in SOURCES + HEADERS]
            + [os.path.join(INCLUDE, h) for h in PUBLIC_HEADERS] + [os.path.abspath(__file__)])


def source_sha(kernel: str = None) -> str:
    """Hash of the library's sources, or of one kernel's files
    (KERNEL_FILES); ties a profile summary to one build."""
    if kernel is None:
        paths = ([os.path.join(CSRC, s) for s in SOURCES + HEADERS]
                 + [os.path.join(INCLUDE, h) for h in PUBLIC_HEADERS])
    else:
        paths = [os.path.join(CSRC, s) for s in KERNEL_FILES[kernel]]
    h = hashlib.sha256()
    for p in paths:
        with open(p, "rb") as f:
            h.update(f.read())
    return h.hexdigest()[:16]


def _newer(out, inputs) -> bool:
    if not os.path.exists(out):
        return False
    t = os.path.getmtime(out)
    return all(os.path.getmtime(p) <= t for p in inputs)


def _native_inputs():
    return [NATIVE_SOURCE, os.path.abspath(__file__)] + [os.path.join(INCLUDE, h) for h in PUBLIC_HEADERS]


def native_tag() -> str:
    """The Python and PyTorch that a binding built now is for.  The binding holds
    this text: built for others, it may not even fail to load."""
    try:
        torch_version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:     # a PyTorch without package data
        import torch
        torch_version = torch.__version__
    return f"mxfp8 binding for {sysconfig.get_config_var('EXT_SUFFIX').strip('.')}, torch {torch_version};"


def native_problem():
    """Why the binding cannot be loaded here (None if it can)."""
    if not os.path.exists(NATIVE):
        return f"{NATIVE} is not built"
    with open(NATIVE, "rb") as f:
        if native_tag().encode() not in f.read():
            return f"{NATIVE} was built for another Python or PyTorch than this one"
    return None


def _native_current() -> bool:
    return _newer(NATIVE, _native_inputs()) and native_problem() is None


def _has_torch() -> bool:
    return importlib.util.find_spec("torch") is not None


def up_to_date() -> bool:
    return _newer(LIB, _inputs()) and (not _has_torch() or _native_current())


def build(force: bool = False, verbose: bool = False) -> str:
    if force or not _newer(LIB, _inputs()):
        cmd = [nvcc(), "-O3", "-std=c++17", *ARCH, "-lineinfo", "-shared", "-Xcompiler", "-fPIC", "--threads", "0",
               "-I", INCLUDE, "-I", CSRC, "-o", LIB + ".tmp"]
        if verbose:
            cmd += ["-Xptxas", "-v"]
        cmd += [os.path.join(CSRC, s) for s in SOURCES]
        subprocess.run(cmd, check=True)
        os.replace(LIB + ".tmp", LIB)
    if _has_torch() and (force or not _native_current()):
        _build_native()
    return LIB


def _build_native() -> None:
    """The binding against the installed PyTorch (its headers need the CUDA
    runtime's, which sit beside nvcc)."""
    import torch
    t = os.path.dirname(torch.__file__)
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    includes = [INCLUDE, os.path.join(t, "include"), os.path.join(t, "include", "torch", "csrc", "api", "include"), cuda,
                sysconfig.get_paths()["include"]]
    lib = os.path.join(t, "lib")
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-shared",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", f'-DMXFP8_BUILT_FOR="{native_tag()}"',
           NATIVE_SOURCE, "-o", NATIVE + ".tmp"]
    cmd += [f"-I{p}" for p in includes]
    cmd += [f"-L{lib}", f"-L{PKG}", "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10",
            "-l:libmxfp8.so", "-Wl,-rpath,$ORIGIN"]
    subprocess.run(cmd, check=True)
    os.replace(NATIVE + ".tmp", NATIVE)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
