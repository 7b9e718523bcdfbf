"""Build libmoe_lora.so (the CUDA library) in-tree with nvcc for sm_103a.

Translation units are compiled in parallel, then linked into
lora_moe_gb300/_build/libmoe_lora.so.  Beside it, where Python's headers and
torch are installed, fastcall.*.so: the serving operators' calls from Python
without ctypes (a C++ extension, named by the Python and the torch that it was
built against).  Where it does not build, a warning says so and the calls go
through ctypes.
Usage: python -m lora_moe_gb300.build
"""
import concurrent.futures
import fcntl
import importlib.metadata
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(OUT_DIR, "libmoe_lora.so")
SOURCES = ["api.cu", "align.cu", "fused_cuda_core.cu", "fused_tcgen05.cu", "stream_pipeline.cu",
           "fused_stream_cluster.cu", "align_static_workspace.cu", "api_fp8.cu", "fp8_rows.cu", "fp8_matmul.cu", "fp8_stream.cu",
           "gather.cu", "api_bf16.cu", "bf16_matmul.cu", "bf16_stream.cu",
           "api_route.cu", "route.cu"]


def _torch_version():
    """torch's version without importing it, or None where it is not installed."""
    try:
        return importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        return None


FASTCALL = os.path.join(OUT_DIR, "fastcall.%s.torch-%s.so" % (sysconfig.get_config_var("SOABI"), _torch_version()))
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def _nvcc():
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found")
    return cand


def _cuda_lib_dir(nvcc):
    return os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "lib64")


def _inputs_mtime():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "moe_lora.h"), __file__]
    return max(os.path.getmtime(f) for f in files)


def _has_python_headers():
    return os.path.exists(os.path.join(sysconfig.get_paths()["include"], "Python.h"))


def _build_fastcall():
    import torch
    root = os.path.dirname(os.path.abspath(torch.__file__))
    include, lib = os.path.join(root, "include"), os.path.join(root, "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    tmp = FASTCALL + ".tmp.%d" % os.getpid()
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
           "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI), "-I", INCLUDE,
           "-isystem", sysconfig.get_paths()["include"], "-isystem", include,
           "-isystem", os.path.join(include, "torch", "csrc", "api", "include"), "-isystem", cuda,
           os.path.join(CSRC, "fastcall.cpp"), "-o", tmp, "-L" + lib, "-lc10", "-lc10_cuda", "-ltorch_cpu",
           "-ltorch_python", "-Wl,-rpath," + lib]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("g++ failed for fastcall.cpp:\n%s\n%s" % (res.stdout, res.stderr))
    os.replace(tmp, FASTCALL)


def _try_fastcall():
    """Build fastcall, or note why it does not build: not tried again until its inputs change."""
    try:
        _build_fastcall()
    except Exception as e:
        with open(FASTCALL + ".failed", "w") as f:
            f.write(str(e))
        warnings.warn("the serving operators' calls go through ctypes: %s" % e)


def _fastcall_settled():
    """Built for this Python and torch from the present sources, known not to build, or not to be built here."""
    if not _has_python_headers() or _torch_version() is None:
        return True
    inputs = max(os.path.getmtime(f) for f in (os.path.join(CSRC, "fastcall.cpp"),
                                               os.path.join(INCLUDE, "moe_lora.h"), __file__))
    return any(os.path.exists(f) and os.path.getmtime(f) >= inputs for f in (FASTCALL, FASTCALL + ".failed"))


def build(force=False, verbose=False, ptxas_info=False):
    always = force or ptxas_info
    if not always and _is_current() and _fastcall_settled():
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    # One process at a time: the object files are shared. One that waited finds the other's result.
    with open(os.path.join(OUT_DIR, "lock"), "w") as lock:
        fcntl.flock(lock, fcntl.LOCK_EX)
        if always or not _is_current():
            _build(verbose, ptxas_info)
        if not _fastcall_settled():     # (the library was current)
            _try_fastcall()
    return LIB


def _is_current():
    return os.path.exists(LIB) and os.path.getmtime(LIB) >= _inputs_mtime()


def _build(verbose, ptxas_info):
    nvcc = _nvcc()
    common = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE,
                     "-Xcompiler", "-Wall", "--expt-relaxed-constexpr"]
    if ptxas_info:
        common += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc] + common + ["-c", os.path.join(CSRC, src), "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, res.stdout, res.stderr))
        if verbose or ptxas_info:
            sys.stderr.write(res.stdout + res.stderr)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        fast = ex.submit(_try_fastcall) if _has_python_headers() and _torch_version() is not None else None
        objs = list(ex.map(compile_one, SOURCES))
        if fast is not None:
            fast.result()
    tmp = LIB + ".tmp.%d" % os.getpid()
    cmd = [nvcc] + ARCH + ["-shared", "-cudart", "shared", "-o", tmp] + objs + [
        "-Xlinker", "-rpath," + _cuda_lib_dir(nvcc)]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (res.stdout, res.stderr))
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force=True, verbose=True, ptxas_info="--ptxas" in sys.argv))
