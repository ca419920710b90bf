"""Build libpkv.so in-tree for sm_103a with nvcc.

Each translation unit of csrc/ compiles in parallel to an object file under
_build/<machine>/, then nvcc links the shared library next to this file. The
_native module beside it (csrc/native.cpp, argument marshalling against torch's
headers) compiles with the host compiler. Each is rebuilt only when a source or
header is newer, _native also when torch or Python changed.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import platform
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
LIB = os.path.join(HERE, "libpkv.so")
NATIVE_SRC = os.path.join(CSRC, "native.cpp")
NATIVE = os.path.join(HERE, "_native.so")
OBJ_DIR = os.path.join(HERE, "_build", platform.machine())
NATIVE_STAMP = os.path.join(OBJ_DIR, "native.built_for")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + [
    "-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
    "-ftz=false", "-prec-div=true", "-prec-sqrt=true", "-fmad=true",
    "-Xcompiler", "-fPIC,-fvisibility=hidden",
]


def nvcc() -> str:
    for c in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if c and os.path.exists(c):
            return c
    raise RuntimeError("nvcc not found: libpkv needs the CUDA toolkit to build")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def native_target() -> str:
    """What a _native module has to be built for: this torch, Python and machine."""
    import torch
    return f"torch {torch.__version__}, Python {'.'.join(map(str, sys.version_info[:2]))}, " \
           f"{platform.machine()}"


def _newer(path, deps) -> bool:
    return os.path.exists(path) and all(os.path.getmtime(d) <= os.path.getmtime(path) for d in deps)


def lib_up_to_date() -> bool:
    return _newer(LIB, sources() + glob.glob(os.path.join(CSRC, "*.cuh"))
                  + glob.glob(os.path.join(CSRC, "*.h"))
                  + [os.path.join(ROOT, "include", "pkv.h"), os.path.abspath(__file__)])


def native_up_to_date() -> bool:
    if not _newer(NATIVE, [NATIVE_SRC, os.path.join(ROOT, "include", "pkv.h"),
                           os.path.abspath(__file__)]):
        return False
    try:
        with open(NATIVE_STAMP) as f:
            return f.read() == native_target()
    except OSError:
        return False


def up_to_date() -> bool:
    return lib_up_to_date() and native_up_to_date()


def _build_native() -> None:
    """Compile and link the _native module against the installed torch."""
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(nvcc())))
    include = [os.path.join(root, "include"),
               os.path.join(root, "include", "torch", "csrc", "api", "include"),
               os.path.join(cuda, "include"), sysconfig.get_paths()["include"]]
    lib = os.path.join(root, "lib")
    tmp = NATIVE + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-std=c++17", "-O2", "-fPIC", "-shared",
           "-fvisibility=hidden", f'-DPKV_BUILT_FOR="{native_target()}"', f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
           *[f"-I{d}" for d in include], NATIVE_SRC, "-o", tmp, f"-L{lib}", f"-Wl,-rpath,{lib}",
           "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on {NATIVE_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, NATIVE)
    with open(NATIVE_STAMP, "w") as f:
        f.write(native_target())


def build(force: bool = False, verbose: bool = False, ptxas_v: bool = False) -> str:
    """Compile and link libpkv (only when a source is newer than the library,
    unless force); ptxas_v prints the registers and spills of every kernel. The
    library is there even if _native, built beside it, fails to compile."""
    os.makedirs(OBJ_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=max(1, min(16, os.cpu_count() or 1))) as ex:
        native = ex.submit(_build_native) if force or not native_up_to_date() else None
        if force or not lib_up_to_date():
            _build_lib(ex, verbose, ptxas_v)
        if native is not None:
            native.result()
    return LIB


def _build_lib(ex: cf.Executor, verbose: bool, ptxas_v: bool) -> None:
    cc = nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_v else []

    def compile_one(src):
        obj = os.path.join(OBJ_DIR, os.path.basename(src) + ".o")
        cmd = [cc, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        if verbose or ptxas_v:
            print(r.stdout + r.stderr)
        return obj

    objs = list(ex.map(compile_one, sources()))
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, *ARCH, "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose=True, ptxas_v="--ptxas-v" in sys.argv))
