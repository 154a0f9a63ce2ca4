"""Build the CUDA library libcpw_moe.so in-tree (nvcc, sm_103a only) and the Python module _ops.so.

The translation units are compiled in parallel and linked into one shared library
that exports the C ABI of include/cpw_moe.h.  The CUDA runtime is linked statically;
the driver's tensor-map encoder is fetched at run time, so no libcuda link is needed.
_ops.so (g++, PyTorch's headers) marshals the operators' arguments over that ABI; the layer itself
does without it.
"""
import concurrent.futures as cf
import glob
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libcpw_moe.so")
OPS = os.path.join(PKG, "_ops.so")
SOURCES = ["api.cu", "routing.cu", "ffn.cu", "ffn_bs.cu", "noalloc.cu", "norm.cu", "router.cu",
           "rows.cu", "grouped_mm.cu", "rms_norm.cu", "scores.cu", "swiglu.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
                "-I" + os.path.join(ROOT, "include")]


def _nvcc():
    cand = os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "bin", "nvcc")
    return cand if os.path.exists(cand) else "nvcc"


HEADER = os.path.join(ROOT, "include", "cpw_moe.h")


def _newer_than(target, deps) -> bool:
    return os.path.exists(target) and all(os.path.getmtime(p) <= os.path.getmtime(target) for p in deps)


def library_up_to_date() -> bool:
    sources = [p for kind in ("*.cu", "*.cuh", "*.h") for p in glob.glob(os.path.join(CSRC, kind))]
    return _newer_than(LIB, sources + [HEADER, __file__])


def _built_against() -> str:
    """What _ops.so depends on besides its sources: the interpreter and PyTorch's binary interface."""
    import sysconfig

    import torch

    return f"torch {torch.__version__} cxx11 {int(torch._C._GLIBCXX_USE_CXX11_ABI)} {sysconfig.get_config_var('EXT_SUFFIX')}"


def binding_up_to_date() -> bool:
    if not _newer_than(OPS, [os.path.join(CSRC, "bind.cpp"), HEADER, __file__]):
        return False
    try:
        with open(OPS + ".for", encoding="utf-8") as f:
            return f.read() == _built_against()
    except OSError:
        return False


def up_to_date() -> bool:
    return library_up_to_date() and binding_up_to_date()


def _compile_binding() -> str:
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    cuda = os.path.dirname(os.path.dirname(_nvcc())) if os.path.isabs(_nvcc()) else "/usr/local/cuda"
    inc = [f"-I{p}" for p in cpp_extension.include_paths()]
    inc += ["-I" + sysconfig.get_paths()["include"], "-I" + os.path.join(cuda, "include")]
    obj = os.path.join(BUILD, "bind.o")
    abi = f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", abi, *inc, "-c", os.path.join(CSRC, "bind.cpp"), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on bind.cpp:\n{r.stdout}\n{r.stderr}")
    return obj


def _link_binding(obj: str) -> None:
    from torch.utils import cpp_extension

    tmp = OPS + f".tmp{os.getpid()}"
    libs = [f"-L{p}" for p in cpp_extension.library_paths()]
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L" + PKG, "-l:libcpw_moe.so", *libs, "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda",
           "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, OPS)
    with open(tmp, "w", encoding="utf-8") as f:
        f.write(_built_against())
    os.replace(tmp, OPS + ".for")


def build_library(force: bool = False, verbose_ptxas: bool = False) -> str:
    """libcpw_moe.so: needs nvcc and its host compiler alone."""
    if not force and library_up_to_date():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.splitext(src)[0] + ".o")
        cmd = [nvcc, *FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    if verbose_ptxas:
        for _, log in results:
            sys.stderr.write(log)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


def build_binding(force: bool = False) -> str:
    """_ops.so, over a built library: needs g++ and the headers of Python and PyTorch too."""
    if force or not binding_up_to_date():
        os.makedirs(BUILD, exist_ok=True)
        _link_binding(_compile_binding())
    return OPS


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Both, side by side; the library is there even where the module cannot be built."""
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(1) as ex:
        binding = ex.submit(_compile_binding) if force or not binding_up_to_date() else None
        build_library(force, verbose_ptxas)
        if binding:
            _link_binding(binding.result())
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv))
