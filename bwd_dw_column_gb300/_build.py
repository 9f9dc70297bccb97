"""Build ``libcake_rmsnorm.so`` in-tree with nvcc for sm_103a.

Each ``.cu`` file of ``csrc``, ``csrc_step`` and ``csrc_block`` compiles in its own nvcc process (in parallel), then
nvcc links them into one shared library next to this file.  The CUDA runtime
is linked statically, so the library needs only the driver at run time.  Beside
them the host compiler builds ``_cake_block.so``, the Python entry points of the
operators between the norms, against torch's headers and this library.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
CSRC_STEP = os.path.join(HERE, "csrc_step")  # the training-step operators around the norm
CSRC_BLOCK = os.path.join(HERE, "csrc_block")  # a block's operators between the norms
INCLUDE = os.path.join(os.path.dirname(HERE), "include")
LIB = os.path.join(HERE, "libcake_rmsnorm.so")
PYTHON_SOURCE = os.path.join(CSRC_BLOCK, "cake_block_python.cpp")
PYTHON_MODULE = os.path.join(HERE, "_cake_block.so")
BUILD_DIR = os.path.join(os.path.dirname(HERE), "_build")
MODULE_STAMP = os.path.join(BUILD_DIR, "cake_block_python.built_for")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2", "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libcake_rmsnorm.so")
    return cand


def sources():
    return sorted(os.path.join(d, f) for d in (CSRC, CSRC_STEP, CSRC_BLOCK) for f in os.listdir(d) if f.endswith(".cu"))


def _inputs():
    files = sources()
    for d in (CSRC, CSRC_STEP, CSRC_BLOCK, INCLUDE):
        files += [os.path.join(d, f) for f in os.listdir(d) if f.endswith((".cuh", ".h"))]
    files += [PYTHON_SOURCE, os.path.abspath(__file__)]
    return files


def _built_for() -> str:
    """What _cake_block.so depends on beside its source: the interpreter, and the torch whose headers it is compiled
    against."""
    import torch
    return f"{sys.version}\n{torch.__version__}\n{torch.__file__}\ncxx11 abi {int(torch.compiled_with_cxx11_abi())}\n"


def _module_stamp() -> str:
    try:
        with open(MODULE_STAMP) as f:
            return f.read()
    except OSError:
        return ""


def up_to_date() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(PYTHON_MODULE) or _module_stamp() != _built_for():
        return False
    t = min(os.path.getmtime(LIB), os.path.getmtime(PYTHON_MODULE))
    return all(os.path.getmtime(f) <= t for f in _inputs())


def build(force: bool = False, verbose_ptxas: bool = False) -> str:
    """Compile (if stale) and return the library path."""
    if not force and up_to_date():
        return LIB
    nvcc = _nvcc()
    os.makedirs(BUILD_DIR, exist_ok=True)
    extra = ["-Xptxas", "-v"] if verbose_ptxas else []

    def compile_one(src):
        obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
        cmd = [nvcc, *ARCH, *NVCC_FLAGS, *extra, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {os.path.basename(src)}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 2)) as ex:
        module = ex.submit(_compile_module, nvcc)
        results = list(ex.map(compile_one, sources()))
        module = module.result()
    if verbose_ptxas:
        for _, log in results:
            sys.stderr.write(log)
    objs = [o for o, _ in results]
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([nvcc, *ARCH, "-shared", "-o", tmp, *objs], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _link_module(module)
    return LIB


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _torch_dir(*parts):
    import torch
    return os.path.join(os.path.dirname(torch.__file__), *parts)


def _compile_module(nvcc: str) -> str:
    """The Python entry points' object file."""
    import sysconfig

    import torch
    include = [_torch_dir("include"), _torch_dir("include", "torch", "csrc", "api", "include"),
               os.path.join(os.path.dirname(os.path.dirname(nvcc)), "include"), sysconfig.get_paths()["include"], INCLUDE]
    obj = os.path.join(BUILD_DIR, "cake_block_python.o")
    _run(["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}",
          *(f"-I{d}" for d in include), "-c", PYTHON_SOURCE, "-o", obj], "g++ on cake_block_python.cpp")
    return obj


def _link_module(obj: str) -> None:
    tmp = PYTHON_MODULE + f".tmp{os.getpid()}"
    _run(["g++", "-shared", "-o", tmp, obj, f"-L{_torch_dir('lib')}", "-ltorch_python", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda",
          f"-L{HERE}", "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN"], "linking _cake_block.so")
    os.replace(tmp, PYTHON_MODULE)
    with open(MODULE_STAMP, "w") as f:
        f.write(_built_for())


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose_ptxas="-v" in sys.argv)
    print(LIB)
