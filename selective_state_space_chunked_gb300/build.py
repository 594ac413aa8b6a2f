"""Builds the CUDA library ``_build/liblrscan.so`` in-tree with nvcc.

Every translation unit under ``csrc/`` is compiled for sm_103a only
(``-gencode arch=compute_103a,code=sm_103a``), in parallel, then linked into
one shared library against the shared CUDA runtime.  ``csrc/lr_torch.cpp``, the
short path of the torch helpers, becomes the extension module ``_build/_lrtorch``
beside it, against the library and the installed torch, whose version is recorded.
The build is skipped when both are newer than every source and header and torch is
still that version.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import importlib.util
import os
import shutil
import subprocess
import sysconfig
import tempfile

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
BUILD_DIR = os.path.join(PKG, "_build")
LIB_NAME = "liblrscan.so"
LIB_PATH = os.path.join(BUILD_DIR, LIB_NAME)
TORCH_SRC = os.path.join(CSRC, "lr_torch.cpp")
TORCH_MODULE = os.path.join(BUILD_DIR, "_lrtorch" + sysconfig.get_config_var("EXT_SUFFIX"))
TORCH_VERSION = os.path.join(BUILD_DIR, "_lrtorch.torch")   # of the torch it was built against

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
              "--expt-relaxed-constexpr", "-I" + INCLUDE, "-I" + CSRC]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"),
                 "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build lrscan")


def _torch_dir() -> str:
    return list(importlib.util.find_spec("torch").submodule_search_locations)[0]


def torch_module_matches() -> bool:
    """Whether the extension module is there and was built against the installed
    torch (its C++ interface is that version's alone)."""
    import torch
    try:
        with open(TORCH_VERSION) as f:
            return f.read() == torch.__version__ and os.path.exists(TORCH_MODULE)
    except OSError:
        return False


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return (_sources() + glob.glob(os.path.join(CSRC, "*.cuh"))
            + glob.glob(os.path.join(CSRC, "*.h"))
            + glob.glob(os.path.join(INCLUDE, "*.h")) + [TORCH_SRC, __file__])


def up_to_date() -> bool:
    if not os.path.exists(LIB_PATH) or not torch_module_matches():
        return False
    t = min(os.path.getmtime(LIB_PATH), os.path.getmtime(TORCH_MODULE))
    return all(os.path.getmtime(p) <= t for p in _deps())


def build(force: bool = False, verbose: bool = False) -> str:
    """Compiles the library if needed and returns its path."""
    if not force and up_to_date():
        return LIB_PATH
    os.makedirs(BUILD_DIR, exist_ok=True)
    nvcc = _nvcc()
    tmpdir = tempfile.mkdtemp(prefix="obj_", dir=BUILD_DIR)
    try:
        torch_dir = _torch_dir()
        cuda_dir = os.path.dirname(os.path.dirname(os.path.realpath(nvcc)))

        def compile_one(src):
            obj = os.path.join(tmpdir, os.path.basename(src) + ".o")
            if src == TORCH_SRC:
                cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-I" + INCLUDE,
                       "-I" + os.path.join(torch_dir, "include"), "-I" + os.path.join(cuda_dir, "include"),
                       "-I" + sysconfig.get_paths()["include"], "-c", src, "-o", obj]
            else:
                cmd = [nvcc, *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj]
            r = subprocess.run(cmd, capture_output=True, text=True)
            if r.returncode != 0:
                raise RuntimeError(f"{cmd[0]} failed on {src}:\n{r.stdout}\n{r.stderr}")
            if verbose and r.stderr:
                print(r.stderr)
            return obj

        def link(cmd, path):
            fd, tmp_lib = tempfile.mkstemp(suffix=".so", dir=BUILD_DIR)
            os.close(fd)
            r = subprocess.run([*cmd, "-o", tmp_lib], capture_output=True, text=True)
            if r.returncode != 0:
                os.unlink(tmp_lib)
                raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
            os.replace(tmp_lib, path)

        with cf.ThreadPoolExecutor(max_workers=max(1, min(8, os.cpu_count() or 1))) as ex:
            torch_obj = ex.submit(compile_one, TORCH_SRC)
            objs = list(ex.map(compile_one, _sources()))
        link([nvcc, *ARCH, "-shared", "-cudart", "shared", *objs, "-Xlinker", "-rpath,/usr/local/cuda/lib64"],
             LIB_PATH)
        # the library stands without the module, and no longer goes with an older one
        if os.path.exists(TORCH_VERSION):
            os.unlink(TORCH_VERSION)
        link(["g++", "-shared", torch_obj.result(), "-Wl,-rpath,$ORIGIN", "-L" + BUILD_DIR, "-l:" + LIB_NAME,
              "-L" + os.path.join(torch_dir, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
              f"-L{cuda_dir}/lib64", "-lcudart"], TORCH_MODULE)
        import torch
        with open(TORCH_VERSION, "w") as f:
            f.write(torch.__version__)
    finally:
        shutil.rmtree(tmpdir, ignore_errors=True)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force=True, verbose=True))
