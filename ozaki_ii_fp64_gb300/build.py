"""Builds libozemu.so in-tree with nvcc for sm_103a (GB300).

Each CUDA translation unit compiles in parallel to an object under
``_build/<machine>/``; the objects link into ``ozaki_ii_fp64_gb300/_lib/libozemu.so``.
Where PyTorch is installed, the binding of the layer operators to its tensors
(``_lib/_ozemu_torch.so``, host code that calls libozemu.so) is built with it.
A stamp next to the library records the host machine, the PyTorch version and
the source hashes, so a library built on another architecture or from older
sources is rebuilt.
"""

import hashlib
import importlib.metadata
import importlib.util
import os
import platform
import shutil
import subprocess
import sysconfig
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIBDIR = os.path.join(PKG, "_lib")
LIBNAME = "libozemu.so"
SOURCES = ["api.cu", "split.cu", "gemm_fp4.cu", "crt.cu", "igemm_mma.cu", "gemv.cu", "linear.cu",
           "layernorm.cu", "mx.cu", "clip.cu"]
ARCH_FLAGS = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def lib_path():
    return os.path.join(LIBDIR, LIBNAME)


def binding_path():
    return os.path.join(LIBDIR, "_ozemu_torch.so")


def _torch_version():
    try:
        return importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        return None


def _fingerprint():
    h = hashlib.sha256()
    h.update(platform.machine().encode())
    h.update(("%s %s" % (_torch_version(), sysconfig.get_python_version())).encode())
    for d in (CSRC, INCLUDE):
        for name in sorted(os.listdir(d)):
            if name.endswith((".cu", ".cuh", ".h", ".cpp")):
                with open(os.path.join(d, name), "rb") as f:
                    h.update(name.encode())
                    h.update(f.read())
    h.update(" ".join(ARCH_FLAGS).encode())
    return h.hexdigest()


def _stamp_path():
    return lib_path() + ".stamp"


def is_current():
    if not os.path.exists(lib_path()) or not os.path.exists(_stamp_path()):
        return False
    if _torch_version() and not os.path.exists(binding_path()):
        return False
    with open(_stamp_path()) as f:
        return f.read().strip() == _fingerprint()


def build(force=False, verbose=False, ptxas_info=False):
    """Compile and link libozemu.so; returns its path."""
    if not force and is_current():
        return lib_path()
    obj_dir = os.path.join(ROOT, "_build", platform.machine())
    os.makedirs(obj_dir, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    cc = nvcc()
    common = ARCH_FLAGS + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE,
                           "--expt-relaxed-constexpr"]
    if ptxas_info:
        common += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(obj_dir, src.replace(".cu", ".o"))
        cmd = [cc] + common + ["-c", os.path.join(CSRC, src), "-o", obj]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError("nvcc failed for %s:\n%s\n%s" % (src, res.stdout, res.stderr))
        if verbose or ptxas_info:
            print(res.stdout + res.stderr)
        return obj

    # The tensor binding's include and library folders, without importing torch.
    torch_dir = None
    if _torch_version():
        torch_dir = os.path.dirname(importlib.util.find_spec("torch").origin)

    def compile_binding():
        obj = os.path.join(obj_dir, "binding.o")
        inc = [os.path.join(torch_dir, "include"), os.path.join(torch_dir, "include", "torch", "csrc", "api", "include"),
               os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(cc))), "include"),
               sysconfig.get_paths()["include"], INCLUDE]
        cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-fPIC", "-c", os.path.join(CSRC, "binding.cpp"),
               "-o", obj] + ["-I" + i for i in inc]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError("g++ failed for binding.cpp:\n%s\n%s" % (res.stdout, res.stderr))
        return obj

    with ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        binding = ex.submit(compile_binding) if torch_dir else None
        objs = list(ex.map(compile_one, SOURCES))
        binding = binding.result() if binding else None
    tmp = lib_path() + ".tmp"
    cmd = [cc] + ARCH_FLAGS + ["-shared", "-o", tmp] + objs + ["-lcuda"] * 0
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (res.stdout, res.stderr))
    os.replace(tmp, lib_path())
    if binding:
        libs = os.path.join(torch_dir, "lib")
        cmd = [os.environ.get("CXX", "g++"), "-shared", "-o", binding_path() + ".tmp", binding, "-L" + LIBDIR, "-lozemu",
               "-L" + libs, "-ltorch_python", "-ltorch_cpu", "-ltorch", "-lc10_cuda", "-lc10", "-Wl,-rpath,$ORIGIN",
               "-Wl,-rpath," + libs]
        res = subprocess.run(cmd, capture_output=True, text=True)
        if res.returncode != 0:
            raise RuntimeError("link failed:\n%s\n%s" % (res.stdout, res.stderr))
        os.replace(binding_path() + ".tmp", binding_path())
    with open(_stamp_path(), "w") as f:
        f.write(_fingerprint())
    return lib_path()


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv))
