"""Build step of libred.so: nvcc for sm_103a, one object per .cu (compiled in
parallel), linked into ``int_tensor_reductions_gb300/libred.so`` in-tree, and
of the losses' Python entry, ``_red_torch`` (g++ against torch and libred.so)."""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import subprocess

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJDIR = os.path.join(ROOT, "_build", "red")
LIB = os.path.join(PKG, "libred.so")
EXT = os.path.join(PKG, "_red_torch.so")
EXT_SRC = os.path.join(CSRC, "red_torch.cpp")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-O2",
                     "-I" + INCLUDE, "-I" + CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", "nvcc"):
        if cand and (os.path.isabs(cand) and os.path.exists(cand) or not os.path.isabs(cand)):
            return cand
    return "nvcc"


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.h")) + glob.glob(os.path.join(CSRC, "*.cuh")) + \
        glob.glob(os.path.join(INCLUDE, "*.h")) + glob.glob(os.path.join(INCLUDE, "*.cuh")) + \
        [EXT_SRC, os.path.abspath(__file__)]


def is_stale() -> bool:
    if not os.path.exists(LIB) or not os.path.exists(EXT):
        return True
    t = min(os.path.getmtime(LIB), os.path.getmtime(EXT))
    return any(os.path.getmtime(d) > t for d in _deps())


def _run(cmd, what):
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("%s failed:\n%s\n%s" % (what, " ".join(cmd), r.stdout + r.stderr))
    return r


def _compile_ext() -> str:
    """The object of the Python entry."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension
    obj = os.path.join(OBJDIR, "red_torch.o")
    cuda = os.path.dirname(os.path.dirname(nvcc())) if os.path.isabs(nvcc()) else "/usr/local/cuda"
    dirs = cpp_extension.include_paths() + [sysconfig.get_paths()["include"], os.path.join(cuda, "include"), INCLUDE]
    _run(["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
          "-D_GLIBCXX_USE_CXX11_ABI=%d" % int(torch._C._GLIBCXX_USE_CXX11_ABI)] + ["-I" + d for d in dirs] +
         ["-c", EXT_SRC, "-o", obj], "g++ on red_torch.cpp")
    return obj


def _link_ext(obj: str) -> None:
    import torch
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = EXT + ".tmp%d" % os.getpid()
    _run(["g++", "-shared", obj, "-o", tmp, "-L" + PKG, "-l:libred.so", "-Wl,-rpath,$ORIGIN", "-L" + libs,
          "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"], "link of _red_torch")
    os.replace(tmp, EXT)


def build_lib(force: bool = False, verbose: bool = False, extra_flags=()) -> str:
    """Compile csrc/*.cu for sm_103a and link libred.so; return its path."""
    if not force and not is_stale():
        return LIB
    os.makedirs(OBJDIR, exist_ok=True)
    cc = nvcc()
    flags = NVCC_FLAGS + list(extra_flags)

    def compile_one(src):
        obj = os.path.join(OBJDIR, os.path.basename(src)[:-3] + ".o")
        cmd = [cc] + flags + ["-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed on %s:\n%s\n%s" % (src, " ".join(cmd), r.stdout + r.stderr))
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr)
        return obj

    srcs = _sources()
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(srcs) + 1, os.cpu_count() or 1))) as ex:
        ext = ex.submit(_compile_ext)
        objs = list(ex.map(compile_one, srcs))
        ext = ext.result()
    tmp = LIB + ".tmp%d" % os.getpid()
    cmd = [cc] + ARCH + ["-shared", "-o", tmp] + objs
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s\n%s" % (" ".join(cmd), r.stdout + r.stderr))
    os.replace(tmp, LIB)
    _link_ext(ext)
    return LIB


if __name__ == "__main__":
    print(build_lib(force=True, verbose=True))
