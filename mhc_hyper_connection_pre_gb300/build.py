"""Build libmhc.so (the seam's C-ABI library) in-tree with nvcc for sm_103a.

Each CUDA translation unit under ``csrc/`` is compiled in parallel to an
object file, then linked into ``_build/libmhc.so`` (CUDA runtime linked
statically, so loading the library needs no GPU).  ``csrc/kv_binding.cpp``, a
CPython extension over PyTorch's headers, becomes ``_build/_mhc_kv.so``, linked
to libmhc.so beside it.  Rebuilds only what changed.  Usage: ``python -m mhc_hyper_connection_pre_gb300.build [--ptxas-v]``.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(PKG, "_build")
LIB = os.path.join(BUILD, "libmhc.so")
BINDING = os.path.join(BUILD, "_mhc_kv.so")
INCLUDE = os.path.join(ROOT, "include")

ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-lineinfo", "-std=c++17", "--expt-relaxed-constexpr",
              "-Xcompiler", "-fPIC", "-I", INCLUDE]


def _nvcc() -> str:
    for cand in (shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmhc.so")


def _newest_dep_mtime() -> float:
    deps = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(INCLUDE, "*.h"))
    return max((os.path.getmtime(d) for d in deps), default=0.0)


def _compile(src: str, ptxas_v: bool) -> tuple[str, str]:
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    dep_t = max(os.path.getmtime(src), _newest_dep_mtime())
    if not ptxas_v and os.path.exists(obj) and os.path.getmtime(obj) >= dep_t:
        return obj, ""
    cmd = [_nvcc(), *ARCH, *NVCC_FLAGS, "-c", src, "-o", obj + ".tmp"]
    if ptxas_v:
        cmd += ["-Xptxas", "-v"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    os.replace(obj + ".tmp", obj)
    return obj, r.stderr


def _run(cmd: list, what: str) -> None:
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")


def _binding_made_for() -> str:
    """What the kv binding's object code depends on beside its sources: the
    interpreter, PyTorch and the toolkit whose headers it was compiled with."""
    import torch
    return "\n".join([sys.version, str(sysconfig.get_config_var("SOABI")), torch.__version__, str(torch.version.git_version),
                      os.path.dirname(torch.__file__), _nvcc()]) + "\n"


def _compile_binding() -> str:
    """The object of the kv binding, for the running interpreter and PyTorch."""
    import torch
    src, obj = os.path.join(CSRC, "kv_binding.cpp"), os.path.join(BUILD, "kv_binding.cpp.o")
    made_for, stamp = _binding_made_for(), obj + ".made_for"
    if os.path.exists(obj) and os.path.getmtime(obj) >= max(os.path.getmtime(src), _newest_dep_mtime()):
        if os.path.exists(stamp) and open(stamp).read() == made_for:
            return obj
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    dirs = [INCLUDE, inc, os.path.join(inc, "torch", "csrc", "api", "include"), cuda, sysconfig.get_paths()["include"]]
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    _run(["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={abi}", *[f"-I{d}" for d in dirs], "-c", src,
          "-o", obj + ".tmp"], "g++ for kv_binding.cpp")
    for old in (stamp, BINDING):              # nothing of the old object stays beside the new one
        if os.path.exists(old):
            os.remove(old)
    os.replace(obj + ".tmp", obj)
    with open(stamp, "w") as f:
        f.write(made_for)
    return obj


def _link_binding(obj: str) -> None:
    import torch
    if os.path.exists(BINDING) and os.path.getmtime(BINDING) >= os.path.getmtime(obj):
        return
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "lib64")
    tmp = BINDING + f".{os.getpid()}.tmp"
    _run(["g++", "-shared", "-o", tmp, obj, f"-L{BUILD}", "-l:libmhc.so", "-Wl,-rpath,$ORIGIN", f"-L{libs}",
          "-ltorch_python", "-ltorch", "-ltorch_cpu", "-lc10", "-lc10_cuda", f"-L{cuda}", "-lcudart_static", "-ldl",
          "-lrt", "-lpthread"], "link of _mhc_kv.so")
    os.replace(tmp, BINDING)


def build(ptxas_v: bool = False, force: bool = False) -> str:
    """Compile ``csrc/``, link ``_build/libmhc.so`` and ``_build/_mhc_kv.so``; returns the former's path."""
    os.makedirs(BUILD, exist_ok=True)
    if force:
        for o in glob.glob(os.path.join(BUILD, "*.o")):
            os.remove(o)
    srcs = sorted(glob.glob(os.path.join(CSRC, "*.cu")))
    with cf.ThreadPoolExecutor(max_workers=min(8, len(srcs)) + 1) as ex:
        binding = ex.submit(_compile_binding)
        results = list(ex.map(lambda s: _compile(s, ptxas_v), srcs))
    if ptxas_v:
        for _, log in results:
            sys.stderr.write(log)
    objs = [o for o, _ in results]
    newest = max(os.path.getmtime(o) for o in objs)
    if force or ptxas_v or not os.path.exists(LIB) or os.path.getmtime(LIB) < newest:
        tmp = LIB + f".{os.getpid()}.tmp"
        cmd = [_nvcc(), *ARCH, "-shared", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link of libmhc.so failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    _link_binding(binding.result())
    return LIB


if __name__ == "__main__":
    print(build(ptxas_v="--ptxas-v" in sys.argv, force="--force" in sys.argv))
