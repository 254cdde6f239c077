"""Build librptq.so in place: every CUDA source compiled for sm_100a (B200) with nvcc; and the Python binding of the
paged-cache calls (host code against PyTorch's and Python's headers; the library and the other calls do without it).

    python -m post_activation_quantization_b200.build [--verbose-ptxas]
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "librptq.so")
BUILD = os.path.join(ROOT, "_build")
SOURCES = ["api.cu", "calib.cu", "kmeans.cu", "ln_quant.cu", "kv_quant.cu", "dequant.cu", "kv_attention.cu", "explicit_reorder.cu", "linear.cu",
           "kv_paged.cu", "kv_paged_attention.cu", "kv_paged_decode.cu", "kv_paged_chunk.cu"]
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), "/usr/local/cuda/bin/nvcc", shutil.which("nvcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def _deps(src: str) -> list[str]:
    return [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".cuh", ".h"))] + [
        os.path.join(ROOT, "include", "rptq.h"), os.path.join(ROOT, "include", "rptq_testing.h"),
        os.path.join(ROOT, "include", "rptq_baseline.h"), src]


def _stale(out: str, deps: list[str]) -> bool:
    if not os.path.exists(out):
        return True
    t = os.path.getmtime(out)
    return any(os.path.getmtime(d) > t for d in deps)


def marshal_path() -> str:
    """The binding's file, named by what it was compiled against: one of another Python or PyTorch is never loaded."""
    import torch
    return os.path.join(PKG, f"_marshal-{sys.implementation.cache_tag}-torch{torch.__version__}.so")


def build_marshal(force: bool = False) -> str:
    out, src = marshal_path(), os.path.join(CSRC, "marshal.cpp")
    if not force and not _stale(out, [src, os.path.join(ROOT, "include", "rptq.h")]):
        return out
    import sysconfig

    import torch
    home, cuda = os.path.dirname(torch.__file__), os.path.dirname(os.path.dirname(nvcc()))
    inc = [f for d in (os.path.join(home, "include"), os.path.join(home, "include", "torch", "csrc", "api", "include"),
                       os.path.join(cuda, "include"), sysconfig.get_paths()["include"]) for f in ("-isystem", d)]
    lib = os.path.join(home, "lib")
    tmp = out + f".tmp{os.getpid()}"
    try:
        subprocess.check_call(["g++", "-O2", "-std=c++17", "-fPIC", "-shared",
                               f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *inc, src, "-o", tmp,
                               "-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python", f"-Wl,-rpath,{lib}"])
    except Exception:
        if os.path.exists(out):
            os.remove(out)  # an older source's: not to be loaded in its place
        raise
    os.replace(tmp, out)
    return out


def build(force: bool = False, ptxas_verbose: bool = False, jobs: int = 8) -> str:
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC,-O2",
                    "--expt-relaxed-constexpr", "-I", os.path.join(ROOT, "include")]
    if ptxas_verbose:
        flags += ["-Xptxas", "-v"]
    objs, cmds = [], []
    for s in SOURCES:
        src = os.path.join(CSRC, s)
        obj = os.path.join(BUILD, s.replace(".cu", ".o"))
        objs.append(obj)
        if force or ptxas_verbose or _stale(obj, _deps(src)):
            cmds.append([cc, *flags, "-c", src, "-o", obj])

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        return cmd, r

    with cf.ThreadPoolExecutor(max_workers=jobs) as ex:
        marshal = ex.submit(build_marshal, force)
        for cmd, r in ex.map(run, cmds):
            if ptxas_verbose or r.returncode != 0:
                sys.stderr.write(r.stdout + r.stderr)
            if r.returncode != 0:
                raise RuntimeError(f"nvcc failed: {' '.join(cmd)}")
    if force or cmds or not os.path.exists(LIB) or any(os.path.getmtime(o) > os.path.getmtime(LIB) for o in objs):
        tmp = LIB + f".tmp{os.getpid()}"
        subprocess.check_call([cc, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart"])
        os.replace(tmp, LIB)
    try:
        marshal.result()
    except (OSError, ImportError, subprocess.CalledProcessError) as e:
        sys.stderr.write(f"the paged-cache calls of rptq.py have no binding, all else is built: {e}\n")
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, ptxas_verbose="--verbose-ptxas" in sys.argv)
    print(LIB)
