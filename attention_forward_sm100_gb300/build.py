"""Builds libattn_fwd.so in-tree with nvcc for sm_103a.

Every translation unit under csrc/ is compiled in parallel into _build/ and
linked into attention_forward_sm100_gb300/libattn_fwd.so (CUDA runtime linked
statically, driver entry points resolved at run time); python_paged.cpp, which
needs Python's and torch's headers, becomes the extension module _paged_native
next to it. The ptxas report of
each persistent kernel is checked: it must be allocated exactly 128 registers
per thread (the kernel redistributes them between warpgroups with setmaxnreg,
whose budget is computed from that number) and may spill at most a few words.
"""
from __future__ import annotations

import concurrent.futures
import glob
import os
import platform
import re
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
BUILD_DIR = os.path.join(ROOT, "_build", platform.machine())
LIB_PATH = os.path.join(HERE, "libattn_fwd.so")
NATIVE_SRC = os.path.join(CSRC, "python_paged.cpp")
NATIVE_PATH = os.path.join(HERE, "_paged_native.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
CFLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xptxas", "-v",
                 "--expt-relaxed-constexpr", "-I" + os.path.join(ROOT, "include")]
PERSISTENT_KERNELS = ("fa_tc05_kernel",)
REGS_EXPECTED = 128
SPILL_LIMIT = 64   # bytes of local-memory spill tolerated per persistent kernel


def _nvcc():
    cand = os.environ.get("NVCC") or shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found; set NVCC")
    return cand


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps_mtime():
    files = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(ROOT, "include", "*.h")) + [os.path.abspath(__file__)]
    return max(os.path.getmtime(f) for f in files)


def _check_ptxas(log: str, src: str):
    """Checks register allocation and spills of the persistent kernels."""
    entries = re.split(r"ptxas info\s*: Compiling entry function", log)
    for chunk in entries[1:]:
        name = chunk.split("'")[1] if "'" in chunk else ""
        if not any(k in name for k in PERSISTENT_KERNELS):
            continue
        m = re.search(r"Used (\d+) registers", chunk)
        spills = re.search(r"(\d+) bytes spill stores, (\d+) bytes spill loads", chunk)
        if m is None:
            raise RuntimeError(f"{src}: no register report for {name}")
        if int(m.group(1)) != REGS_EXPECTED:
            raise RuntimeError(f"{src}: {name} uses {m.group(1)} registers, the register split needs "
                               f"exactly {REGS_EXPECTED}")
        if spills and max(int(spills.group(1)), int(spills.group(2))) > SPILL_LIMIT:
            raise RuntimeError(f"{src}: {name} spills ({spills.group(0)})")
        if spills and int(spills.group(1)):
            print(f"warning: {src}: {name}: {spills.group(0)}", file=sys.stderr)


def _compile(src: str, force: bool) -> str:
    obj = os.path.join(BUILD_DIR, os.path.basename(src)[:-3] + ".o")
    log_path = obj + ".ptxas.txt"
    if not force and os.path.exists(obj) and os.path.getmtime(obj) >= max(os.path.getmtime(src), _deps_mtime()):
        return obj
    cmd = [_nvcc()] + CFLAGS + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    with open(log_path, "w") as f:
        f.write(" ".join(cmd) + "\n" + r.stdout + r.stderr)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {os.path.basename(src)}:\n{r.stderr[-6000:]}")
    _check_ptxas(r.stdout + r.stderr, os.path.basename(src))
    return obj


def _compile_native(force: bool) -> str:
    """Object file of the extension module (host code only)."""
    import torch
    obj = os.path.join(BUILD_DIR, "python_paged.o")
    stamp = obj + ".torch"   # the torch it was compiled against
    known = open(stamp).read() if os.path.exists(stamp) else ""
    headers = glob.glob(os.path.join(ROOT, "include", "*.h")) + [os.path.abspath(__file__), NATIVE_SRC,
                                                                   os.path.join(CSRC, "paged_host.h")]
    if not force and known == torch.__version__ and os.path.exists(obj) and \
            os.path.getmtime(obj) >= max(os.path.getmtime(f) for f in headers):
        return obj
    inc = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden", "-w",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-isystem", inc, "-isystem",
           os.path.join(inc, "torch", "csrc", "api", "include"), "-isystem", cuda, "-isystem",
           sysconfig.get_paths()["include"], "-c", NATIVE_SRC, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for python_paged.cpp:\n{r.stderr[-6000:]}")
    with open(stamp, "w") as f:
        f.write(torch.__version__)
    return obj


def _link_native(obj: str, force: bool):
    """_paged_native.so: finds libattn_fwd.so beside it and torch's libraries where torch loaded them."""
    import torch
    if not force and os.path.exists(NATIVE_PATH) and \
            os.path.getmtime(NATIVE_PATH) >= max(os.path.getmtime(obj), os.path.getmtime(LIB_PATH)):
        return
    libs = os.path.join(os.path.dirname(torch.__file__), "lib")
    cuda_rt = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "lib64")
    tmp = NATIVE_PATH + ".tmp"
    cmd = ["g++", "-shared", "-o", tmp, obj, "-L" + HERE, "-lattn_fwd", "-Wl,-rpath,$ORIGIN", "-L" + libs,
           "-ltorch_python", "-ltorch_cuda", "-ltorch_cpu", "-lc10_cuda", "-lc10", "-Wl,-rpath," + libs, "-L" + cuda_rt,
           "-lcudart_static", "-ldl", "-lrt", "-lpthread"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link of _paged_native failed:\n{r.stderr[-4000:]}")
    os.replace(tmp, NATIVE_PATH)


def build(force: bool = False, jobs: int | None = None) -> str:
    """Compiles (incrementally) and links the library and the extension module; returns the library's path."""
    os.makedirs(BUILD_DIR, exist_ok=True)
    srcs = _sources()
    jobs = jobs or min(len(srcs) + 1, (os.cpu_count() or 4) + 1)
    with concurrent.futures.ThreadPoolExecutor(max_workers=jobs) as ex:
        native = ex.submit(_compile_native, force)
        objs = list(ex.map(lambda s: _compile(s, force), srcs))
        native_obj = native.result()
    if force or not os.path.exists(LIB_PATH) or os.path.getmtime(LIB_PATH) < max(os.path.getmtime(o) for o in objs):
        tmp = LIB_PATH + ".tmp"
        cmd = [_nvcc()] + ARCH + ["-shared", "-o", tmp, "-Xlinker", "-soname=libattn_fwd.so"] + objs
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stderr[-4000:]}")
        os.replace(tmp, LIB_PATH)
    _link_native(native_obj, force)
    return LIB_PATH


if __name__ == "__main__":
    print(build(force="--force" in sys.argv))
