"""Build libvv.so in-tree with nvcc for sm_100a (B200).

    python -m int4_blockwise_quantised_b200.build [--force] [-j N] [--lib-only]

Each csrc/*.cu compiles to an object under _build/ (in parallel, skipped when up to date), then
all objects link into int4_blockwise_quantised_b200/libvv.so with the CUDA runtime linked
statically.  csrc/marshal.cpp (tensor arguments of the batch operators) compiles with the host
compiler against torch into the extension module _marshal (its file name carries the Python ABI; it is
built again for another torch), which links libvv.so; it needs
Python's headers and a CUDA build of torch, and --lib-only leaves it out (C callers, and every
Python entry point but the batch operators').
"""

import argparse
import concurrent.futures as cf
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build")
LIB = os.path.join(PKG, "libvv.so")
MARSHAL = os.path.join(PKG, "_marshal" + sysconfig.get_config_var("EXT_SUFFIX"))
INCLUDE = os.path.join(ROOT, "include")

ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-rdc=true", "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr",
         "-Xptxas", "-warn-spills", "-I", INCLUDE]


def nvcc():
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith(".cu"))


def headers():
    hs = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if f.endswith((".h", ".cuh"))]
    return hs + [os.path.join(INCLUDE, f) for f in os.listdir(INCLUDE) if f.endswith(".h")]


def _compile(src, force, extra):
    obj = os.path.join(BUILD, os.path.basename(src)[:-3] + ".o")
    newest_dep = max([os.path.getmtime(src)] + [os.path.getmtime(h) for h in headers()])
    if not force and os.path.exists(obj) and os.path.getmtime(obj) >= newest_dep:
        return obj, ""
    cmd = [nvcc()] + ARCH + FLAGS + extra + ["-c", src, "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def _made_for():
    """The Python and the torch that _marshal is compiled against (torch is not imported)."""
    spec = importlib.util.find_spec("torch")
    where = os.path.dirname(spec.origin) if spec else "none"
    return f"{sysconfig.get_config_var('SOABI')} torch {importlib.metadata.version('torch')} {where}"


def _compile_marshal(force):
    src, obj, stamp = os.path.join(CSRC, "marshal.cpp"), os.path.join(BUILD, "marshal.o"), os.path.join(BUILD, "marshal.txt")
    newest_dep = max(os.path.getmtime(p) for p in (src, os.path.join(INCLUDE, "vv.h")))
    made_for = open(stamp).read() if os.path.exists(stamp) else None
    if (not force and made_for == _made_for() and os.path.exists(obj) and os.path.getmtime(obj) >= newest_dep):
        return obj
    from torch.utils import cpp_extension as ext

    inc = ext.include_paths() + [sysconfig.get_paths()["include"], "/usr/local/cuda/include"]
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-Wall", "-c", src, "-o", obj]
    cmd += [f for d in inc for f in ("-isystem", d)]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {src}:\n{r.stdout}\n{r.stderr}")
    with open(stamp, "w") as f:
        f.write(_made_for())
    return obj


def _link_marshal(obj):
    import torch

    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    cmd = ["g++", "-shared", "-o", MARSHAL, obj, "-L", PKG, "-l:libvv.so", "-L", lib, "-ltorch_python",
           "-ltorch", "-ltorch_cpu", "-ltorch_cuda", "-lc10", "-lc10_cuda", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")


def build(force=False, jobs=None, verbose=False, extra=(), lib_only=False):
    os.makedirs(BUILD, exist_ok=True)
    srcs = sources()
    jobs = jobs or min(len(srcs), os.cpu_count() or 4)
    with cf.ThreadPoolExecutor(jobs + 1) as ex:
        marshal = None if lib_only else ex.submit(_compile_marshal, force)
        results = list(ex.map(lambda s: _compile(s, force, list(extra)), srcs))
    objs = [o for o, _ in results]
    if verbose:
        for _, log in results:
            if log.strip():
                print(log, file=sys.stderr)
    newest = max(os.path.getmtime(o) for o in objs)
    if force or not os.path.exists(LIB) or os.path.getmtime(LIB) < newest:
        cmd = [nvcc()] + ARCH + ["-rdc=true", "-shared", "-o", LIB] + objs + ["-cudart", "static"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    if lib_only:
        return LIB
    try:
        obj = marshal.result()
        if force or not os.path.exists(MARSHAL) or os.path.getmtime(MARSHAL) < max(
                os.path.getmtime(obj), os.path.getmtime(LIB)):
            _link_marshal(obj)
        untagged = os.path.join(PKG, "_marshal.so")  # an earlier build's: every Python would load it
        if os.path.exists(untagged):
            os.remove(untagged)
    except Exception as e:
        raise RuntimeError(f"{os.path.basename(LIB)} is built, {os.path.basename(MARSHAL)} (the batch "
                           "operators' Python side; --lib-only leaves it out) is not") from e
    return LIB


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--force", action="store_true")
    ap.add_argument("-j", type=int, default=None)
    ap.add_argument("-v", action="store_true", help="print ptxas resource usage")
    ap.add_argument("--lib-only", action="store_true", help="libvv.so without _marshal")
    a = ap.parse_args()
    extra = ["-Xptxas", "-v"] if a.v else []
    print(build(force=a.force or a.v, jobs=a.j, verbose=a.v, extra=extra, lib_only=a.lib_only))


if __name__ == "__main__":
    main()
