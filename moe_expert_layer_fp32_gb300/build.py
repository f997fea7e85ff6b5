"""Builds libmoe_gb300.so (the C ABI of include/moe.h) from csrc/ with nvcc for
sm_103a, in-tree.  One nvcc process per translation unit, run in parallel, then
one link; beside them g++ builds _tensor_calls.so (csrc/tensor_calls.cpp, the
tensor calls' fast path) against torch's headers; a host without g++ or those headers
goes without it, and the package calls the library from Python alone.  Usage:
``python moe_expert_layer_fp32_gb300/build.py [--force] [-v]`` (run it by path: importing the
package itself needs the built library)."""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
BUILD = os.path.join(ROOT, "_build", "moe_gb300")
LIB = os.path.join(PKG, "libmoe_gb300.so")
CALLS_SRC = os.path.join(CSRC, "tensor_calls.cpp")
CALLS = os.path.join(PKG, "_tensor_calls.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def headers():
    return sorted(glob.glob(os.path.join(CSRC, "*.cuh")) +
                  [os.path.join(ROOT, "include", "moe.h")])


def built_for_this_machine(path: str) -> bool:
    """The library's ELF machine field matches this host (x86_64 or aarch64): a
    library copied from a machine of the other architecture is rebuilt."""
    import platform
    want = {"x86_64": 0x3E, "amd64": 0x3E, "aarch64": 0xB7, "arm64": 0xB7}.get(
        platform.machine().lower())
    try:
        with open(path, "rb") as f:
            head = f.read(20)
    except OSError:
        return False
    if len(head) < 20 or head[:4] != b"\x7fELF":
        return False
    return want is None or int.from_bytes(head[18:20], "little") == want


def newest_source() -> float:
    return max(os.path.getmtime(p) for p in sources() + headers() + [CALLS_SRC, __file__])


def up_to_date() -> bool:
    built = [LIB] if calls_missing() else [LIB, CALLS]
    return (all(built_for_this_machine(p) for p in built) and
            newest_source() <= min(os.path.getmtime(p) for p in built))


def cxx() -> str:
    return os.environ.get("CXX", "g++")


def calls_includes():
    import sysconfig
    from torch.utils import cpp_extension
    return cpp_extension.include_paths() + [
        sysconfig.get_paths()["include"], os.path.join(os.path.dirname(nvcc()), "..", "include"),
        os.path.join(ROOT, "include")]


def calls_missing():
    """What _tensor_calls.so cannot be built without and is not here, or None."""
    if shutil.which(cxx()) is None:
        return f"no compiler {cxx()}"
    inc = calls_includes()
    for h in ("Python.h", "torch/csrc/autograd/python_variable.h"):
        if not any(os.path.exists(os.path.join(i, h)) for i in inc):
            return f"no header {h}"
    return None


def build_calls() -> None:
    import torch
    from torch.utils import cpp_extension
    missing = calls_missing()
    if missing:
        print(f"_tensor_calls.so: not built ({missing}); the tensor calls go through Python",
              file=sys.stderr)
        if os.path.exists(CALLS):  # an older one would not match the sources
            os.remove(CALLS)
        return
    tmp = CALLS + f".tmp{os.getpid()}"
    r = subprocess.run(
        [cxx(), "-O2", "-std=c++17", "-fPIC", "-shared", CALLS_SRC, "-o", tmp,
         f'-DMOE_BUILT_WITH_TORCH="{torch.__version__}"', *["-I" + i for i in calls_includes()],
         *["-L" + d for d in cpp_extension.library_paths()], "-lc10", "-lc10_cuda", "-ltorch_cpu",
         "-ltorch_python", "-ldl"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cxx()} failed on {CALLS_SRC}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALLS)


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and up_to_date():
        print(f"{LIB}: up to date (built here, newer than every source)", file=sys.stderr)
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    cc = nvcc()
    flags = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
                    "-I", os.path.join(ROOT, "include")]
    if verbose:
        flags += ["-Xptxas", "-v"]

    def compile_one(src):
        obj = os.path.join(BUILD, os.path.basename(src) + ".o")
        r = subprocess.run([cc, *flags, "-c", src, "-o", obj], capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    # (the longest first: the routers, then the rest)
    order = sorted(sources(), key=os.path.getsize, reverse=True)
    with cf.ThreadPoolExecutor(max_workers=min(12, os.cpu_count() or 1)) as ex:
        calls = ex.submit(build_calls)
        results = list(ex.map(compile_one, sorted(order, key=lambda p: "route" not in p)))
        calls.result()
    if verbose:
        for obj, log in results:
            sys.stderr.write(log)
    tmp = LIB + f".tmp{os.getpid()}"
    r = subprocess.run([cc, *ARCH, "-shared", "-o", tmp, *[o for o, _ in results]],
                       capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
