"""Build the CUDA library libexl3_gb300.so in-tree with nvcc (sm_103a only), and
_native.so, the Python calls of its smallest operators, with g++ against the
installed torch and Python (and again when these are others).

Every translation unit compiles in parallel; the link uses the static CUDA
runtime so the library has no runtime search-path dependency.
"""
from __future__ import annotations

import concurrent.futures as cf
import glob
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OUT_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(OUT_DIR, "libexl3_gb300.so")
NATIVE_PATH = os.path.join(OUT_DIR, "_native.so")
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-O3", "-std=c++17", "-lineinfo", "-Xcompiler", "-fPIC,-O2",
              "--expt-relaxed-constexpr", "-Xptxas", "-warn-spills"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found; the CUDA toolkit is required to build the library")
    return cand


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale(obj: str, src: str, headers) -> bool:
    if not os.path.exists(obj):
        return True
    t = os.path.getmtime(obj)
    return any(os.path.getmtime(f) > t for f in [src] + headers)


def native_stamp() -> str:
    """What _native.so is built against (torch's C++ side and Python's have no
    stable ABI): written beside it, and compared before it is loaded."""
    import torch
    return (f"torch {torch.__version__}, C++11 ABI {int(torch._C._GLIBCXX_USE_CXX11_ABI)}, "
            f"Python {'.'.join(map(str, sys.version_info[:3]))} {sysconfig.get_config_var('SOABI')}")


def _stamp_path() -> str:
    return os.path.splitext(NATIVE_PATH)[0] + ".stamp"


def built_stamp():
    """native_stamp() of the built _native.so, None where there is none."""
    try:
        with open(_stamp_path()) as f:
            return f.read()
    except FileNotFoundError:
        return None


def _native_commands(tmp: str):
    """Compile and link lines of _native.so."""
    import torch
    root = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    obj = os.path.join(OUT_DIR, "binding.o") + f".tmp{os.getpid()}"
    inc = [os.path.join(root, "include"), os.path.join(root, "include/torch/csrc/api/include"),
           sysconfig.get_paths()["include"], os.path.join(cuda, "include")]
    abi = int(torch._C._GLIBCXX_USE_CXX11_ABI)
    return obj, ["g++", "-O2", "-std=c++17", "-fPIC", f"-D_GLIBCXX_USE_CXX11_ABI={abi}",
                 *[f"-I{i}" for i in inc], "-c", os.path.join(CSRC, "binding.cpp"), "-o", obj], \
        ["g++", "-shared", obj, "-o", tmp, f"-L{OUT_DIR}", "-lexl3_gb300",
         f"-L{os.path.join(root, 'lib')}", "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda",
         "-Wl,-rpath,$ORIGIN"]


def build(verbose: bool = False, force: bool = False, extra_flags=None) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    nvcc = _nvcc()
    headers = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        glob.glob(os.path.join(HERE, "..", "include", "*.h"))
    flags = NVCC_FLAGS + (extra_flags or [])
    jobs = []
    objs = []
    for src in sources():
        obj = os.path.join(OUT_DIR, os.path.basename(src).replace(".cu", ".o"))
        objs.append(obj)
        if force or _stale(obj, src, headers):
            # compiled to a private name and renamed, so processes building at
            # the same time (ranks of one job) never see a half-written object
            jobs.append(([nvcc, *ARCH, *flags, "-c", src, "-o", obj + f".tmp{os.getpid()}"], obj))

    def run(cmd):
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{os.path.basename(cmd[0])} failed: {' '.join(cmd)}\n{r.stdout}\n"
                               f"{r.stderr}")
        return r.stdout + r.stderr

    def compile_one(job):
        cmd, obj = job
        out = run(cmd)
        os.replace(cmd[-1], obj)
        return out

    binding = os.path.join(CSRC, "binding.cpp")
    native = native_obj = None
    stamp = native_stamp()
    if force or jobs or _stale(NATIVE_PATH, binding, headers) or not os.path.exists(LIB_PATH) or \
            built_stamp() != stamp:
        native = NATIVE_PATH + f".tmp{os.getpid()}"
        native_obj, compile_cmd, link_cmd = _native_commands(native)
    with cf.ThreadPoolExecutor(max_workers=max(1, min(len(jobs) + 1, os.cpu_count() or 4))) as ex:
        also = ex.submit(run, compile_cmd) if native else None
        for out in ex.map(compile_one, jobs):
            if verbose and out.strip():
                print(out)
        # (the library, which C programs use, needs nothing of the binding)
        if force or jobs or not os.path.exists(LIB_PATH):
            tmp = LIB_PATH + f".tmp{os.getpid()}"
            run([nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"])
            os.replace(tmp, LIB_PATH)
        if also:
            also.result()
    if native:
        run(link_cmd)
        os.remove(native_obj)
        os.replace(native, NATIVE_PATH)
        tmp = _stamp_path() + f".tmp{os.getpid()}"
        with open(tmp, "w") as f:
            f.write(stamp)
        os.replace(tmp, _stamp_path())
    return LIB_PATH


if __name__ == "__main__":
    print(build(verbose=True))
