"""Build in-tree: libkda.so, every csrc/*.cu compiled for sm_100a and linked into one library; and _check.so,
the binding's checks of a call's tensors in one go (csrc/kda_check.cpp, compiled against this Python and torch).
The library needs nvcc alone.  Without what the second needs the binding checks tensors in Python."""
import concurrent.futures as cf
import glob
import os
import subprocess
import sys
import warnings

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libkda.so")
CHECK_SRC = os.path.join(CSRC, "kda_check.cpp")
CHECK_LIB = os.path.join(HERE, "_check.so")
CHECK_FOR = os.path.join(HERE, "_check.for")  # the Python and torch that _check.so was built for
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
ARCH = ["-gencode", "arch=compute_100a,code=sm_100a"]
FLAGS = ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
         "--expt-relaxed-constexpr"]


def _sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _deps():
    return _sources() + glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h")) + \
        [os.path.join(HERE, "..", "include", "kda.h"), os.path.abspath(__file__)]


def _stale():
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(p) > t for p in _deps())


def _compile(src, verbose):
    obj = os.path.join(BUILD, os.path.basename(src) + ".o")
    cmd = [NVCC, *ARCH, *FLAGS, "-c", src, "-o", obj]
    if verbose:
        cmd.insert(1, "-Xptxas=-v")
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    return obj, r.stderr


def check_target():
    """The Python and torch of this process, as _check.for names them."""
    import torch
    return f"{sys.implementation.cache_tag} torch-{torch.__version__} abi-{int(torch._C._GLIBCXX_USE_CXX11_ABI)}\n"


def check_fits():
    """Whether _check.so is there and was built for this Python and torch; another one must not be loaded."""
    try:
        with open(CHECK_FOR) as f:
            return os.path.exists(CHECK_LIB) and f.read() == check_target()
    except OSError:
        return False


def build_check(force=False):
    """_check.so, if it is missing, older than its source, or built for another Python or torch."""
    if not force and check_fits() and os.path.getmtime(CHECK_LIB) >= os.path.getmtime(CHECK_SRC):
        return CHECK_LIB
    import sysconfig

    import torch
    root = os.path.dirname(torch.__file__)
    lib = os.path.join(root, "lib")
    tmp = CHECK_LIB + ".tmp"
    r = subprocess.run(["g++", "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
                        f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
                        "-isystem", os.path.join(root, "include"),
                        "-isystem", os.path.join(root, "include", "torch", "csrc", "api", "include"),
                        "-isystem", sysconfig.get_paths()["include"], CHECK_SRC, "-o", tmp, "-L" + lib,
                        "-Wl,-rpath," + lib, "-ltorch_python", "-ltorch_cpu", "-lc10"], capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on {CHECK_SRC}:\n{r.stdout}\n{r.stderr}")
    if os.path.exists(CHECK_FOR):
        os.remove(CHECK_FOR)
    os.replace(tmp, CHECK_LIB)
    with open(CHECK_FOR, "w") as f:
        f.write(check_target())
    return CHECK_LIB


def build(force=False, verbose=False):
    lib = _build_library(force, verbose)
    try:
        build_check(force)
    except (RuntimeError, OSError, ImportError) as e:
        warnings.warn(f"_check.so was not built, tensors are checked in Python: {str(e)[:500]}")
    return lib


def _build_library(force, verbose):
    if not force and not _stale():
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=min(8, os.cpu_count() or 1)) as ex:
        results = list(ex.map(lambda s: _compile(s, verbose), _sources()))
    if verbose:
        for _, log in results:
            sys.stderr.write(log)
    objs = [o for o, _ in results]
    tmp = LIB + ".tmp"
    subprocess.run([NVCC, *ARCH, "-shared", "-o", tmp, *objs, "-lcudart", "-lcuda"], check=True)
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
