"""Build libgemm_nt.so in-tree for sm_103a (GB300).

    python -m dense_fp16_tensor_gemm_gb300._build [--force] [--verbose]

Each CUDA translation unit is compiled in parallel with nvcc, then linked into
dense_fp16_tensor_gemm_gb300/_build/libgemm_nt.so with the static CUDA runtime
(no libcuda link: the driver's tensor-map encoder is fetched at run time), so
the library loads on machines without a GPU driver.  Beside it, with g++,
_build/_tensor_calls.so: the common case of the feed-forward tensor forms as a
Python extension (csrc/tensor_calls.cpp).  Where it does not compile, a warning says
so and the forms are marshalled in Python.
"""
import concurrent.futures as cf
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(PKG, "csrc")
ROOT = os.path.dirname(PKG)
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(OUT_DIR, "libgemm_nt.so")
CALLS = os.path.join(OUT_DIR, "_tensor_calls.so")
CALLS_FOR = CALLS + ".for"  # what it was last built for, or tried to be, and the outcome
BUILT, FAILED = "built\n", "did not compile\n"

SOURCES = ["gemm_nt_api.cu", "tc05_gemm.cu", "tc05_small.cu", "tc05_pair.cu", "mmasync_gemm.cu", "gemm_nt_no_alloc.cu", "mx_scales.cu",
           "block128_api.cu", "block128_any.cu", "block128_pair.cu", "block128_swap.cu",
           "block128_quant.cu", "moe.cu",
           "ffn_api.cu", "ffn_any.cu", "ffn_few.cu", "ffn_swap.cu", "ffn_swap_f16.cu", "ffn_swap_plain.cu",
           "ffn_swap_plain_f16.cu", "gated_pair.cu", "gated_grad.cu", "w4_quant.cu",
           "copy_rows.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ["-std=c++17", "-O3", "-lineinfo", "-Xcompiler", "-fPIC", "-Xcompiler", "-Wall",
         "--expt-relaxed-constexpr", "-I", CSRC, "-I", INCLUDE]


def nvcc():
    exe = shutil.which("nvcc")
    if exe:
        return exe
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found")


def _deps():
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC)]
    files.append(os.path.join(INCLUDE, "gemm_nt.h"))
    files.append(os.path.abspath(__file__))
    return files


def _calls_command(out):
    """The g++ command of the Python extension; None where it cannot be built (no
    torch, no Python headers, no CUDA toolkit): the tensor forms are then marshalled in
    Python alone."""
    spec = importlib.util.find_spec("torch")
    include = sysconfig.get_paths()["include"]
    if spec is None or not os.path.exists(os.path.join(include, "Python.h")):
        return None
    torch = list(spec.submodule_search_locations)[0]
    lib = os.path.join(torch, "lib")
    if not os.path.exists(os.path.join(lib, "libc10_cuda.so")):  # a torch without CUDA
        return None
    try:
        cuda = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc()))), "include")
    except RuntimeError:
        return None
    return ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-I", INCLUDE, "-isystem", os.path.join(torch, "include"),
            "-isystem", os.path.join(torch, "include", "torch", "csrc", "api", "include"), "-isystem", include,
            "-isystem", cuda, os.path.join(CSRC, "tensor_calls.cpp"), "-o", out, "-L", lib, "-ltorch_python", "-ltorch_cpu",
            "-lc10", "-lc10_cuda", "-Wl,-rpath," + lib]


def _calls_key():
    """What the extension depends on beside its sources: the torch release, the Python and
    its headers' place."""
    spec = importlib.util.find_spec("torch")
    if spec is None:
        return ""
    try:
        release = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        release = "unknown"
    return "torch %s in %s\npython %s\n" % (release, list(spec.submodule_search_locations)[0],
                                            sysconfig.get_config_var("EXT_SUFFIX"))


def _calls_stale():
    """Whether the extension is missing or for another torch or Python than this one's.  One
    that did not compile is not tried again until those or the sources change; nothing is
    where the folder cannot be written."""
    if _calls_command(CALLS) is None or not os.access(OUT_DIR, os.W_OK):
        return False
    try:
        with open(CALLS_FOR) as f:
            record = f.read()
    except OSError:
        return True
    if record == _calls_key() + BUILT:
        return not os.path.exists(CALLS)
    return record != _calls_key() + FAILED


def build_calls():
    """Compiles the Python extension, without which the library is whole: where that fails,
    what the compiler said is a warning."""
    tmp = CALLS + ".tmp.%d" % os.getpid()
    cmd = _calls_command(tmp)
    if cmd is None:
        return
    os.makedirs(OUT_DIR, exist_ok=True)
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
        said = None if r.returncode == 0 else r.stdout + r.stderr
    except OSError as e:  # no g++
        said = str(e)
    if said is None:
        os.replace(tmp, CALLS)
    else:
        warnings.warn("csrc/tensor_calls.cpp does not compile; the feed-forward tensor forms are marshalled in Python, at "
                      "about three times the host time a call:\n%s" % said[-2000:], stacklevel=2)
        if os.path.exists(CALLS):
            os.remove(CALLS)  # (of other sources, or another torch)
    with open(CALLS_FOR, "w") as f:
        f.write(_calls_key() + (BUILT if said is None else FAILED))


def _stale():
    if not os.path.exists(LIB):
        return True
    t = os.path.getmtime(LIB)
    return any(os.path.getmtime(f) > t for f in _deps())


def build(force=False, verbose=False, extra_flags=()):
    """Compile (if needed) and return the path of libgemm_nt.so."""
    if not force and not _stale():
        if _calls_stale():
            build_calls()
        return LIB
    os.makedirs(OUT_DIR, exist_ok=True)
    cc = nvcc()
    objs = []

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.splitext(src)[0] + ".o")
        cmd = [cc, *ARCH, *FLAGS, *extra_flags, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError("nvcc failed on %s:\n%s%s" % (src, r.stdout, r.stderr))
        if verbose and (r.stdout or r.stderr):
            print(r.stdout + r.stderr, flush=True)
        return obj

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        calls = ex.submit(build_calls)
        objs = list(ex.map(compile_one, SOURCES))
        calls.result()
    tmp = LIB + ".tmp.%d" % os.getpid()
    cmd = [cc, *ARCH, "-shared", "-cudart", "static", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError("link failed:\n%s%s" % (r.stdout, r.stderr))
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="--verbose" in sys.argv))
