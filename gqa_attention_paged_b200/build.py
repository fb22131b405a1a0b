"""Build libgqa_paged.so (the sm_100a CUDA library behind include/gqa_paged.h) in-tree
with nvcc, and beside it the compiled half of the binding, without which calls from Python take
longer.  `python -m gqa_attention_paged_b200.build [--force]`."""
import glob
import importlib.metadata
import importlib.util
import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libgqa_paged.so")


def _torch_version():
    try:
        return importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        return "-unknown"


# of one Python and one torch, which its name tells
FASTCALL = os.path.join(PKG, "_fastcall-torch" + _torch_version() + (sysconfig.get_config_var("EXT_SUFFIX") or ".so"))
NVCC = os.environ.get("NVCC", "/usr/local/cuda/bin/nvcc")
CXX = os.environ.get("CXX", "g++")

FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
         "-Xcompiler", "-fPIC", "--expt-relaxed-constexpr", "-Xptxas", "-v"]


def _old(target, deps):
    return not os.path.exists(target) or any(os.path.getmtime(d) > os.path.getmtime(target) for d in deps)


def _torch_include():
    """Of torch's headers only the DLPack one is used, which includes nothing of torch."""
    spec = importlib.util.find_spec("torch")
    return os.path.join(os.path.dirname(spec.origin), "include")


def sources():
    return sorted(glob.glob(os.path.join(CSRC, "*.cu")))


def _stale():
    return _old(LIB, sources() + [f for pat in ("*.cuh", "*.h") for f in glob.glob(os.path.join(CSRC, pat))] +
                glob.glob(os.path.join(INCLUDE, "*.h")))


def _fastcall_stale():
    return _old(FASTCALL, [os.path.join(CSRC, "fastcall.cpp")] + glob.glob(os.path.join(INCLUDE, "*.h")))


def build_fastcall():
    """The binding's C half, a CPython extension that knows the library by its functions' addresses.
    Returns why it could not be built (no C++ compiler, no Python headers, a torch whose DLPack header has
    no exchange table), or None."""
    tmp = FASTCALL + f".tmp{os.getpid()}"
    try:
        cmd = [CXX, "-O2", "-std=c++17", "-shared", "-fPIC", "-Wall", "-I", INCLUDE, "-I",
               os.path.join(os.path.dirname(os.path.dirname(NVCC)), "include"), "-I",
               sysconfig.get_paths()["include"], "-I", _torch_include(),
               os.path.join(CSRC, "fastcall.cpp"), "-o", tmp]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            return f"{CXX} failed on fastcall.cpp:\n{r.stdout}\n{r.stderr}"
        os.replace(tmp, FASTCALL)
    except OSError as e:
        return f"{CXX}: {e}"
    return None


def _report(why):
    if why:
        print(f"the binding's compiled half is left out: {why}", file=sys.stderr)
    return why or ""


def build(force: bool = False, verbose: bool = False) -> str:
    if not force and not _stale():
        if _fastcall_stale():
            _report(build_fastcall())
        return LIB
    objdir = os.path.join(PKG, "_build")
    os.makedirs(objdir, exist_ok=True)
    objs = []
    log = []
    for src in sources():
        obj = os.path.join(objdir, os.path.basename(src) + ".o")
        cmd = [NVCC, *FLAGS, "-I", INCLUDE, "-I", CSRC, "-c", src, "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        log.append(r.stdout + r.stderr)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        objs.append(obj)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [NVCC, "-gencode", "arch=compute_100a,code=sm_100a", "-shared", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    log.append(_report(build_fastcall()))
    with open(os.path.join(objdir, "ptxas.log"), "w") as f:
        f.write("\n".join(log))
    if verbose:
        print("\n".join(log))
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
