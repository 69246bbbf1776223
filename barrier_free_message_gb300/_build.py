"""Build libsfar.so in-tree with nvcc for sm_103a.

Each .cu file is compiled on its own (in parallel) and the objects are linked
into ``barrier_free_message_gb300/_build/libsfar.so``.  A stamp of the sources
and flags skips the build when nothing changed.

Beside it the host compiler builds ``sfar_tensors.so``, the Python module that
reads the torch tensors of the paged cache's and the 8-bit projection's calls,
with a stamp of its own (torch's and Python's versions too).  The library does
not need it: where it cannot be built, without torch or a header of it, a
warning says so and the calls that need it raise with the reason.
"""
import concurrent.futures as cf
import hashlib
import importlib.metadata
import importlib.util
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT_DIR = os.path.join(PKG, "_build")
LIB = os.path.join(OUT_DIR, "libsfar.so")
TENSORS = os.path.join(OUT_DIR, "sfar_tensors.so")

SOURCES = ["sfar_host.cu", "k_ll.cu", "k_ll128.cu", "k_sentinel.cu", "k_db.cu", "k_twoshot.cu", "k_twoshot_sent.cu", "k_tma.cu",
           "k_atomic.cu", "k_fused.cu", "k_fused8.cu", "k_fused_ts.cu", "k_gemv.cu",
           "k_misc.cu", "sfar_noalloc.cu", "k_kv_plan.cu", "k_kv_append.cu", "k_kv_attn.cu",
           "k_kv_prompt.cu", "k_quant8.cu", "k_gemm8.cu", "sfar_kv_host.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ["-std=c++17", "-O3", "-lineinfo", *ARCH, "-Xcompiler", "-fPIC", "-I" + INCLUDE, "-I" + CSRC]


def nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libsfar")


def _stamp(flags: str, dirs) -> str:
    h = hashlib.sha256()
    h.update(flags.encode())
    for d in dirs:
        for name in sorted(os.listdir(d)):
            with open(os.path.join(d, name), "rb") as f:
                h.update(name.encode())
                h.update(f.read())
    return h.hexdigest()


def _stamped(out: str, stamp: str) -> bool:
    if not (os.path.exists(out) and os.path.exists(out + ".stamp")):
        return False
    with open(out + ".stamp") as f:
        return f.read() == stamp


def _write(path: str, text: str) -> None:
    with open(path, "w") as f:
        f.write(text)


def _build_tensors(cc: str) -> None:
    spec = importlib.util.find_spec("torch")
    if spec is None:
        raise RuntimeError("torch is not installed")
    torch = os.path.dirname(spec.origin)
    libs = os.path.join(torch, "lib")
    inc = [INCLUDE, os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(cc))), "include")]
    tmp = TENSORS + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           os.path.join(CSRC, "sfar_tensors.cpp"), "-o", tmp, *["-I" + i for i in inc], "-L" + libs, "-Wl,-rpath," + libs,
           "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    try:
        r = subprocess.run(cmd, capture_output=True, text=True)
    except OSError as e:
        raise RuntimeError(f"{cmd[0]}: {e}") from e
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on sfar_tensors.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, TENSORS)


def tensors_error() -> str:
    """Why the module that reads tensors is not there ("" if it is)."""
    if os.path.exists(TENSORS):
        return ""
    if os.path.exists(TENSORS + ".err"):
        with open(TENSORS + ".err") as f:
            return f.read()
    return "not built"


def _tensors(force: bool) -> None:
    try:
        version = importlib.metadata.version("torch")
    except importlib.metadata.PackageNotFoundError:
        version = "none"
    stamp = _stamp(f"{version} {sys.version}", (CSRC, INCLUDE))
    if not force and _stamped(TENSORS, stamp):
        return
    for old in (TENSORS, TENSORS + ".stamp", TENSORS + ".err"):
        if os.path.exists(old):
            os.remove(old)                      # built from other sources
    try:
        _build_tensors(nvcc())
    except RuntimeError as e:
        _write(TENSORS + ".err", str(e))
        warnings.warn(f"libsfar's Python calls on whole tensors are not available: {e}", RuntimeWarning, stacklevel=3)
        return
    _write(TENSORS + ".stamp", stamp)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    with cf.ThreadPoolExecutor(max_workers=1) as ex:
        tensors = ex.submit(_tensors, force)
        _library(force, verbose)
        tensors.result()
    return LIB


def _library(force: bool, verbose: bool) -> None:
    stamp = _stamp(" ".join(NVCC_FLAGS), (CSRC, INCLUDE))
    if not force and _stamped(LIB, stamp):
        return
    cc = nvcc()

    def compile_one(src):
        obj = os.path.join(OUT_DIR, os.path.splitext(src)[0] + ".o")
        cmd = [cc, *NVCC_FLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            cmd.insert(1, "-Xptxas=-v")
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
        return obj, r.stderr

    with cf.ThreadPoolExecutor(max_workers=min(len(SOURCES), os.cpu_count() or 4)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    if verbose:
        for _, log in results:
            print(log)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, "-shared", *ARCH, "-o", tmp, *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    _write(LIB + ".stamp", stamp)


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
