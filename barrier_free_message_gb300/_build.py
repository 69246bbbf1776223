"""Build libsfar.so in-tree with nvcc for sm_103a.

Each .cu file is compiled on its own (in parallel) and the objects are linked
into ``barrier_free_message_gb300/_build/libsfar.so``.  Beside it the host
compiler builds ``sfar_tensors.so``, the Python module that reads the torch
tensors of the paged cache's and the 8-bit projection's calls.  A stamp of the
sources, flags and torch's and Python's versions skips the build when nothing
changed.
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


def _stamp() -> str:
    h = hashlib.sha256()
    h.update(" ".join(NVCC_FLAGS).encode())
    h.update(f"{importlib.metadata.version('torch')} {sys.version}".encode())
    for d in (CSRC, INCLUDE):
        for name in sorted(os.listdir(d)):
            with open(os.path.join(d, name), "rb") as f:
                h.update(name.encode())
                h.update(f.read())
    return h.hexdigest()


def _build_tensors(cc: str) -> None:
    torch = os.path.dirname(importlib.util.find_spec("torch").origin)
    libs = os.path.join(torch, "lib")
    inc = [INCLUDE, os.path.join(torch, "include"), os.path.join(torch, "include", "torch", "csrc", "api", "include"),
           sysconfig.get_paths()["include"], os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(cc))), "include")]
    tmp = TENSORS + f".tmp{os.getpid()}"
    cmd = [os.environ.get("CXX", "g++"), "-O2", "-std=c++17", "-shared", "-fPIC", "-fvisibility=hidden",
           os.path.join(CSRC, "sfar_tensors.cpp"), "-o", tmp, *["-I" + i for i in inc], "-L" + libs, "-Wl,-rpath," + libs,
           "-ltorch_python", "-ltorch_cpu", "-lc10_cuda", "-lc10"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"{cmd[0]} failed on sfar_tensors.cpp:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, TENSORS)


def build(force: bool = False, verbose: bool = False) -> str:
    os.makedirs(OUT_DIR, exist_ok=True)
    stamp_file = os.path.join(OUT_DIR, "stamp")
    stamp = _stamp()
    if not force and os.path.exists(LIB) and os.path.exists(TENSORS) and os.path.exists(stamp_file):
        with open(stamp_file) as f:
            if f.read() == stamp:
                return LIB
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

    with cf.ThreadPoolExecutor(max_workers=min(len(SOURCES) + 1, os.cpu_count() or 4)) as ex:
        tensors = ex.submit(_build_tensors, cc)
        results = list(ex.map(compile_one, SOURCES))
        tensors.result()
    if verbose:
        for _, log in results:
            print(log)
    tmp = LIB + f".tmp{os.getpid()}"
    cmd = [cc, "-shared", *ARCH, "-o", tmp, *[o for o, _ in results]]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    with open(stamp_file, "w") as f:
        f.write(stamp)
    return LIB


if __name__ == "__main__":
    import sys
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
