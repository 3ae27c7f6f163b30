"""Build libb2pa.so (the C-ABI library) in-tree with nvcc for sm_103a.

Each .cu file under csrc/ is compiled in parallel to _build/, then linked
into paged_kv_prefill_gb300/libb2pa.so with the CUDA runtime linked
statically.  csrc/native.cpp, the Python module of direct bindings, is compiled
with g++ against this machine's Python and torch headers to _native.so.  The driver API is reached at run time through
cudaGetDriverEntryPointByVersion, so nothing links against libcuda.
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
BUILD = os.path.join(HERE, "_build")
LIB = os.path.join(HERE, "libb2pa.so")
NATIVE = os.path.join(HERE, "_native.so")
SOURCES = ["b2pa.cu", "attn_tc.cu", "attn_win.cu", "sched_gather.cu", "generic.cu", "append.cu", "decode.cu",
           "ops.cu", "rope.cu", "kv_scaled.cu", "attn_tree.cu", "ops_pages.cu", "pages.cu",
           "verify.cu", "attn_prefix.cu",
           "attn_split.cu", "attn_split64.cu", "attn_split8.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
FLAGS = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
                "--expt-relaxed-constexpr", "-I", os.path.join(os.path.dirname(HERE), "include")]


def _nvcc() -> str:
    p = shutil.which("nvcc")
    if p:
        return p
    cand = "/usr/local/cuda/bin/nvcc"
    if os.path.exists(cand):
        return cand
    raise RuntimeError("nvcc not found")


def _deps_mtime() -> float:
    m = 0.0
    for d in (CSRC, os.path.join(os.path.dirname(HERE), "include")):
        for f in os.listdir(d):
            m = max(m, os.path.getmtime(os.path.join(d, f)))
    return m


def _native_commands(tmp: str) -> list:
    """Compile and link commands of _native.so (to tmp)."""
    import torch

    root = os.path.dirname(torch.__file__)
    inc = [sysconfig.get_paths()["include"], os.path.join(root, "include"),
           os.path.join(root, "include", "torch", "csrc", "api", "include"),
           os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(_nvcc()))), "include")]
    obj = os.path.join(BUILD, "native.o")
    cxx = ["g++", "-O2", "-std=c++17", "-fPIC", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
    return [
        cxx + [x for i in inc for x in ("-isystem", i)] + ["-c", os.path.join(CSRC, "native.cpp"), "-o", obj],
        ["g++", "-shared", "-o", tmp, obj, "-L", HERE, "-l:libb2pa.so", "-Wl,-rpath,$ORIGIN",
         "-L", os.path.join(root, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_cuda"],
    ]


def _native_key() -> str:
    """What _native.so is compiled against: it reaches into torch's C++ objects."""
    import torch

    return f"{sys.version}\n{torch.__version__}\n{torch._C._GLIBCXX_USE_CXX11_ABI}\n"


def _native_is_current(key_file: str) -> bool:
    try:
        with open(key_file) as f:
            return f.read() == _native_key()
    except OSError:
        return False


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile and link what is older than its sources; return libb2pa.so's path.

    _native.so is made anew for another Python or torch too.  Where it cannot be made, the
    library is there all the same, and this raises."""
    newest, key_file = _deps_mtime(), os.path.join(BUILD, "native.key")

    def fresh(path: str) -> bool:
        return not force and os.path.exists(path) and os.path.getmtime(path) >= newest

    sources = [] if fresh(LIB) else SOURCES
    if not sources and fresh(NATIVE) and _native_is_current(key_file):
        return LIB
    os.makedirs(BUILD, exist_ok=True)
    nvcc = _nvcc()

    def one(src: str) -> str:
        obj = os.path.join(BUILD, src.replace(".cu", ".o"))
        cmd = [nvcc] + FLAGS + (["-Xptxas", "-v"] if ptxas_info else []) + ["-c", os.path.join(CSRC, src), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {src}:\n{r.stdout}\n{r.stderr}")
        if verbose or ptxas_info:
            sys.stderr.write(r.stdout + r.stderr)
        return obj

    def run(cmd: list, what: str) -> None:
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"{what} failed:\n{r.stdout}\n{r.stderr}")

    native_tmp = NATIVE + f".tmp{os.getpid()}"

    def compile_native() -> list:
        compile_, link = _native_commands(native_tmp)
        run(compile_, "compiling native.cpp")
        return link

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        native = ex.submit(compile_native)
        objs = list(ex.map(one, sources))
    if objs:
        tmp = LIB + f".tmp{os.getpid()}"
        run([nvcc] + ARCH + ["-shared", "-o", tmp] + objs + ["-cudart", "static", "-Xcompiler", "-fPIC",
                                                            "-Xlinker", "-soname=libb2pa.so"], "link")
        os.replace(tmp, LIB)
    run(native.result(), "linking native.o")
    os.replace(native_tmp, NATIVE)
    with open(key_file, "w") as f:
        f.write(_native_key())
    return LIB


if __name__ == "__main__":
    build(force="--force" in sys.argv, verbose=True, ptxas_info="--ptxas" in sys.argv)
    print(LIB)
