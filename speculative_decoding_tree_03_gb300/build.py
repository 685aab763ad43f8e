"""Build libspecverify.so (the C-ABI library) for sm_103a with nvcc.

Every .cu file under csrc/ compiles to an object in parallel; the objects link
into _build/libspecverify.so with the CUDA runtime linked statically, so the
library needs only the driver at run time and shares the process's primary
context (and therefore torch's streams). fastcall.cpp, the binding's checks of
its short calls, compiles beside them with g++ against torch's headers, into a
file named by what it was made from; without it (no headers, another compiler)
the binding makes the same checks itself.
"""

from __future__ import annotations

import concurrent.futures as cf
import contextlib
import glob
import hashlib
import os
import platform
import subprocess
import sys
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT = os.path.join(HERE, "_build")
LIB = os.path.join(OUT, "libspecverify.so")
SOURCES = ["mask.cu", "attn_simt.cu", "attn_tc.cu", "attn_sk.cu", "accept.cu", "accept_stream.cu",
           "accept_target_stream.cu",
           "accept_noalloc.cu", "accept_target.cu", "eagle2.cu",
           "kv_commit.cu", "lm_head.cu", "lora_proj.cu", "lora_shrink.cu", "pages.cu",
           "rope_kv.cu", "selftest.cu", "api.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc() -> str:
    cand = os.environ.get("CUDA_HOME", "/usr/local/cuda")
    path = os.path.join(cand, "bin", "nvcc")
    return path if os.path.exists(path) else "nvcc"


def _flags(verbose: bool):
    f = ARCH + ["-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE,
                "-I", CSRC, "--expt-relaxed-constexpr"]
    if verbose:
        f += ["-Xptxas", "-v"]
    return f


def _deps_mtime() -> float:
    paths = [os.path.join(CSRC, n) for n in os.listdir(CSRC)] + [os.path.join(INCLUDE, "specverify.h")]
    return max(os.path.getmtime(p) for p in paths)


def fastcall_path() -> str:
    """Where the compiled checks of the present sources, interpreter and torch are."""
    import torch

    h = hashlib.sha256("\0".join((torch.__version__, sys.implementation.cache_tag,
                                  platform.machine())).encode())
    for path in (os.path.join(CSRC, "fastcall.cpp"), os.path.join(INCLUDE, "specverify.h")):
        with open(path, "rb") as f:
            h.update(f.read())
    return os.path.join(OUT, f"_fastcall_{h.hexdigest()[:16]}.so")


def _build_fastcall(force: bool = False) -> None:
    why = ""
    try:
        import torch

        path = fastcall_path()
        if os.path.exists(path) and not force:
            return
        root = os.path.dirname(torch.__file__)
        inc = [INCLUDE, os.path.join(root, "include"),
               os.path.join(root, "include", "torch", "csrc", "api", "include"),
               sysconfig.get_paths()["include"],
               os.path.join(os.environ.get("CUDA_HOME", "/usr/local/cuda"), "include")]
        tmp = path + f".{os.getpid()}.tmp"
        cmd = (["g++", "-O2", "-std=c++17", "-shared", "-fPIC",
                f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}"]
               + [f"-I{p}" for p in inc] + [os.path.join(CSRC, "fastcall.cpp"), "-o", tmp,
                                            "-L" + os.path.join(root, "lib"), "-ltorch_python",
                                            "-ltorch_cpu", "-ltorch", "-lc10", "-lc10_cuda"])
        r = subprocess.run(cmd, capture_output=True, text=True)
        why = r.stderr or "g++ failed" if r.returncode != 0 else ""
    except (ImportError, AttributeError, OSError) as e:
        why = str(e)
    # modules of other sources are not kept, whether this one could be built or not
    for old in glob.glob(os.path.join(OUT, "_fastcall*.so")):
        with contextlib.suppress(FileNotFoundError):
            os.remove(old)
    if why:
        sys.stderr.write(f"fastcall.cpp was not built, its checks run in Python:\n{why[-2000:]}\n")
        return
    os.replace(tmp, path)


def build(force: bool = False, verbose: bool = False, jobs: int = 0) -> str:
    if not force and os.path.exists(LIB) and os.path.getmtime(LIB) >= _deps_mtime():
        _build_fastcall()
        return LIB
    os.makedirs(OUT, exist_ok=True)
    flags = _flags(verbose)

    def compile_one(name):
        obj = os.path.join(OUT, name.replace(".cu", ".o"))
        cmd = [nvcc()] + flags + ["-c", os.path.join(CSRC, name), "-o", obj]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed on {name}:\n{r.stderr}")
        return obj, r.stderr

    jobs = jobs or min(len(SOURCES), os.cpu_count() or 1)
    with cf.ThreadPoolExecutor(jobs + 1) as ex:
        fast = ex.submit(_build_fastcall, force)
        results = list(ex.map(compile_one, SOURCES))
        fast.result()
    if verbose:
        for _, err in results:
            sys.stderr.write(err)
    tmp = LIB + f".{os.getpid()}.tmp"
    cmd = [nvcc()] + ARCH + ["-shared", "-cudart=static", "-o", tmp] + [o for o, _ in results]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    return LIB


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
