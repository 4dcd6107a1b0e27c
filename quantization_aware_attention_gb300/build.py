"""Builds the in-tree C-ABI library ``libqat_attn.so`` for sm_103a with nvcc, and the torch extension
``_qat_torch`` (host code over that library) with the host compiler.

Translation units are compiled in parallel, then linked with ``nvcc -shared``; the CUDA
runtime is linked statically.  An object is rebuilt when its source or any header of
the library is newer than it.
"""

from __future__ import annotations

import concurrent.futures
import glob
import hashlib
import importlib.util
import os
import shutil
import subprocess
import sysconfig

HERE = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(HERE)
CSRC = os.path.join(HERE, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJDIR = os.path.join(HERE, "_build_tmp")
LIB_PATH = os.path.join(HERE, "libqat_attn.so")
EXT_PATH = os.path.join(HERE, "_qat_torch.so")
EXT_SOURCE = "torch_ops.cpp"

SOURCES = ["qat_api.cu", "attn_fwd_sm100.cu", "attn_bwd_sm100.cu", "attn_bwd_dq_sm100.cu",
           "quant_debug.cu", "qat_noalloc.cu", "qkv_quant.cu", "attn_merge.cu", "debug_wait.cu",
           "qk_norm_rope.cu", "kv_cache.cu", "attn_decode.cu"]
GENCODE = "-gencode=arch=compute_103a,code=sm_103a"
NVCC_FLAGS = [GENCODE, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC",
              "-Xcompiler", "-fvisibility=hidden", "--expt-relaxed-constexpr",
              "-I", INCLUDE, "-I", CSRC]


def _nvcc() -> str:
    path = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(path):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libqat_attn.so")
    return path


def _headers_mtime() -> float:
    hdrs = glob.glob(os.path.join(CSRC, "*.cuh")) + glob.glob(os.path.join(CSRC, "*.h"))
    hdrs += glob.glob(os.path.join(INCLUDE, "*.h"))
    return max((os.path.getmtime(h) for h in hdrs), default=0.0)


def _compile(src: str, extra: list[str], verbose: bool) -> str:
    obj = os.path.join(OBJDIR, os.path.splitext(src)[0] + ".o")
    srcp = os.path.join(CSRC, src)
    if (os.path.exists(obj) and os.path.getmtime(obj) >= os.path.getmtime(srcp)
            and os.path.getmtime(obj) >= _headers_mtime()):
        return obj
    cmd = [_nvcc(), "-c", srcp, "-o", obj] + NVCC_FLAGS + extra
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"nvcc failed on {src}:\n{r.stdout}\n{r.stderr}")
    if verbose and (r.stdout or r.stderr):
        print(r.stdout + r.stderr, flush=True)
    return obj


def _ext_key() -> str:
    """What the extension is compiled and linked against: torch's version and place, and the interpreter."""
    import torch

    where = os.path.dirname(torch.__file__) + sysconfig.get_paths()["include"]
    return (f"{torch.__version__}-{sysconfig.get_config_var('SOABI')}-"
            f"{hashlib.sha256(where.encode()).hexdigest()[:12]}")


def _compile_ext(verbose: bool) -> str:
    """The torch extension's object, compiled against the installed torch's headers."""
    import torch

    obj = os.path.join(OBJDIR, f"torch_ops-{_ext_key()}.o")
    src = os.path.join(CSRC, EXT_SOURCE)
    newest = max(os.path.getmtime(src), os.path.getmtime(os.path.join(INCLUDE, "qat_attn.h")))
    if os.path.exists(obj) and os.path.getmtime(obj) >= newest:
        return obj
    base = os.path.join(os.path.dirname(torch.__file__), "include")
    cuda = os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")
    cmd = [shutil.which("g++") or "c++", "-c", src, "-o", obj, "-O2", "-std=c++17", "-fPIC",
           "-fvisibility=hidden", f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE]
    for path in (base, os.path.join(base, "torch", "csrc", "api", "include"),
                 sysconfig.get_paths()["include"], cuda):
        cmd += ["-isystem", path]
    _run(cmd, EXT_SOURCE, verbose)
    return obj


def _link_ext(obj: str, verbose: bool) -> None:
    import torch

    # the object that the extension was linked from: another torch's is newer or older as it happens
    stamp = os.path.join(OBJDIR, "_qat_torch.linked")
    linked = ""
    if os.path.exists(stamp):
        with open(stamp) as f:
            linked = f.read()
    if (linked == os.path.basename(obj) and os.path.exists(EXT_PATH)
            and os.path.getmtime(EXT_PATH) >= os.path.getmtime(obj)):
        return
    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = EXT_PATH + ".tmp"
    _run([shutil.which("g++") or "c++", "-shared", obj, "-o", tmp, "-L", HERE, "-l:libqat_attn.so",
          "-L", lib, "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_cuda", "-ltorch", "-ltorch_python",
          "-Wl,-rpath,$ORIGIN", f"-Wl,-rpath,{lib}"], "_qat_torch", verbose)
    if os.path.exists(stamp):
        os.remove(stamp)
    os.replace(tmp, EXT_PATH)
    with open(stamp, "w") as f:
        f.write(os.path.basename(obj))


def _run(cmd: list[str], what: str, verbose: bool) -> None:
    if verbose:
        print(" ".join(cmd), flush=True)
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"building {what} failed:\n{r.stdout}\n{r.stderr}")


def build(verbose: bool = False, ptxas_verbose: bool = False) -> str:
    """Compile every source and link ``libqat_attn.so``, then the torch extension, for which torch must be
    installed (without it the library is built alone); returns the library's path."""
    os.makedirs(OBJDIR, exist_ok=True)
    extra = ["-Xptxas", "-v"] if ptxas_verbose else []
    workers = min(len(SOURCES) + 1, os.cpu_count() or 1)
    with concurrent.futures.ThreadPoolExecutor(max_workers=workers) as ex:
        ext = None
        if importlib.util.find_spec("torch") is not None:
            ext = ex.submit(_compile_ext, verbose or ptxas_verbose)
        objs = list(ex.map(lambda s: _compile(s, extra, verbose or ptxas_verbose), SOURCES))
    newest = max(os.path.getmtime(o) for o in objs)
    if not os.path.exists(LIB_PATH) or os.path.getmtime(LIB_PATH) < newest:
        tmp = LIB_PATH + ".tmp"
        cmd = [_nvcc(), "-shared", GENCODE, "-o", tmp] + objs + ["-cudart", "static"]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB_PATH)
    if ext is not None:  # the library stands by itself, whatever becomes of the extension
        _link_ext(ext.result(), verbose or ptxas_verbose)
    return LIB_PATH


if __name__ == "__main__":
    import sys
    print(build(verbose=True, ptxas_verbose="-v" in sys.argv))
