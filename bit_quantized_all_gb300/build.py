"""Build libqr.so in-tree with nvcc for sm_103a (no GPU needed to compile).

Each translation unit under csrc/ compiles in parallel; the objects link into
``libqr.so`` next to this file with the CUDA runtime linked statically and
every symbol hidden except the ``qr_*`` entry points of include/qr.h.
csrc/qr_fast.cpp becomes the extension module ``_qr_fast`` beside it, the
compiled form of the calls in layer.py, where the interpreter's and torch's headers
are there; without them the library is built all the same, after a warning.
"""
from __future__ import annotations

import concurrent.futures as cf
import fcntl
import os
import shutil
import subprocess
import sys
import sysconfig
import warnings

import torch

HERE = os.path.dirname(os.path.abspath(__file__))
CSRC = os.path.join(HERE, "csrc")
OBJ_DIR = os.path.join(HERE, "_build")
LIB_PATH = os.path.join(HERE, "libqr.so")
# csrc/qr_fast.cpp, an extension module; it uses inline parts of torch's classes, so that
# one built for another torch or interpreter, which this name is not, must not be loaded
FAST_PATH = os.path.join(HERE, f"_qr_fast-torch{torch.__version__}.{sysconfig.get_config_var('SOABI')}.so")
FAST_FAILED = os.path.join(OBJ_DIR, os.path.basename(FAST_PATH) + ".failed")  # why it could not be built
INCLUDE = os.path.join(os.path.dirname(HERE), "include")

SOURCES = ["qr_capi.cu", "qr_grid.cu", "qr_encode.cu", "qr_decode.cu", "qr_reduce.cu", "qr_allreduce.cu",
           "qr_allreduce16_b3.cu", "qr_allreduce16_b4.cu", "qr_allreduce16_b6.cu", "qr_allreduce16_b8.cu",
           "qr_fc.cu", "qr_fc_allreduce_44.cu", "qr_fc_allreduce_48.cu", "qr_fc_allreduce_88.cu",
           "qr_twoshot.cu", "qr_twoshot_static.cu", "qr_twoshot_flags.cu", "qr_twoshot_peer.cu", "qr_timeouts.cu", "qr_fp4.cu",
           "qr_fc_twoshot.cu", "qr_fp4_twoshot.cu", "qr_codec_peer.cu",
           "qr_serving_capi.cu", "qr_kv_plan.cu", "qr_kv_append.cu", "qr_kv_attention.cu", "qr_kv_split_f16.cu",
           "qr_kv_split_bf16.cu", "qr_kv_tc.cu", "qr_w4.cu", "qr_w4_matvec.cu", "qr_w4_tc.cu",
           "qr_layer_capi.cu", "qr_norm_f16.cu", "qr_norm_bf16.cu", "qr_rope.cu", "qr_w8.cu", "qr_w8_few.cu",
           "qr_w8_tc.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]
NVCC_FLAGS = ARCH + [
    "-O3", "-lineinfo", "-std=c++17",
    # every rounding step is an explicit _rn intrinsic; keep nvcc from fusing the rest
    "-fmad=false",
    "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
    "-I", INCLUDE,
]


def _nvcc() -> str:
    for cand in (os.environ.get("NVCC"), shutil.which("nvcc"), "/usr/local/cuda/bin/nvcc"):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libqr.so")


def _deps() -> list[str]:
    files = [os.path.join(CSRC, f) for f in os.listdir(CSRC) if not f.endswith(".cpp")]
    files.append(os.path.join(INCLUDE, "qr.h"))
    files.append(os.path.abspath(__file__))
    return files


def _older(made: str, sources: list[str]) -> bool:
    if not os.path.exists(made):
        return True
    t = os.path.getmtime(made)
    return any(os.path.getmtime(f) > t for f in sources)


def _stale() -> bool:
    return _older(LIB_PATH, _deps())


def _fast_stale() -> bool:
    """Whether the extension module is to be built: not where it is up to date, nor
    where it could not be built from these sources (which build(force=True) tries again)."""
    sources = [os.path.join(CSRC, "qr_fast.cpp"), os.path.join(INCLUDE, "qr.h"), os.path.abspath(__file__)]
    return _older(FAST_PATH, sources) and _older(FAST_FAILED, sources)


def _try_fast() -> None:
    """The extension module where it can be built; the calls in layer.py run without
    it too, so what is missing for it (the interpreter's headers, say) stops nothing else."""
    try:
        _build_fast()
    except (RuntimeError, OSError) as e:
        if os.path.exists(FAST_PATH):  # of other sources
            os.remove(FAST_PATH)
        with open(FAST_FAILED, "w") as f:
            f.write(f"{e}\n")
        warnings.warn(f"{os.path.basename(FAST_PATH)} could not be built: the calls of layer.py run without it ({e})",
                      RuntimeWarning, stacklevel=2)
    else:
        if os.path.exists(FAST_FAILED):
            os.remove(FAST_FAILED)


def _build_fast() -> None:
    """The extension module, against the running interpreter's and torch's headers."""
    root = os.path.dirname(torch.__file__)
    includes = [sysconfig.get_paths()["include"], os.path.join(root, "include"),
                os.path.join(root, "include", "torch", "csrc", "api", "include"),
                os.path.join(os.path.dirname(os.path.dirname(_nvcc())), "include")]
    tmp = FAST_PATH + f".tmp{os.getpid()}"
    cmd = ["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *(f"-I{i}" for i in includes),
           os.path.join(CSRC, "qr_fast.cpp"), "-o", tmp, "-L" + os.path.join(root, "lib"), "-ltorch_python", "-ltorch",
           "-ltorch_cpu", "-lc10", "-lc10_cuda"]
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError(f"g++ failed on qr_fast.cpp:\n{' '.join(cmd)}\n{p.stdout}\n{p.stderr}")
    os.replace(tmp, FAST_PATH)


def build(force: bool = False, verbose: bool = False, ptxas_info: bool = False) -> str:
    """Compile csrc/*.cu into libqr.so (skipped when up to date).  Processes
    that build at the same time (the ranks of one job, parallel test
    workers) take turns on a lock file, and each re-checks whether the
    library is still stale once it holds the lock, so the objects are never
    written by two compilers at once."""
    if not force and not ptxas_info and not _stale() and not _fast_stale():
        return LIB_PATH
    os.makedirs(OBJ_DIR, exist_ok=True)
    with open(os.path.join(OBJ_DIR, ".lock"), "w") as lock:
        fcntl.flock(lock, fcntl.LOCK_EX)
        try:
            with cf.ThreadPoolExecutor(max_workers=1) as ex:
                fast = ex.submit(_try_fast) if force or _fast_stale() else None
                if force or ptxas_info or _stale():
                    _build_locked(verbose, ptxas_info)
                if fast is not None:
                    fast.result()
            return LIB_PATH
        finally:
            fcntl.flock(lock, fcntl.LOCK_UN)


def _build_locked(verbose: bool, ptxas_info: bool) -> None:
    nvcc = _nvcc()
    extra = ["-Xptxas", "-v"] if ptxas_info else []

    def compile_one(src: str) -> tuple[str, str]:
        obj = os.path.join(OBJ_DIR, src.replace(".cu", ".o"))
        cmd = [nvcc, *NVCC_FLAGS, *extra, "-c", os.path.join(CSRC, src), "-o", obj]
        p = subprocess.run(cmd, capture_output=True, text=True)
        if p.returncode != 0:
            raise RuntimeError(f"nvcc failed on {src}:\n{' '.join(cmd)}\n{p.stdout}\n{p.stderr}")
        return obj, p.stdout + p.stderr

    with cf.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        results = list(ex.map(compile_one, SOURCES))
    if verbose or ptxas_info:
        for _, log in results:
            if log.strip():
                sys.stderr.write(log)
    tmp = LIB_PATH + f".tmp{os.getpid()}"
    cmd = [nvcc, *ARCH, "-shared", "-Xcompiler", "-fPIC", "-o", tmp] + [o for o, _ in results]
    p = subprocess.run(cmd, capture_output=True, text=True)
    if p.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{p.stdout}\n{p.stderr}")
    os.replace(tmp, LIB_PATH)


if __name__ == "__main__":
    build(force=True, verbose=True, ptxas_info="--ptxas" in sys.argv)
    print(LIB_PATH)
