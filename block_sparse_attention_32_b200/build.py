"""Build ``libmsa.so`` (the C-ABI library of the MSA hot path) and ``msa_calls.so``
(Python calls of the operators around the path) in-tree.

Every CUDA source under ``csrc/`` is compiled for sm_100a only
(``-gencode arch=compute_100a,code=sm_100a``) and linked into
``block_sparse_attention_32_b200/lib/libmsa.so``; ``csrc/calls.cpp`` is compiled
against torch's headers and linked to it.  Run
``python -m block_sparse_attention_32_b200.build`` (or call ``build()``).
"""
from __future__ import annotations

import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
OUT_DIR = os.path.join(PKG, "lib")
LIB = os.path.join(OUT_DIR, "libmsa.so")
CALLS = os.path.join(OUT_DIR, "msa_calls.so")
OBJ_DIR = os.path.join(ROOT, "_build", "msa")
CALLS_TAG = os.path.join(OBJ_DIR, "msa_calls.built_for")

SOURCES = ["msa_api.cu", "index_score.cu", "topk.cu", "block_lists.cu", "block_lists_noalloc.cu",
           "sparse_attn.cu", "sparse_attn_decode.cu", "merge.cu", "recall.cu",
           "token_select.cu", "sparse_attn_bwd.cu", "norm_rope.cu", "paged_decode.cu",
           "window_attn.cu", "window_attn_bwd.cu"]
HEADERS = ["common.cuh", "layer_args.cuh", "window_tiles.cuh"]

NVCC_FLAGS = ["-gencode", "arch=compute_100a,code=sm_100a", "-O3", "-lineinfo", "-std=c++17",
              "-Xcompiler", "-fPIC", "-Xcompiler", "-fvisibility=hidden",
              "--expt-relaxed-constexpr", "-Xptxas", "-v"]


def _nvcc() -> str:
    cand = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(cand):
        raise RuntimeError("nvcc not found: the CUDA toolkit is required to build libmsa.so")
    return cand


def _stale(target: str, deps) -> bool:
    if not os.path.exists(target):
        return True
    t = os.path.getmtime(target)
    return any(os.path.getmtime(d) > t for d in deps)


def build(force: bool = False, verbose: bool = False) -> str:
    """Compile (if needed) and return the path of libmsa.so."""
    os.makedirs(OUT_DIR, exist_ok=True)
    os.makedirs(OBJ_DIR, exist_ok=True)
    nvcc = _nvcc()
    inc = os.path.join(ROOT, "include")
    hdrs = [os.path.join(CSRC, h) for h in HEADERS] + [os.path.join(inc, "msa.h")]
    jobs = []
    objs = []
    for src in SOURCES:
        s = os.path.join(CSRC, src)
        o = os.path.join(OBJ_DIR, src + ".o")
        objs.append(o)
        if force or _stale(o, [s] + hdrs):
            jobs.append((s, o))

    def compile_one(so):
        s, o = so
        cmd = [nvcc, *NVCC_FLAGS, "-I", inc, "-c", s, "-o", o]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"nvcc failed for {s}:\n{r.stdout}\n{r.stderr}")
        return s, r.stderr

    if jobs:
        with cf.ThreadPoolExecutor(max_workers=min(len(jobs), os.cpu_count() or 4)) as ex:
            for s, log in ex.map(compile_one, jobs):
                if verbose:
                    print(f"== {os.path.basename(s)}\n{log}", file=sys.stderr)
    if force or jobs or _stale(LIB, objs):
        tmp = LIB + f".tmp{os.getpid()}"
        cmd = [nvcc, "-shared", "-gencode", "arch=compute_100a,code=sm_100a", "-o", tmp, *objs]
        r = subprocess.run(cmd, capture_output=True, text=True)
        if r.returncode != 0:
            raise RuntimeError(f"link failed:\n{r.stdout}\n{r.stderr}")
        os.replace(tmp, LIB)
    build_calls(force)
    return LIB


def _calls_for() -> str:
    """What msa_calls.so is bound to: torch's C++ interface and Python's."""
    import torch
    return f"torch {torch.__version__} {sysconfig.get_config_var('SOABI')}"


def calls_stale() -> bool:
    """msa_calls.so is missing, older than its sources, or built for another torch or Python."""
    if _stale(CALLS, [os.path.join(CSRC, "calls.cpp"), os.path.join(ROOT, "include", "msa.h")]):
        return True
    try:
        with open(CALLS_TAG) as f:
            return f.read() != _calls_for()
    except OSError:
        return True


def build_calls(force: bool = False) -> str:
    """Compile (if needed) and return the path of msa_calls.so."""
    if not force and not calls_stale():
        return CALLS
    import torch
    src = os.path.join(CSRC, "calls.cpp")
    troot = os.path.dirname(torch.__file__)
    cuda = os.path.dirname(os.path.dirname(os.path.realpath(_nvcc())))
    tmp = CALLS + f".tmp{os.getpid()}"
    cmd = [shutil.which("g++") or "g++", "-O2", "-std=c++17", "-shared", "-fPIC",
           "-fvisibility=hidden",
           f'-DMSA_TORCH_VERSION="{torch.__version__}"',
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-isystem", os.path.join(troot, "include"),
           "-isystem", os.path.join(troot, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"],
           "-isystem", os.path.join(cuda, "include"), src, "-o", tmp,
           "-L", OUT_DIR, "-l:libmsa.so", "-L", os.path.join(troot, "lib"), "-lc10", "-lc10_cuda",
           "-ltorch_cpu", "-ltorch", "-ltorch_python", "-Wl,-rpath,$ORIGIN"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed for {src}:\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, CALLS)
    os.makedirs(OBJ_DIR, exist_ok=True)
    with open(CALLS_TAG, "w") as f:
        f.write(_calls_for())
    return CALLS


if __name__ == "__main__":
    print(build(force="--force" in sys.argv, verbose="-v" in sys.argv))
