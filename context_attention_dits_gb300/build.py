"""Builds libcpattn.so in-tree with nvcc for sm_103a (no cmake; it needs no torch).

    python -m context_attention_dits_gb300.build [--verbose-ptxas]

Translation units compile in parallel; the shared library links the CUDA
runtime statically and fetches the one driver entry point it needs
(cuTensorMapEncodeTiled) at run time, so it loads on machines without a GPU
driver. Beside it _cpbind-*.so (bind.cpp, by the host compiler against torch's
headers) marshals the tensors of the calls whose host time counts. It is bound to
one Python and one torch, which its name says, and left out where there is no torch
for CUDA; libcpattn.so is in place before anything of it can fail.
"""
from __future__ import annotations

import argparse
import concurrent.futures as cf
import os
import shutil
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIBDIR = os.path.join(PKG, "lib")
LIB = os.path.join(LIBDIR, "libcpattn.so")
SOURCES = ["attn_tc.cu", "attn_bwd.cu", "attn_bwd_tc.cu", "kernels_simt.cu", "score_fwd_tc.cu", "score_bwd_tc.cu",
           "score_attn_f32.cu", "paged.cu", "paged_q4.cu", "rope.cu", "cp_score_api.cu", "cp_rope_api.cu", "cp_q4_api.cu", "cp_api.cu"]
ARCH = ["-gencode", "arch=compute_103a,code=sm_103a"]


def nvcc_path() -> str:
    for cand in (os.environ.get("CUDA_HOME"), os.environ.get("CUDA_PATH"), "/usr/local/cuda"):
        if cand and os.path.exists(os.path.join(cand, "bin", "nvcc")):
            return os.path.join(cand, "bin", "nvcc")
    found = shutil.which("nvcc")
    if not found:
        raise RuntimeError("nvcc not found (set CUDA_HOME)")
    return found


def _torch():
    """torch, or None where there is none that works."""
    try:
        import torch
    except (ImportError, OSError):
        return None
    return torch


def bind_path():
    """_cpbind-*.so of this Python and this torch; None without a torch for CUDA."""
    torch = _torch()
    if torch is None or torch.version.cuda is None:
        return None
    return os.path.join(LIBDIR, f"_cpbind-{torch.__version__}.{sysconfig.get_config_var('SOABI')}.so")


def _bind_command(to):
    torch = _torch()
    at, cuda = os.path.dirname(torch.__file__), os.path.dirname(os.path.dirname(nvcc_path()))
    return [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}", "-I", INCLUDE, "-I", os.path.join(at, "include"),
            "-I", os.path.join(at, "include", "torch", "csrc", "api", "include"), "-I", sysconfig.get_paths()["include"],
            "-I", os.path.join(cuda, "include"), os.path.join(CSRC, "bind.cpp"), "-o", to, "-L", os.path.join(at, "lib"),
            "-lc10", "-lc10_cuda", "-ltorch_cpu", "-ltorch_python"]


def _run(cmd):
    p = subprocess.run(cmd, stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True)
    return p.returncode, p.stdout


def build(verbose_ptxas: bool = False, force: bool = False) -> str:
    nvcc = nvcc_path()
    build_dir = os.path.join(PKG, "_build")
    os.makedirs(build_dir, exist_ok=True)
    os.makedirs(LIBDIR, exist_ok=True)
    deps = [os.path.join(CSRC, f) for f in os.listdir(CSRC)] + [os.path.join(INCLUDE, "cp_attn.h")]
    newest = max(os.path.getmtime(d) for d in deps)
    bind = bind_path()

    def stale(path):
        return force or not os.path.exists(path) or os.path.getmtime(path) < newest

    need_lib, need_bind = stale(LIB) or verbose_ptxas, bind is not None and stale(bind)
    common = [nvcc, *ARCH, "-O3", "-lineinfo", "-std=c++17", "-Xcompiler", "-fPIC", "-I", INCLUDE, "-I", CSRC,
              "--expt-relaxed-constexpr"]
    if verbose_ptxas:
        common += ["-Xptxas", "-v"]
    objs = [os.path.join(build_dir, os.path.splitext(src)[0] + ".o") for src in SOURCES]
    with cf.ThreadPoolExecutor(max_workers=len(SOURCES) + 1) as ex:
        bound = ex.submit(_run, _bind_command(bind + ".tmp")) if need_bind else None
        if need_lib:
            results = list(ex.map(_run, (common + ["-c", os.path.join(CSRC, src), "-o", obj] for src, obj in zip(SOURCES, objs))))
            log = "\n".join(out for _, out in results)
            if any(rc != 0 for rc, _ in results):
                raise RuntimeError("nvcc failed:\n" + log)
            if verbose_ptxas:
                print(log)
            tmp = LIB + ".tmp"
            rc, out = _run([nvcc, *ARCH, "-shared", "-o", tmp, *objs, "-cudart", "static"])
            if rc != 0:
                raise RuntimeError("link failed:\n" + out)
            os.replace(tmp, LIB)
    if bound is not None:
        rc, out = bound.result()
        if rc != 0:
            raise RuntimeError(f"{LIB} is built, but not {os.path.basename(bind)}, by which torch calls a part of it:\n" + out)
        os.replace(bind + ".tmp", bind)
    return LIB


def main(argv=None):
    ap = argparse.ArgumentParser()
    ap.add_argument("--verbose-ptxas", action="store_true")
    ap.add_argument("--force", action="store_true")
    args = ap.parse_args(argv)
    print(build(verbose_ptxas=args.verbose_ptxas, force=args.force))


if __name__ == "__main__":
    sys.exit(main())
