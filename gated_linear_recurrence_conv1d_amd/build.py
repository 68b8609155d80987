"""Builds librglru.so in-tree with hipcc for gfx950 (cross-compiles without a GPU), and the binding's
module _rglru_torch.so with the host compiler."""
from __future__ import annotations

import os
import subprocess
import sys
import sysconfig

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
LIB = os.path.join(PKG, "librglru.so")
EXT = os.path.join(PKG, "_rglru_torch.so")
SOURCES = ["rglru_api.cpp", "rglru_gates.hip", "rglru_scan.hip", "rglru_decode.hip",
           "rglru_fused.hip", "rglru_backward.hip", "rglru_bwd_tiles.hip", "rglru_bwd_fused.hip",
           "rglru_mqa.hip", "rglru_noalloc.hip", "rglru_attn_api.cpp", "rglru_rope.hip",
           "rglru_paged.hip", "rglru_mqa_bwd.hip", "rglru_attn.hip"]
EXT_SOURCE = "rglru_torch.cpp"
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
CXX = os.environ.get("CXX", "g++")

FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-shared", "-Wall",
    # no packed fp32 (v_pk_*_f32) in generated device code
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    # keep single-lane atomics (work tickets) as plain atomics: the wave-aggregating rewrite
    # consumes the returned value right after the atomic, which would stall on its round trip
    "-mllvm", "-amdgpu-atomic-optimizer-strategy=None",
    "-I" + os.path.join(ROOT, "include"), "-I" + CSRC,
]


def _compile(compiler, args, target, verbose):
    tmp = target + ".tmp"
    cmd = [compiler] + args + ["-o", tmp]
    if verbose:
        print(" ".join(cmd), flush=True)
    res = subprocess.run(cmd, capture_output=True, text=True)
    out = "\n".join(l for l in (res.stdout + res.stderr).splitlines()
                    if "packed-fp32-ops' is not a recognized feature" not in l)
    if res.returncode != 0:
        raise RuntimeError(f"{compiler} failed:\n" + out)
    if verbose and out.strip():
        print(out, flush=True)
    os.replace(tmp, target)


def build_ext(verbose: bool = False) -> str:
    """The binding's module, against this interpreter's torch and the librglru.so beside it."""
    import torch

    base = os.path.dirname(torch.__file__)
    args = ["-O2", "-std=c++17", "-fPIC", "-shared", "-Wall",
            f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
            "-I" + os.path.join(ROOT, "include"),
            "-isystem", sysconfig.get_paths()["include"],
            "-isystem", os.path.join(base, "include"),
            "-isystem", os.path.join(base, "include", "torch", "csrc", "api", "include"),
            os.path.join(CSRC, EXT_SOURCE),
            "-L" + PKG, "-l:" + os.path.basename(LIB), "-Wl,-rpath,$ORIGIN",
            "-L" + os.path.join(base, "lib"), "-lc10", "-ltorch_cpu", "-ltorch_python"]
    _compile(CXX, args, EXT, verbose)
    return EXT


def build(verbose: bool = False) -> str:
    _compile(HIPCC, FLAGS + [os.path.join(CSRC, s) for s in SOURCES], LIB, verbose)
    build_ext(verbose)
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
