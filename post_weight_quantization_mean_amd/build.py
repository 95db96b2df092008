"""Builds libawq.so (all HIP kernels + the C-ABI host code) in-tree for gfx950 with hipcc, and _a8.so (the
native Python binding of the 8-bit activation calls: host code, no kernels) with g++.

Usage: python -m post_weight_quantization_mean_amd.build   (or __graft_entry__.build()).
"""
from __future__ import annotations

import concurrent.futures
import os
import shutil
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libawq.so")
BINDING = os.path.join(PKG, "_a8.so")

SOURCES = ["stats.hip", "scales.hip", "search.hip", "gram.hip", "pack.hip", "clip.hip", "fold.hip", "w4a16.hip",
           "rows8.hip", "w4a8.hip", "moe.hip", "lora.hip", "awq_api.cpp", "a8_api.cpp", "moe_api.cpp", "lora_api.cpp"]

# -ffp-contract=off: every fp32 operation of the quantizer contract is rounded on its own
#   (fused multiply-adds are written explicitly where the search wants them).
# packed-fp32-ops disabled: hipcc would otherwise emit v_pk_{add,mul,fma}_f32 on its own.
HIP_FLAGS = [
    "--offload-arch=gfx950", "-O3", "-std=c++17", "-fPIC", "-fvisibility=hidden",
    "-ffp-contract=off", "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-I" + INCLUDE, "-I" + CSRC,
]


def hipcc() -> str:
    for cand in (os.environ.get("HIPCC"), "/opt/rocm/bin/hipcc", shutil.which("hipcc")):
        if cand and os.path.exists(cand):
            return cand
    raise RuntimeError("hipcc not found: the HIP toolchain is required to build libawq")


def build_binding() -> None:
    """Compile _a8.so against this interpreter and torch."""
    import sysconfig

    import torch
    root = os.path.join(os.path.dirname(torch.__file__))
    tmp = BINDING + ".tmp"
    cmd = [os.environ.get("CXX") or "g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-fvisibility=hidden",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", "-I" + INCLUDE,
           "-I" + os.path.join(root, "include"), "-I" + os.path.join(root, "include", "torch", "csrc", "api", "include"),
           "-I" + sysconfig.get_paths()["include"], os.path.join(CSRC, "a8_binding.cpp"), "-o", tmp,
           "-L" + os.path.join(root, "lib"), "-lc10", "-ltorch_cpu", "-ltorch_python"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"g++ failed on a8_binding.cpp:\n{r.stderr}")
    os.replace(tmp, BINDING)


def build(verbose: bool = False) -> str:
    """Compile every source, link libawq.so and build _a8.so; always rebuilds.  Returns the library path."""
    cc = hipcc()
    objdir = os.path.join(PKG, "_build")
    os.makedirs(objdir, exist_ok=True)

    def compile_one(src: str) -> str:
        obj = os.path.join(objdir, src + ".o")
        lang = ["-x", "hip"] if src.endswith(".cpp") else []
        cmd = [cc, *HIP_FLAGS, *lang, "-c", os.path.join(CSRC, src), "-o", obj]
        if verbose:
            print(" ".join(cmd), flush=True)
        r = subprocess.run(cmd, capture_output=True, text=True)
        err = "\n".join(l for l in r.stderr.splitlines() if "not a recognized feature" not in l)
        if r.returncode != 0:
            raise RuntimeError(f"hipcc failed on {src}:\n{err}")
        if verbose and err.strip():
            print(err, file=sys.stderr)
        return obj

    with concurrent.futures.ThreadPoolExecutor(max_workers=4) as pool:
        binding = pool.submit(build_binding)
        objs = list(pool.map(compile_one, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [cc, "--offload-arch=gfx950", "-shared", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{r.stderr}")
    os.replace(tmp, LIB)
    binding.result()  # its failure is raised behind the library, which needs no binding
    return LIB


if __name__ == "__main__":
    print(build(verbose="-v" in sys.argv))
