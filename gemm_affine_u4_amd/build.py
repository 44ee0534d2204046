"""Build libqmm.so (the C-ABI library) for gfx950 with hipcc, in-tree, and
libqmm_ceiling.so (the benchmark's measurement kernels: plain streaming read and
register-only MFMA loop).

    python -m gemm_affine_u4_amd.build        # or __graft_entry__.build()
"""
from __future__ import annotations

import os
import shutil
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OUT = os.path.join(PKG, "libqmm.so")
CEILING_OUT = os.path.join(PKG, "libqmm_ceiling.so")
BINDINGS = (("mix_binding.cpp", os.path.join(PKG, "_qmm_mix.so")), ("serve_binding.cpp", os.path.join(PKG, "_qmm_serve.so")))
BUILD_DIR = os.path.join(ROOT, "_build")

# (source, extra flags, object): the GEMV and GEMM sources are built once per code width.
WIDTHS = (2, 3, 4, 6, 8)
SOURCES = ([("qmm_api.cpp", [], "qmm_api.o"), ("qmm_validate.cpp", [], "qmm_validate.o"),
            ("moe_route.hip", [], "moe_route.o"), ("bmv_u4.hip", [], "bmv_u4.o"),
            ("qmm_noalloc.hip", [], "qmm_noalloc.o"), ("gemv_step.hip", [], "gemv_step.o"),
            ("moe_gemm.hip", [], "moe_gemm.o"), ("qmm_mix_api.cpp", [], "qmm_mix_api.o"),
            ("kv4_append.hip", [], "kv4_append.o"), ("kv4_decode.hip", [], "kv4_decode.o"),
            ("kv4_prefill.hip", [], "kv4_prefill.o"),
            ("gdn.hip", [], "gdn.o"),
            ("gdn_chunk.hip", [], "gdn_chunk.o"), ("qmm_serve_api.cpp", [], "qmm_serve_api.o"),
            ("kv8_append.hip", [], "kv8_append.o"), ("kv8_decode.hip", [], "kv8_decode.o"),
            ("kv8_prefill.hip", [], "kv8_prefill.o"),
            ("spec_verify.hip", [], "spec_verify.o"), ("lora.hip", [], "lora.o")]
           + [(src, [f"-DQMM_BITS={b}"], f"{src.split('.')[0]}_b{b}.o") for src in ("gemv_u4.hip", "gemm_u4.hip")
              for b in WIDTHS]
           + [(src, ["-DQMM_BITS=8", "-DQMM_FP8=1"], f"{src.split('.')[0]}_f8.o")
              for src in ("gemv_u4.hip", "gemm_u4.hip")])

ARCH = "gfx950"
HIPCC = os.environ.get("HIPCC", shutil.which("hipcc") or "/opt/rocm/bin/hipcc")
# Packed fp32 ops are kept out of the device code (compiler-generated v_pk_*_f32).
DEVICE_FLAGS = ["-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops"]
COMMON = ["-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}", "-I", INCLUDE, "-I", CSRC, "-Wall"]


def _compile(entry) -> str:
    src, extra, obj_name = entry
    obj = os.path.join(BUILD_DIR, obj_name)
    lang = ["-x", "hip"] if src.endswith(".hip") else []
    cmd = [HIPCC, *COMMON, *DEVICE_FLAGS, *extra, *lang, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    noise = "is not a recognized feature for this target"
    msgs = [ln for ln in (r.stderr or "").splitlines() if noise not in ln and ln.strip()]
    if msgs:
        sys.stderr.write("\n".join(msgs) + "\n")
    return obj


CEILING = ("ceiling.hip", [], "ceiling.o")


def _link(objs, out):
    tmp = out + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", *objs, "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)


def _compile_binding(src: str) -> str:
    """The Python side of the token mixers and of the serving step: host code against torch's headers."""
    import sysconfig

    import torch
    from torch.utils import cpp_extension

    obj = os.path.join(BUILD_DIR, src.replace(".cpp", ".o"))
    inc = [INCLUDE, sysconfig.get_paths()["include"], *cpp_extension.include_paths("cuda")]
    cmd = [HIPCC, "-O2", "-std=c++17", "-fPIC", "-x", "c++", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}", *sum((["-isystem", i] for i in inc), []),
           "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"compilation failed for {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def _link_binding(obj: str, out: str) -> None:
    import torch

    lib = os.path.join(os.path.dirname(torch.__file__), "lib")
    tmp = out + ".tmp"
    cmd = [HIPCC, "-shared", "-fPIC", obj, f"-L{lib}", "-lc10", "-lc10_hip", "-ltorch_cpu",
           "-ltorch_python", "-o", tmp]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)


def build(jobs: int = 8) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    with ThreadPoolExecutor(max_workers=jobs) as ex:
        bindings = [(ex.submit(_compile_binding, src), out) for src, out in BINDINGS]
        objs = list(ex.map(_compile, SOURCES + [CEILING]))
    _link(objs[:-1], OUT)
    _link(objs[-1:], CEILING_OUT)
    for obj, out in bindings:
        _link_binding(obj.result(), out)
    return OUT


if __name__ == "__main__":
    print(build())
