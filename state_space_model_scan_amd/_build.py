"""Builds libssmscan.so in-tree with hipcc for gfx950 (MI355X).

Every HIP source is compiled with the packed-FP32 feature switched off
(``-Xclang -target-feature -Xclang -packed-fp32-ops``): hipcc then emits only
scalar fp32 VALU instructions.  hipcc's host pass warns that it does not know
the feature; that warning is harmless.  ``-mllvm -amdgpu-mfma-vgpr-form``
keeps matrix-core results in ordinary VGPRs, so the VALU reads them without
an accumulator-register copy.
"""
from __future__ import annotations

import os
import subprocess
import sys
from concurrent.futures import ThreadPoolExecutor

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
LIB = os.path.join(PKG, "libssmscan.so")
# instruction-rate and bandwidth probes (bench.py --microbench), a library of
# their own so that the operator's ABI holds only the operator
MICRO_LIB = os.path.join(PKG, "libssmmicro.so")
BUILD_DIR = os.path.join(PKG, "_build")

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"
COMMON = ["-O3", "-std=c++17", "-fPIC", f"-I{INCLUDE}", "-Wall"]
HIP_FLAGS = [f"--offload-arch={ARCH}", "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
             "-mllvm", "-amdgpu-mfma-vgpr-form", "-fno-gpu-rdc"]

SOURCES = [
    ("scan_bf16.hip", True),
    ("scan_f32.hip", True),
    ("scan_f16.hip", True),
    ("scan_bf16_ew.hip", True),
    ("scan_f32_ew.hip", True),
    ("scan_f16_ew.hip", True),
    ("ssm_scan.hip", True),
    ("scan_complex.hip", True),
    ("decode.hip", True),
    ("ssd.hip", True),
    ("ssd_varlen.hip", True),
    ("ssd_varlen_bwd.hip", True),
    ("conv_varlen.hip", True),
    ("step.hip", True),
    ("bwd.hip", True),
    ("bwd_complex.hip", True),
    ("validate.cpp", False),
]
MICRO_SOURCES = [("microbench.hip", True)]
# the torch binding of the packed-token operators: host code only, linked
# against the operators' library beside it
PACKED_SOURCE = "packed_binding.cpp"
PACKED_LIB = os.path.join(PKG, "_packed.so")


def _compile(src: str, is_hip: bool) -> str:
    os.makedirs(BUILD_DIR, exist_ok=True)
    obj = os.path.join(BUILD_DIR, os.path.basename(src) + ".o")
    cmd = [HIPCC] + COMMON + (HIP_FLAGS if is_hip else ["-x", "c++"]) + ["-c", os.path.join(CSRC, src), "-o", obj]
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"hipcc failed on {src}")
    return obj


def _link(objs, lib):
    tmp = lib + ".tmp"
    cmd = [HIPCC, "-shared", "-fPIC", f"--offload-arch={ARCH}", "-o", tmp] + objs
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"linking {os.path.basename(lib)} failed")
    os.replace(tmp, lib)


def _build_packed() -> None:
    import sysconfig
    import torch
    base = os.path.dirname(torch.__file__)
    lib_dir = os.path.join(base, "lib")
    include = [os.path.join(base, "include"), os.path.join(base, "include", "torch", "csrc", "api", "include"),
               "/opt/rocm/include", sysconfig.get_paths()["include"]]
    tmp = PACKED_LIB + ".tmp"
    cmd = (["g++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__=1", "-DUSE_ROCM=1", f"-I{INCLUDE}"]
           + [f"-isystem{d}" for d in include] + [os.path.join(CSRC, PACKED_SOURCE), "-o", tmp, f"-L{PKG}", "-l:libssmscan.so",
              "-Wl,-rpath,$ORIGIN", f"-L{lib_dir}", "-lc10", "-lc10_hip", "-ltorch_cpu", "-ltorch_python"])
    res = subprocess.run(cmd, capture_output=True, text=True)
    if res.returncode != 0:
        sys.stderr.write(res.stdout + res.stderr)
        raise RuntimeError(f"building {os.path.basename(PACKED_LIB)} failed")
    os.replace(tmp, PACKED_LIB)


def build(verbose: bool = False) -> str:
    """Compile every source and link libssmscan.so, libssmmicro.so and
    _packed.so (always rebuilds)."""
    srcs = SOURCES + MICRO_SOURCES
    with ThreadPoolExecutor(max_workers=len(srcs)) as ex:
        objs = list(ex.map(lambda s: _compile(*s), srcs))
    _link(objs[:len(SOURCES)], LIB)
    _link(objs[len(SOURCES):], MICRO_LIB)
    _build_packed()
    if verbose:
        print(f"built {LIB}, {MICRO_LIB} and {PACKED_LIB}")
    return LIB


if __name__ == "__main__":
    build(verbose=True)
