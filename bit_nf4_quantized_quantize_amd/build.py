"""Build libqlora_nf4.so (HIP kernels + C ABI) for gfx950 with hipcc, and
_decoder.so and _kvcache.so, the Python modules of decoder.py and kvcache.py
(host code, against torch's headers).

Usage: python -m bit_nf4_quantized_quantize_amd.build
All are written next to this file; objects go to _build/.
"""

import concurrent.futures
import os
import subprocess
import sys

PKG = os.path.dirname(os.path.abspath(__file__))
ROOT = os.path.dirname(PKG)
CSRC = os.path.join(PKG, "csrc")
INCLUDE = os.path.join(ROOT, "include")
OBJDIR = os.path.join(PKG, "_build")
LIB = os.path.join(PKG, "libqlora_nf4.so")
BINDING = os.path.join(PKG, "_decoder.so")  # the CPython module of decoder.py
KV_BINDING = os.path.join(PKG, "_kvcache.so")  # that of kvcache.py

SOURCES = ["quantize.hip", "linear.hip", "optim.hip", "dropout.hip", "noalloc.hip", "probe.hip", "norm.hip", "rope.hip", "paged.hip",
           "kv_write.hip", "kv_attention.hip", "kv_prefix.hip", "host.cpp", "abi.cpp", "decoder_abi.cpp", "kv_abi.cpp"]
HEADERS = ["device.h", "launch.h", "codebooks.h", "decoder.h", "rotary.h", "paged_device.h", "kvcache.h",
           "kv_codes.h", "abi_checks.h"]
# csrc/decoder_binding.cpp and kv_binding.cpp are modules of their own, see _build_module

HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")
ARCH = "gfx950"

# -ffp-contract=off and correctly rounded fp32 division: stored codes and
# constants are decided by fp32 arithmetic with one rounding per operation.
# Denormals are kept.  Packed-fp32 instructions are disabled.
CFLAGS = [
    "-O3", "-std=c++17", "-fPIC", f"--offload-arch={ARCH}",
    "-ffp-contract=off",
    "-fhip-fp32-correctly-rounded-divide-sqrt",
    "-fno-gpu-flush-denormals-to-zero",
    "-Xclang", "-target-feature", "-Xclang", "-packed-fp32-ops",
    "-Wall", "-Wno-unused-function",
    "-I", INCLUDE, "-I", CSRC,
]


def _compile(src):
    obj = os.path.join(OBJDIR, os.path.splitext(src)[0] + ".o")
    cmd = [HIPCC, *CFLAGS, "-c", os.path.join(CSRC, src), "-o", obj]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {src}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    return obj


def _build_module(source, out):
    """Compile a CPython module over the ABI (host code against torch's headers)
    next to the library it links."""
    import sysconfig

    import torch

    t = os.path.dirname(torch.__file__)
    tmp = out + ".tmp"
    cmd = [HIPCC, "-x", "c++", "-O2", "-std=c++17", "-fPIC", "-shared", "-Wall", "-D__HIP_PLATFORM_AMD__=1",
           f"-D_GLIBCXX_USE_CXX11_ABI={int(torch._C._GLIBCXX_USE_CXX11_ABI)}",
           "-I", INCLUDE, "-isystem", os.path.join(t, "include"),
           "-isystem", os.path.join(t, "include", "torch", "csrc", "api", "include"),
           "-isystem", sysconfig.get_paths()["include"],
           "-isystem", os.path.join(os.path.dirname(os.path.dirname(HIPCC)), "include"),
           os.path.join(CSRC, source), "-o", tmp,
           "-L", PKG, "-lqlora_nf4", "-Wl,-rpath,$ORIGIN",
           "-L", os.path.join(t, "lib"), "-ltorch_python", "-ltorch_cpu", "-lc10", "-lc10_hip"]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"hipcc failed for {source}:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, out)


def _build_binding():
    _build_module("decoder_binding.cpp", BINDING)


def build(verbose=True):
    """Compile every source and link the shared library and the Python modules;
    returns the library's path."""
    os.makedirs(OBJDIR, exist_ok=True)
    with concurrent.futures.ThreadPoolExecutor(max_workers=len(SOURCES)) as ex:
        objs = list(ex.map(_compile, SOURCES))
    tmp = LIB + ".tmp"
    cmd = [HIPCC, f"--offload-arch={ARCH}", "-shared", "-fPIC", "-o", tmp, *objs]
    r = subprocess.run(cmd, capture_output=True, text=True)
    if r.returncode != 0:
        raise RuntimeError(f"link failed:\n{' '.join(cmd)}\n{r.stdout}\n{r.stderr}")
    os.replace(tmp, LIB)
    with concurrent.futures.ThreadPoolExecutor(max_workers=2) as ex:
        for f in [ex.submit(_build_binding), ex.submit(_build_module, "kv_binding.cpp", KV_BINDING)]:
            f.result()
    if verbose:
        print(f"built {LIB}")
    return LIB


if __name__ == "__main__":
    build()
    sys.exit(0)
