"""The decoder-block entry points' host logic (argument checks, workspace sizes)
under AddressSanitizer and UndefinedBehaviorSanitizer, without a GPU: built for
the CPU with stand-ins for the launchers and driven over ordinary and extreme
sizes (tests/host/decoder_sanitize_main.cpp).  The sanitizers apply to host code
only (-Xarch_host)."""

import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "bit_nf4_quantized_quantize_amd", "csrc")
HOST = os.path.join(ROOT, "tests", "host")
HIPCC = os.environ.get("HIPCC", "/opt/rocm/bin/hipcc")


def test_decoder_abi_host_logic_under_asan_ubsan(tmp_path):
    if not os.path.exists(HIPCC):
        pytest.skip("hipcc not available")
    exe = str(tmp_path / "decoder_sanitized")
    cmd = [HIPCC, "-O1", "-g", "-std=c++17", "--offload-arch=gfx950",
           "-Xarch_host", "-fsanitize=address", "-Xarch_host", "-fsanitize=undefined",
           "-Xarch_host", "-fno-sanitize-recover=all",
           "-I", os.path.join(ROOT, "include"), "-I", CSRC, os.path.join(HOST, "decoder_sanitize_main.cpp"),
           os.path.join(CSRC, "decoder_abi.cpp"), "-o", exe]
    r = subprocess.run(cmd, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0, r.stderr[-4000:]
    env = dict(os.environ, ASAN_OPTIONS="detect_leaks=0:abort_on_error=1", UBSAN_OPTIONS="print_stacktrace=1")
    r = subprocess.run([exe], capture_output=True, text=True, timeout=300, env=env)
    assert r.returncode == 0, (r.stdout + r.stderr)[-4000:]
    assert r.stdout.startswith("ok ") and int(r.stdout.split()[1]) > 1000, r.stdout
