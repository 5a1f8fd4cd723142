"""The build of the decoder operators' Python module: with the compiler of the
library alone, and imported by the build check."""

import os
import subprocess
import sys

import pytest

from bit_nf4_quantized_quantize_amd import build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_the_module_needs_no_other_compiler(tmp_path, monkeypatch):
    """Nothing but hipcc is called (no compiler is to be found by name), and the
    result loads."""
    if not (os.path.exists(build.HIPCC) and os.path.exists(build.LIB)):
        pytest.skip("hipcc or the library not available")
    out = str(tmp_path / "_decoder.so")
    monkeypatch.setattr(build, "BINDING", out)
    called, run = [], subprocess.run

    def watch(cmd, *a, **k):
        called.append(cmd[0])
        return run(cmd, *a, **k)
    monkeypatch.setattr(subprocess, "run", watch)
    build._build_binding()
    assert called == [build.HIPCC]
    code = ("import torch, ctypes, importlib.util as u; ctypes.CDLL(%r, ctypes.RTLD_GLOBAL); "
            "s = u.spec_from_file_location('_decoder', %r); m = u.module_from_spec(s); s.loader.exec_module(m); "
            "print(sorted(n for n in dir(m) if n[0] != '_'))" % (build.LIB, out))
    env = dict(os.environ, LD_LIBRARY_PATH=build.PKG + ":" + os.environ.get("LD_LIBRARY_PATH", ""))
    r = run([sys.executable, "-c", code], capture_output=True, text=True, env=env, timeout=120)
    assert r.returncode == 0, r.stderr[-2000:]
    assert r.stdout.strip() == str(["attention", "cache_write", "norm_bwd", "norm_fwd", "plan", "rope"])


def test_the_build_check_imports_the_module(monkeypatch):
    """__graft_entry__.build() fails if the module it built does not load."""
    import __graft_entry__ as entry
    from bit_nf4_quantized_quantize_amd import decoder
    if not os.path.exists(build.LIB):
        pytest.skip("the library is not built")
    monkeypatch.setattr(build, "build", lambda *a, **k: build.LIB)
    entry.build()
    monkeypatch.setattr(decoder, "_native", None)
    monkeypatch.setitem(sys.modules, "bit_nf4_quantized_quantize_amd._decoder", None)
    import bit_nf4_quantized_quantize_amd as pkg
    monkeypatch.delattr(pkg, "_decoder", raising=False)
    with pytest.raises(decoder.B.QLoraLibraryError):
        entry.build()
