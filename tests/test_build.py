"""The build and the loading of the library where torch or the module that
marshals its tensors is missing: the C library does not depend on either."""
import subprocess
import sys

import pytest

from fp8_quantized_linear_mxq_amd import build as b


def _stub(monkeypatch, tmp_path, fail=()):
    """Commands are recorded instead of run; each writes what it would have."""
    ran = []

    class Done:
        stdout = stderr = ""

    def run(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        ran.append(out)
        r = Done()
        r.returncode = int(any(f in out for f in fail))
        if not r.returncode:
            open(out, "w").close()
        return r

    monkeypatch.setattr(b.subprocess, "run", run)
    for name in ("LIB", "PROBE_LIB", "BINDING_LIB", "BUILD"):
        monkeypatch.setattr(b, name, str(tmp_path / name))
    return ran


def test_build_without_torch(monkeypatch, tmp_path):
    ran = _stub(monkeypatch, tmp_path)
    monkeypatch.setitem(sys.modules, "torch", None)      # an import of it fails
    assert b.build(verbose=False) == b.LIB
    assert (tmp_path / "LIB").exists() and (tmp_path / "PROBE_LIB").exists()
    assert not any("BINDING_LIB" in r for r in ran)


def test_build_without_host_compiler(monkeypatch, tmp_path):
    """The error is raised, with the libraries in place."""
    _stub(monkeypatch, tmp_path, fail=["BINDING_LIB"])
    with pytest.raises(RuntimeError, match="binding build failed"):
        b.build(verbose=False)
    assert (tmp_path / "LIB").exists() and (tmp_path / "PROBE_LIB").exists()


def test_load_without_the_module():
    code = """
import sys
sys.modules["fp8_quantized_linear_mxq_amd._torch_binding"] = None
import fp8_quantized_linear_mxq_amd as mxq
assert mxq.load().mxq_version() == 1 and mxq.storage(mxq.INT8, 64) == (64, 4)
try:
    mxq.gemm(*[mxq.QTensor(mxq.INT8, 1, 64, None, None)] * 2)
except RuntimeError as e:
    assert "fp8_quantized_linear_mxq_amd.build" in str(e)
else:
    raise SystemExit("no error")
"""
    subprocess.run([sys.executable, "-c", code], check=True, cwd=b.ROOT, timeout=100)
