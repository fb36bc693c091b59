"""The C library builds with nvcc alone: without torch, and not again for another torch or Python."""
import importlib.util
import subprocess
import sys
from pathlib import Path

BUILD = Path(__file__).resolve().parents[1] / "speculative_decoding_token_temperature_gb300" / "build.py"


def _module():
    spec = importlib.util.spec_from_file_location("specdec_build", BUILD)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def test_the_library_builds_without_torch(built_library):
    """In a Python that has no torch (and with the library up to date, so that nothing is compiled here)."""
    code = ("import runpy, sys, importlib.util as u; sys.modules['torch'] = None; find = u.find_spec\n"
            "u.find_spec = lambda n, *a: None if n == 'torch' else find(n, *a)\n"
            f"sys.argv = ['build.py']; runpy.run_path({str(BUILD)!r}, run_name='__main__')")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True, timeout=120)
    assert r.returncode == 0, r.stderr
    assert r.stdout.strip().endswith("libspecdec.so")


def test_another_torch_rebuilds_the_binding_alone(built_library, monkeypatch):
    import torch
    m = _module()
    library, calls = m._fingerprint(), m._calls_fingerprint()
    monkeypatch.setattr(torch, "__version__", "0.0")
    assert m._fingerprint() == library and m._calls_fingerprint() != calls
    monkeypatch.setattr(sys, "version", "0.0")
    assert m._fingerprint() == library
    assert m._current(m.LIB_PATH, m.BUILD_DIR / "stamp", library)
