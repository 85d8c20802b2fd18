"""The package without its extension module: the denoiser's users need only the library, and the token calls go through
ctypes with the same checks."""

import importlib.util
import os
import re
import shutil
import subprocess
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
PACKAGE = os.path.join(ROOT, "conv2d_implicit_gemm_gb300")


def _module(path):
    spec = importlib.util.spec_from_file_location("_tested", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


def test_package_imports_and_refuses_without_the_extension(tmp_path):
    """A copy of the package with the library alone passes every test of what the token calls refuse."""
    copy = tmp_path / "conv2d_implicit_gemm_gb300"
    copy.mkdir()
    for name in os.listdir(PACKAGE):
        if name.endswith(".py"):
            shutil.copy(os.path.join(PACKAGE, name), copy)
    os.symlink(os.path.join(PACKAGE, "liboidnx.so"), copy / "liboidnx.so")
    (tmp_path / "tests").mkdir()
    shutil.copy(os.path.join(ROOT, "tests", "test_token_refusals.py"), tmp_path / "tests")
    (tmp_path / "tests" / "test_which.py").write_text(
        "def test_which():\n    import conv2d_implicit_gemm_gb300 as ox\n    import types\n"
        f"    assert ox.__file__.startswith({str(tmp_path)!r})\n"
        "    assert isinstance(ox._calls, types.SimpleNamespace)\n    assert ox.oidnx_version()\n")
    run = subprocess.run([sys.executable, "-m", "pytest", "-q", "-p", "no:cacheprovider", "tests"], cwd=tmp_path,
                         env={**os.environ, "PYTHONPATH": str(tmp_path)}, capture_output=True, text=True, timeout=300)
    assert run.returncode == 0, run.stdout[-2000:] + run.stderr[-2000:]


def test_both_entries_take_the_same_arguments():
    kinds = _module(os.path.join(PACKAGE, "_calls_ctypes.py")).KINDS
    with open(os.path.join(PACKAGE, "csrc", "calls.c")) as f:
        assert dict(re.findall(r'convert\("(\w+)", "(\w+)"', f.read())) == kinds


def test_a_build_without_a_c_compiler_goes_on(tmp_path, monkeypatch, capsys):
    build = _module(os.path.join(PACKAGE, "build.py"))
    monkeypatch.setattr(build, "PKG", str(tmp_path))
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "_calls.abi3.so"))
    monkeypatch.setattr(build.shutil, "which", lambda name: str(tmp_path / "no-such-compiler"))
    assert build._build_calls() is False
    assert "ctypes" in capsys.readouterr().err and not os.listdir(tmp_path)
    monkeypatch.setattr(build.shutil, "which", lambda name: "/bin/false")
    assert build._build_calls() is False
