"""When the Python binding's compiled part is built: with another PyTorch again, without one not at all."""
import os
import subprocess
import sys
import types

import pytest

from grouped_gemm_03_b200 import build as b


@pytest.fixture
def ops(tmp_path, monkeypatch):
    """_build_ops on files of its own, the compiler a fake that writes its output file."""
    calls = []

    def compiler(cmd, **_):
        calls.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(b, "BUILD", str(tmp_path))
    monkeypatch.setattr(b, "OPS", str(tmp_path / "_ops.so"))
    monkeypatch.setattr(b.subprocess, "run", compiler)
    return calls


def test_built_once_for_one_pytorch(ops):
    b._build_ops(False, False)
    b._build_ops(False, False)
    assert len(ops) == 1 and os.path.exists(b.OPS)
    b._build_ops(True, False)
    assert len(ops) == 2


def test_built_again_for_another_pytorch(ops, monkeypatch):
    b._build_ops(False, False)
    monkeypatch.setattr(b, "_ops_made_for", lambda: "torch of another version")
    b._build_ops(False, False)
    b._build_ops(False, False)
    assert len(ops) == 2


def test_left_out_without_pytorch(ops, monkeypatch):
    monkeypatch.setattr(b.importlib.util, "find_spec", lambda name: None)
    b._build_ops(False, True)
    assert not ops and not os.path.exists(b.OPS)


def test_the_c_librarys_build_imports_no_pytorch():
    # as a script, with both files there: nothing to compile, and PyTorch is not loaded to find that out
    b.build()
    code = (f"import runpy, sys; sys.argv = ['build.py']\n"
            f"try:\n    runpy.run_path({b.__file__!r}, run_name='__main__')\n"
            f"except SystemExit as e:\n    assert not e.code, e.code\n"
            f"assert 'torch' not in sys.modules")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
