"""What needs no torch is built where there is none: the library, the oracle and the input generator."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("program", ["import __graft_entry__; __graft_entry__.build()",
                                     "from communication_compressed_sign_gb300 import build; assert build.build_tensors(force=True) is None"])
def test_build_without_torch(program):
    r = subprocess.run([sys.executable, "-c", f"import sys; sys.modules['torch'] = None; {program}"], cwd=ROOT, capture_output=True,
                       text=True, timeout=600)
    assert r.returncode == 0, r.stderr
    assert "_tensors" in r.stderr  # what was left out is said


def test_build_without_pythons_headers(monkeypatch, tmp_path, capsys):
    pytest.importorskip("torch")
    from communication_compressed_sign_gb300 import build
    monkeypatch.setattr(build.sysconfig, "get_paths", lambda: {"include": str(tmp_path)})
    assert build.build_tensors(force=True) is None and "_tensors" in capsys.readouterr().err
