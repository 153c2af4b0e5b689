"""The native binding: only the calls that it serves need it, and it follows the torch it was built against."""
import os
import subprocess
import sys

import pytest

from learned_sparse_kv_b200 import build as lbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

WITHOUT = """
import os.path
real = os.path.exists
os.path.exists = lambda p: not str(p).endswith("_binding.so") and real(p)
from learned_sparse_kv_b200 import lsa
assert lsa.sparse_decode_workspace_size(1, 16, 128, 128, 512, 8000) > 0
for call in (lambda: lsa.build_tables(None, None, None, 1, 1), lambda: lsa.read_q4(None, None)):
    try:
        call()
    except ImportError as e:
        assert "build" in str(e)
    else:
        raise SystemExit("no error")
os.path.exists = real
try:
    lsa.build_tables(None, None, None, 1, 1)
except lsa.LSAError as e:
    assert "CUDA tensor" in str(e)
print("ok")
"""


def test_other_calls_do_without_the_binding():
    lbuild.build()
    r = subprocess.run([sys.executable, "-c", WITHOUT], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0 and r.stdout.strip() == "ok", r.stderr[-800:]


def test_the_binding_is_rebuilt_for_another_torch(monkeypatch):
    """It links torch's internals: an unchanged source is not enough to keep it."""
    lbuild.build()
    done = []
    monkeypatch.setattr(lbuild, "_compile", lambda src, verbose: pytest.fail("a CUDA source is compiled again"))
    monkeypatch.setattr(lbuild, "_compile_binding", lambda: done.append("compile") or "binding.o")
    monkeypatch.setattr(lbuild, "_link_binding", lambda obj: done.append("link"))
    lbuild.build()
    assert not done
    real = lbuild._torch_version
    monkeypatch.setattr(lbuild, "_torch_version", lambda: "another torch\n")
    written = []
    monkeypatch.setattr(lbuild, "_note_torch", lambda: written.append(1))
    lbuild.build()
    assert done == ["compile", "link"] and written
    monkeypatch.setattr(lbuild, "_torch_version", real)
    done.clear()
    lbuild.build()
    assert not done
