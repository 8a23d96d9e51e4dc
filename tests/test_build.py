"""Building without a GPU: what the C library needs, and when the torch module is built anew."""
import os
import subprocess
import sys

import pytest

from mtp_speculative_draft_lm_b200 import build as B

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# the built objects, linked to a library elsewhere by a Python whose torch cannot be imported
WITHOUT_TORCH = """
import sys
sys.path.insert(0, {root!r})
sys.modules["torch"] = None
from mtp_speculative_draft_lm_b200 import build as B
B.LIB, B.CALLS, B.CALLS_KEY = {lib!r}, {calls!r}, {calls!r} + ".key"
B.build()
import ctypes
assert ctypes.CDLL(B.LIB).mtp_abi_version() >= 1
"""


@pytest.fixture(scope="module", autouse=True)
def built():
    B.build()


def test_the_library_builds_without_torch(tmp_path):
    lib, calls = str(tmp_path / "libmtp.so"), str(tmp_path / "_block.so")
    r = subprocess.run([sys.executable, "-c", WITHOUT_TORCH.format(root=ROOT, lib=lib, calls=calls)], capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    assert os.path.exists(lib) and not os.path.exists(calls)


def test_the_library_is_linked_where_the_module_fails(tmp_path, monkeypatch):
    """A torch whose headers do not compile (here: another compiler's absence) leaves the library built."""
    monkeypatch.setattr(B, "LIB", str(tmp_path / "libmtp.so"))
    monkeypatch.setattr(B, "CALLS", str(tmp_path / "_block.so"))
    monkeypatch.setattr(B, "CALLS_SRC", str(tmp_path / "none.cpp"))
    (tmp_path / "none.cpp").write_text("#error no\n")
    with pytest.raises(RuntimeError, match="none.cpp"):
        B.build()
    assert os.path.exists(B.LIB) and not os.path.exists(B.CALLS)


def test_another_torch_builds_the_module_anew(tmp_path, monkeypatch):
    """A module newer than its source, but of another torch, is not taken for the current one."""
    calls, key = tmp_path / "_block.so", tmp_path / "key"
    monkeypatch.setattr(B, "CALLS", str(calls))
    monkeypatch.setattr(B, "CALLS_KEY", str(key))
    ran = []
    monkeypatch.setattr(B.subprocess, "run", lambda cmd, **kw: ran.append(cmd) or open(cmd[cmd.index("-o") + 1], "w").close()
                        or subprocess.CompletedProcess(cmd, 0, "", ""))
    B._build_calls(False)
    assert len(ran) == 1 and calls.exists()
    B._build_calls(False)
    assert len(ran) == 1
    key.write_text(key.read_text().replace("torch ", "torch 0."))
    B._build_calls(False)
    assert len(ran) == 2 and key.read_text() == B._calls_key()
