"""The compiled marshal belongs to one header, source, Python and torch: no other is loaded, and none is left
behind by a build that cannot make the one that belongs (CPU only)."""
import os
import shutil
import subprocess
import sys

import pytest

from bitlinear_w1_a8_gb300 import build as blbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def loaded(before):
    """Whether a fresh process that runs `before` first loads the marshal."""
    code = f"{before}\nimport torch, bitlinear_w1_a8_gb300 as bl\nbl.load_library()\nprint(bl._marshal is not None)"
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return {"True": True, "False": False}[r.stdout.split()[-1]]


@pytest.fixture(scope="module")
def built():
    blbuild.build()
    if not loaded(""):
        pytest.skip("bitlinear_marshal was not built")


@pytest.mark.parametrize("change", [
    "import torch; torch.__version__ = torch.__version__ + '.1'",
    "import torch; torch.version.git_version = '0'",
    "import sysconfig; was = sysconfig.get_config_var; sysconfig.get_config_var = lambda n: 'cpython-39' if n == 'SOABI' else was(n)",
])
def test_a_marshal_of_another_python_or_torch_is_not_loaded(built, change):
    assert not loaded(change)


@pytest.mark.parametrize("name", ["bitlinear.h", "marshal.cpp"])
def test_a_marshal_of_another_source_is_not_loaded(built, name, tmp_path):
    folder = "INCLUDE" if name.endswith(".h") else "CSRC"
    shutil.copy(os.path.join(getattr(blbuild, folder), name), tmp_path / name)
    with open(tmp_path / name, "a") as f:
        f.write("/* changed */\n")
    assert not loaded(f"from bitlinear_w1_a8_gb300 import build\nbuild.{folder} = {str(tmp_path)!r}")


@pytest.mark.parametrize("command", [None, ["false"]])
def test_a_build_that_fails_leaves_none_behind(monkeypatch, tmp_path, command):
    monkeypatch.setattr(blbuild, "BUILD", str(tmp_path))
    old = tmp_path / "bitlinear_marshal.so"
    monkeypatch.setattr(blbuild, "MARSHAL", str(old), raising=False)
    old.write_bytes(b"of an older header")
    os.utime(old, (1, 1))
    monkeypatch.setattr(blbuild, "_marshal_command", lambda out: command)
    assert blbuild._build_marshal(False, False) is None
    assert list(tmp_path.iterdir()) == []


def test_builds_at_the_same_time(monkeypatch, tmp_path):
    """What another build has removed already is no error."""
    monkeypatch.setattr(blbuild, "BUILD", str(tmp_path))
    monkeypatch.setattr(blbuild.glob, "glob", lambda pattern: [str(tmp_path / "bitlinear_marshal-gone.so")])
    monkeypatch.setattr(blbuild, "_marshal_command", lambda out: None)
    assert blbuild._build_marshal(False, False) is None


def test_a_torch_that_is_still_importing_leaves_the_c_abi(built):
    assert not loaded("import torch; del torch.__version__")
