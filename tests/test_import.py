"""The package and the C ABI need no torch until a call takes tensors (CPU only)."""
import os
import subprocess
import sys

import pytest

from bitlinear_w1_a8_gb300 import build as blbuild

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def run(code, path=""):
    blbuild.build()
    env = {**os.environ, "PYTHONPATH": path}
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, env=env, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


USE = """
import sys
import bitlinear_w1_a8_gb300 as bl
lib = bl.load_library()
assert bl.bitlinear_packed_bytes(128, 64) == 2048
assert bl.bitlinear_attention_workspace(1, 8, 8, 128) > 0
assert lib.bitlinear_kv_read(None, 1, None, None, None, 1, 1, 1, None, 1, None, 1, 0, None) == -1
"""


def test_import_brings_no_torch():
    run(USE + "assert 'torch' not in sys.modules")


@pytest.mark.parametrize("error", ["ImportError", "OSError", "RuntimeError"])
def test_a_torch_that_does_not_import_leaves_the_c_abi(error, tmp_path):
    (tmp_path / "torch.py").write_text(f"raise {error}('no torch here')\n")
    run(USE, str(tmp_path))


@pytest.mark.parametrize("error", ["ImportError", "RuntimeError"])
def test_a_torch_that_does_not_import_leaves_the_build(error, tmp_path):
    (tmp_path / "torch.py").write_text(f"raise {error}('no torch here')\n")
    run(f"from bitlinear_w1_a8_gb300 import build\nbuild.BUILD = {str(tmp_path)!r}\n"
        "assert build._build_marshal(False, False) is None", str(tmp_path))


@pytest.mark.parametrize("first", ["torch", "bitlinear_w1_a8_gb300"])
def test_the_order_of_imports_does_not_matter(first):
    """Either way the attention calls are ready: the marshal loaded where it was built, tensors refused as tensors."""
    run(f"import {first}" + USE + """
import os, torch
x, p = torch.zeros(1, 1, 64), torch.zeros(1, dtype=torch.int32)
f = bl.bitlinear_rope_frequencies(64)
for _ in range(2):
    try:
        bl.bitlinear_rope(x, p, (f, 0), x)
        raise SystemExit('took CPU tensors')
    except TypeError:
        pass
from bitlinear_w1_a8_gb300 import build
assert (bl._marshal is not None) == os.path.exists(build.marshal_path())
""")
