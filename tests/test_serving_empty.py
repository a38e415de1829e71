"""Calls of a serving step's entry points on a batch without rows (CPU only: they return before they touch a GPU)."""
import bitlinear_w1_a8_gb300 as bl
from test_attention_abi import SHAPE, lib  # noqa: F401
from test_serving_abi import SHARED


def test_a_batch_without_rows_has_no_groups(lib):  # noqa: F811
    """No rows, no groups: what a program has whose batch has just emptied."""
    nothing = {**SHARED, "B": 0, "q": None, "lengths": None, "shared": None, "out": None, "workspace": None, "workspace_bytes": 0}
    f = lib.bitlinear_attention_shared
    for groups, want in ((0, 0), (1, 0), (3, 0), (-1, SHAPE)):
        assert f(*{**nothing, "groups": groups}.values(), None) == want
    assert f(*{**SHARED, "groups": 0}.values(), None) == SHAPE
    assert bl.bitlinear_attention_shared_workspace(0, 4, 2, 64, 0) == 0
