"""The compiled marshal's calls into the library, made with stand-ins for its entry points: nothing is launched."""
import ctypes

import pytest
import torch

import bitlinear_w1_a8_gb300 as bl

pytestmark = pytest.mark.gpu


@pytest.fixture
def marshal():
    lib = bl.load_library()
    if bl._marshal is None:
        pytest.skip("bitlinear_marshal was not built")
    address = lambda f: ctypes.cast(f, ctypes.c_void_p).value  # noqa: E731
    yield lambda f: bl._marshal.bind(*[address(f)] * 4)
    bl._marshal.bind(*(address(getattr(lib, "bitlinear_" + n)) for n in ("rope", "kv_append", "kv_read", "attention")))


def calls():
    """Each call's arguments in the common case -> {name: the marshal's answer}."""
    x = torch.zeros(2, 2, 64, device="cuda")
    cache = tuple(torch.zeros(4, 2, 16, 64, dtype=torch.int8, device="cuda") for _ in "kv") + tuple(
        torch.zeros(4, 2, 16, device="cuda") for _ in "kv")
    ints, table = torch.zeros(2, dtype=torch.int32, device="cuda"), torch.zeros(2, 2, dtype=torch.int32, device="cuda")
    rope = (torch.ones(32, dtype=torch.float64, device="cuda"), 0)
    m = bl._marshal
    return {"rope": m.rope(x, ints, rope, x, 0, None),
            "kv_append": m.kv_append(x, x, cache, ints, table, None, x, x, rope, 0, None),
            "kv_read": m.kv_read(cache, ints, table, x, x, None, 0, None),
            "attention": m.attention(x, cache, table, ints, x, None, None, 0, 0, None)}


def test_a_call_returns_the_librarys_status(marshal):
    status = bl.load_library().bitlinear_abi_version
    marshal(status)
    assert set(calls().values()) == {status()}


def test_other_threads_run_while_the_library_is_called(marshal):
    """An entry point that says whether its thread holds Python's lock."""
    marshal(ctypes.pythonapi.PyGILState_Check)
    assert calls() == {"rope": 0, "kv_append": 0, "kv_read": 0, "attention": 0}
    assert ctypes.pythonapi.PyGILState_Check() == 1
