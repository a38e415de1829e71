"""Calls of the serving operators at the edges of what they allow."""
import pytest

import bitlinear_w1_a8_gb300 as bl
from test_gpu_serving import filled_cache, ints, new_summary

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    bl.load_library()


# ------------------------------------------------------------------ summaries


@pytest.mark.parametrize("first,lengths", [([5, 16, 40], [5, 16, 40]), ([37, 39, 47], [35, 33, 41]), ([0, 10 ** 9, 2 ** 31 - 1], [0, 40, 48]),
                                           ([1, 3, 20], [0, -5, 20])])
def test_summarise_of_no_token_writes_nothing(first, lengths):
    """first at or behind the length, in the page of the last token among them: a sequence that has nothing new."""
    cache, table = filled_cache("int8", 3, 2, 80, [48, 48, 48], 16, 5)
    bounds, step = new_summary(cache)
    bl.bitlinear_kv_summarise(cache, (bounds, step), ints(table), ints(first), ints(lengths))
    assert (bounds == 99).all() and (step == 5.0).all()
