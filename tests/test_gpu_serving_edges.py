"""Calls of the serving operators at the edges of what they allow."""
import numpy as np
import pytest
import torch

import bitlinear_w1_a8_gb300 as bl
from test_gpu_serving import filled_cache, ints, new_summary, normal, random_summary

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


# ------------------------------------------------------------------ the choice


@pytest.mark.parametrize("compiled", [True, False])
def test_kept_pages_beyond_32_bits(compiled, monkeypatch):
    """Counts of kept pages that an int cannot hold are all pages, or refused below 0: never what is left of them in 32 bits."""
    if not compiled:
        monkeypatch.setattr(bl, "_marshal", None)
    page, D, columns, count = 16, 64, 40, 8
    bounds, step = (torch.as_tensor(x).cuda() for x in random_summary(columns, 1, D, 1))
    sizes = torch.empty(columns, 1, page, D, dtype=torch.bfloat16, device="cuda")
    q, table, n = normal((1, 1, D), 2).cuda(), ints(np.arange(columns)[None]), ints([columns * page])

    def run(**keep):
        blocks = torch.full((1, 1, count), 7, dtype=torch.int32, device="cuda")
        bl.bitlinear_attention_select(q, (sizes, sizes), (bounds, step), table, n, blocks, **keep)
        return blocks[0, 0].tolist()

    everything = list(range(count))  # of more kept than count the first
    assert run(keep_first=2 ** 31 - 1, keep_last=0) == everything
    for many in (2 ** 31, 2 ** 32, 2 ** 32 + 1, 2 ** 70):
        assert run(keep_first=many, keep_last=0) == everything
        assert run(keep_first=0, keep_last=many) == everything
        for keep in (dict(keep_first=-many), dict(keep_last=-many)):
            with pytest.raises(bl.BitLinearError):
                run(**keep)
