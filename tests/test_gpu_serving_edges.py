"""Calls of the serving operators at the edges of what they allow."""
import numpy as np
import pytest
import torch

import attention_plain
import bitlinear_w1_a8_gb300 as bl
import serving_plain as plain
from harness import check_canary, guarded
from serving_ways import way
from test_gpu_serving import filled_cache, ints, new_summary, normal, random_summary, shared_case, wide_table, within

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


# ------------------------------------------------------------------ a row's own tokens


@pytest.mark.parametrize("fmt", attention_plain.FORMATS)
@pytest.mark.parametrize("R,G,want", [(4, 1, "eight"), (24, 4, "wide"), (160, 1, "wide"), (39, 8, "wide"), (20, 1, "eight"), (150, 1, "wide")])
def test_a_number_that_is_not_finite_stays_with_its_row(fmt, R, G, want):
    """A NaN in one row's own token, in a page of its own: that row's heads of that key head alone, over clusters and in packed rows."""
    S, page, D, Hkv = 90, 16, 64, 2
    lengths = S + 25 + np.arange(R) % 11
    cache, q, table = shared_case(fmt, 1, R, Hkv * G, Hkv, D, [S], lengths, page, 31)
    columns = wide_table(table, cache)
    assert way(fmt, 1, R, Hkv * G, Hkv, D, columns.shape[1], page) == want
    out = torch.empty(q.shape, device="cuda")
    ws = torch.empty(bl.bitlinear_attention_shared_workspace(R, Hkv * G, Hkv, D, 1), dtype=torch.uint8, device="cuda")
    run = lambda: (bl.bitlinear_attention_shared(q.cuda(), cache, columns, ints(lengths), ints([S]), out, ws), out.cpu())[1]  # noqa: E731
    clean = run()
    assert torch.isfinite(clean).all()
    row = R // 2 + 1
    t = int(lengths[row]) - 1
    at = table[row, t // page]
    assert t >= S and (table[:, t // page] == at).sum() == 1  # this row's alone
    rest = torch.ones(R, dtype=torch.bool)
    rest[row] = False
    for i in (0, 1):  # keys, then values
        held = cache[i] if fmt == "bf16" else cache[2 + i]
        kept = held[at, 0, t % page].clone()
        held[at, 0, t % page] = float("nan")
        got = run()
        assert torch.isnan(got[row, :G]).all()
        assert torch.equal(got[rest], clean[rest]) and torch.equal(got[row, G:], clean[row, G:])
        held[at, 0, t % page] = kept
    assert torch.equal(run(), clean)


# ------------------------------------------------------------------ probabilities


TEMPERATURES = [1.0, 0.3, 7.0, 0.0, 1e-20, 2e30, float("nan"), -1.0, float("inf")]


@pytest.mark.parametrize("V", [3, 129, 1000, 2000, 4099, 7171, 14000, 50001, 57348, 65536, 65537, 131075, 300008])
def test_softmax_of_every_temperature(V):
    """Each way of a row (held by one CTA, by up to eight, read again), at every kind of temperature, out of place and in place: maxima
    in the first and the last run, equal ones in two of them, a masked end, logits far apart."""
    M = len(TEMPERATURES)
    y = normal((M, V), V, 3.0)
    y[:, V - 1] = y[:, V // 3] = 40.0       # the largest in two CTAs; where one is chosen it is the earlier
    y[0, V // 2] = -np.inf
    y[4, V // 3] = 39.0                     # and in the last alone
    y[5] *= 1e30                            # of 1e30, which the temperature counts as, and not of 2e30
    y[8] *= 1e30
    t = torch.tensor(TEMPERATURES)
    p, full = guarded(M * V, torch.float32, 4.5)
    p = p.view(M, V)
    bl.bitlinear_softmax(y.cuda(), p, t.cuda())
    want, bound = plain.softmax(y.numpy(), t.numpy())
    within(p, want, bound)
    check_canary(full, 4.5)
    for m in (3, 4, 6, 7):
        assert p[m].sum() == 1 and p[m].argmax().item() == (V - 1 if m == 4 else V // 3)
    both, full = guarded(M * V, torch.float32, 4.5)
    both = both.view(M, V)
    both.copy_(y)
    bl.bitlinear_softmax(both, both, t.cuda())
    assert torch.equal(both, p)
    check_canary(full, 4.5)


@pytest.mark.parametrize("M,V", [(320, 129), (700, 1003), (320, 4096), (64, 65536), (33, 100003)])
def test_softmax_in_place_of_many_rows(M, V):
    """p is y: what another buffer gets, and the same in every call."""
    y, t = normal((M, V), M, 3.0).cuda(), (torch.arange(M) % 5 * 0.4).cuda()
    p = torch.empty_like(y)
    bl.bitlinear_softmax(y, p, t)
    for _ in range(3):
        x = y.clone()
        bl.bitlinear_softmax(x, x, t)
        assert torch.equal(x, p)


# ------------------------------------------------------------------ nothing to do


@pytest.mark.parametrize("compiled", [True, False])
def test_a_batch_without_rows(compiled, monkeypatch):
    """Every call of a step takes an empty batch: no groups, no rows, no sequences."""
    if not compiled:
        monkeypatch.setattr(bl, "_marshal", None)
    cache = tuple(torch.zeros(2, 2, 16, 64, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    summary, none = new_summary(cache), torch.empty(0, dtype=torch.int32, device="cuda")
    x, table = torch.empty(0, 4, 64, device="cuda"), none.view(0, 1).expand(0, 3)
    blocks = torch.empty(0, 2, 5, dtype=torch.int32, device="cuda")
    bl.bitlinear_attention_shared(x, cache, table, none, none, x.clone())
    bl.bitlinear_kv_summarise(cache, summary, table, none, none)
    bl.bitlinear_attention_select(x, cache, summary, table, none, blocks)
    bl.bitlinear_attention_blocks(x, cache, table, none, blocks, x.clone())
    y = torch.empty(0, 7, device="cuda")
    bl.bitlinear_softmax(y, y)
    p = torch.empty(0, 3, 7, device="cuda")
    bl.bitlinear_verify(p, p[:, :2], none.view(0, 1).expand(0, 2), torch.empty(0, 3, device="cuda"), none.view(0, 1).expand(0, 3), none)
    torch.cuda.synchronize()
    assert (summary[0] == 99).all()
