"""Refusals of a serving step's entry points (CPU only: every call fails, or returns for an empty batch, before it
touches a GPU), and its plain forms against worked examples."""
import math

import numpy as np
import pytest
import torch

import bitlinear_w1_a8_gb300 as bl
import serving_plain as plain
from test_attention_abi import A, ALIGN, BAD_PAGES, NULL, SHAPE, U, UNSUPPORTED, WORKSPACE, lib, pages, refusals  # noqa: F401


def summary(**kw):
    return bl.BitLinearKVSummary(**{**dict(bounds=A, step=A), **kw})


BIG = 1 << 40
SHARED = dict(q=A, q_stride=256, B=6, Hq=4, cache=pages(), table=A, table_stride=5, max_pages=5, lengths=A, shared=A, groups=2,
              scale=0.125, out=A, out_stride=256, workspace=A, workspace_bytes=BIG, flags=0)
BLOCKS = dict(q=A, q_stride=256, B=3, Hq=4, cache=pages(), table=A, table_stride=5, max_pages=5, lengths=A, blocks=A, count=3,
              scale=0.125, out=A, out_stride=256, flags=0)
SUMMARISE = dict(cache=pages(), summary=summary(), table=A, table_stride=5, B=3, max_pages=5, first=A, lengths=A, flags=0)
SELECT = dict(q=A, q_stride=256, B=3, Hq=4, cache=pages(), summary=summary(), table=A, table_stride=5, max_pages=5, lengths=A,
              keep_first=1, keep_last=1, blocks=A, count=3, flags=0)
SOFTMAX = dict(y=A, M=3, N=7, temperature=A, p=A, flags=0)
VERIFY = dict(p=A, q=A, B=3, K=2, N=7, draft=A, uniform=A, tokens=A, accepted=A, flags=0)

ATTENDED = [(dict(q=None), NULL), (dict(out=None), NULL), (dict(table=None), NULL), (dict(lengths=None), NULL), (dict(q=U), ALIGN),
            (dict(out=U), ALIGN), (dict(table=A + 1), ALIGN), (dict(lengths=A + 2), ALIGN), (dict(B=-1), SHAPE),
            (dict(Hq=3), SHAPE), (dict(Hq=0), SHAPE), (dict(q_stride=252), SHAPE), (dict(out_stride=258), SHAPE),
            (dict(table_stride=4), SHAPE), (dict(max_pages=0), SHAPE), (dict(scale=math.nan), SHAPE), (dict(scale=math.inf), SHAPE),
            (dict(flags=2), UNSUPPORTED), (dict(cache=None), NULL)]


def empty(**kw):
    return {**kw, "B": 0, "q": None, "lengths": None}


def test_shared_refusals(lib):  # noqa: F811
    f = lib.bitlinear_attention_shared
    refusals(f, SHARED, ATTENDED + [(dict(cache=pages(**c)), w) for c, w in BAD_PAGES])
    need = bl.bitlinear_attention_shared_workspace(6, 4, 2, 64, 2)
    assert need > 0
    refusals(f, SHARED, [(dict(shared=None), NULL), (dict(shared=A + 2), ALIGN), (dict(groups=0), SHAPE), (dict(groups=-2), SHAPE),
                         (dict(groups=4), SHAPE), (dict(groups=12), SHAPE), (dict(B=1 << 30, groups=1), SHAPE),
                         (dict(workspace=None), WORKSPACE), (dict(workspace_bytes=need - 1), WORKSPACE), (dict(workspace=U), ALIGN)])
    assert f(*{**SHARED, **empty(shared=None, workspace=None)}.values(), None) == 0


@pytest.mark.parametrize("sizes", [(0, 4, 2, 64, 1), (6, 4, 3, 64, 2), (6, 4, 2, 72, 2), (6, 4, 2, 64, 4), (6, 4, 2, 64, 0), (1 << 30, 4, 2, 64, 1),
                                   (6, 0, 2, 64, 2), (6, 4, 0, 64, 2)])
def test_shared_workspace_of_bad_sizes(lib, sizes):  # noqa: F811
    assert bl.bitlinear_attention_shared_workspace(*sizes) == 0


def test_shared_workspace_of_rows_that_share_nothing_is_attentions(lib):  # noqa: F811
    for B, Hq, Hkv, D in ((1, 32, 8, 128), (3, 8, 8, 80), (64, 32, 32, 80)):
        assert bl.bitlinear_attention_shared_workspace(B, Hq, Hkv, D, B) == bl.bitlinear_attention_workspace(B, Hq, Hkv, D)


def test_blocks_refusals(lib):  # noqa: F811
    f = lib.bitlinear_attention_blocks
    refusals(f, BLOCKS, ATTENDED + [(dict(cache=pages(**c)), w) for c, w in BAD_PAGES])
    refusals(f, BLOCKS, [(dict(blocks=None), NULL), (dict(blocks=A + 2), ALIGN), (dict(count=0), SHAPE), (dict(count=4097), SHAPE)])
    assert f(*{**BLOCKS, **empty(blocks=None)}.values(), None) == 0


def test_summarise_refusals(lib):  # noqa: F811
    f = lib.bitlinear_kv_summarise
    refusals(f, SUMMARISE, [(dict(cache=pages(**c)), w) for c, w in BAD_PAGES])
    refusals(f, SUMMARISE, [(dict(cache=None), NULL), (dict(summary=None), NULL), (dict(summary=summary(bounds=None)), NULL),
                            (dict(summary=summary(step=None)), NULL), (dict(summary=summary(bounds=U)), ALIGN), (dict(summary=summary(step=U)), ALIGN),
                            (dict(table=None), NULL), (dict(first=None), NULL), (dict(lengths=None), NULL), (dict(table=A + 1), ALIGN),
                            (dict(first=A + 2), ALIGN), (dict(lengths=A + 2), ALIGN), (dict(B=-1), SHAPE), (dict(table_stride=4), SHAPE),
                            (dict(max_pages=0), SHAPE), (dict(flags=2), UNSUPPORTED)])
    assert f(*{**SUMMARISE, "B": 0, "table": None, "first": None, "lengths": None}.values(), None) == 0


def test_select_refusals(lib):  # noqa: F811
    f = lib.bitlinear_attention_select
    own = [(c, w) for c, w in ATTENDED if not {"out", "out_stride", "scale"} & set(c)]
    refusals(f, SELECT, own + [(dict(cache=pages(**c)), w) for c, w in BAD_PAGES])
    refusals(f, SELECT, [(dict(summary=None), NULL), (dict(summary=summary(bounds=None)), NULL), (dict(summary=summary(step=U)), ALIGN),
                         (dict(blocks=None), NULL), (dict(blocks=A + 2), ALIGN), (dict(count=0), SHAPE), (dict(count=4097), SHAPE),
                         (dict(keep_first=-1), SHAPE), (dict(keep_last=-1), SHAPE), (dict(max_pages=131073, table_stride=131073), UNSUPPORTED)])
    assert f(*{**SELECT, **empty(blocks=None, table=None)}.values(), None) == 0


def test_softmax_refusals(lib):  # noqa: F811
    f = lib.bitlinear_softmax
    refusals(f, SOFTMAX, [(dict(y=None), NULL), (dict(p=None), NULL), (dict(y=U), ALIGN), (dict(p=U), ALIGN), (dict(temperature=A + 2), ALIGN),
                          (dict(M=-1), SHAPE), (dict(N=0), SHAPE), (dict(N=1 << 31), SHAPE), (dict(M=1 << 30, N=1 << 19), SHAPE),
                          (dict(flags=2), UNSUPPORTED)])
    assert f(*{**SOFTMAX, "M": 0, "y": None, "p": None}.values(), None) == 0


def test_verify_refusals(lib):  # noqa: F811
    f = lib.bitlinear_verify
    refusals(f, VERIFY, [(dict(p=None), NULL), (dict(q=None), NULL), (dict(draft=None), NULL), (dict(uniform=None), NULL), (dict(tokens=None), NULL),
                         (dict(accepted=None), NULL), (dict(p=U), ALIGN), (dict(q=U), ALIGN), (dict(draft=A + 1), ALIGN), (dict(uniform=A + 1), ALIGN),
                         (dict(tokens=A + 1), ALIGN), (dict(accepted=A + 1), ALIGN), (dict(B=-1), SHAPE), (dict(K=-1), SHAPE), (dict(K=65536), SHAPE),
                         (dict(N=0), SHAPE), (dict(N=1 << 31), SHAPE), (dict(B=1 << 30, N=1 << 18), SHAPE), (dict(flags=2), UNSUPPORTED)])
    assert f(*{**VERIFY, "B": 0, "p": None, "uniform": None}.values(), None) == 0


def test_binding_refuses_cpu_tensors(lib):  # noqa: F811
    x, i = torch.zeros(2, 2, 64), torch.zeros(2, dtype=torch.int32)
    cache = tuple(torch.zeros(4, 2, 16, 64, dtype=torch.int8) for _ in "kv") + tuple(torch.zeros(4, 2, 16) for _ in "kv")
    table, s = torch.zeros(2, 2, dtype=torch.int32), (torch.zeros(4, 2, 2, 64, dtype=torch.int8), torch.zeros(4, 2))
    blocks = torch.zeros(2, 2, 1, dtype=torch.int32)
    for call in (lambda: bl.bitlinear_attention_shared(x, cache, table, i, i, x), lambda: bl.bitlinear_kv_summarise(cache, s, table, i, i),
                 lambda: bl.bitlinear_attention_select(x, cache, s, table, i, blocks), lambda: bl.bitlinear_attention_blocks(x, cache, table, i, blocks, x),
                 lambda: bl.bitlinear_softmax(x[0], x[0]), lambda: bl.bitlinear_verify(x, x, i, x, i, i)):
        with pytest.raises(TypeError):
            call()


# ------------------------------------------------------------------ the plain forms


def test_plain_verify_of_worked_rows():
    p = np.array([[[0.5, 0.25, 0.25, 0], [0, 0, 1, 0]]], np.float32)
    q = np.array([[[0.25, 0.75, 0, 0]]], np.float32)
    case = lambda x, u0, u1: tuple(a.tolist() for a in plain.verify(p, q, np.array([[x]]), np.array([[u0, u1]], np.float32)))  # noqa: E731
    assert case(0, 0.999, 0.5) == ([[0, 2]], [1])         # p > q: always taken
    assert case(1, 0.25, 0.5) == ([[1, 2]], [1])          # 0.25 * 0.75 < 0.25
    assert case(1, 0.5, 0.49) == ([[0, -1]], [0])         # refused; what is left: 0.25 at 0 and at 2
    assert case(1, 0.5, 0.5) == ([[2, -1]], [0])
    assert case(-1, 0.0, 0.7) == ([[1, -1]], [0])         # no draft: from p itself
    assert case(3, 0.0, 0.1) == ([[0, -1]], [0])          # 0 < 0 is false
    same = np.array([[[0, 1.0, 0, 0], [1, 0, 0, 0]]], np.float32)
    assert plain.verify(same, same[:, :1], np.array([[0]]), np.zeros((1, 2), np.float32))[0].tolist() == [[1, -1]]  # nothing left: from p


def test_plain_bounds_hold_every_product():
    """No key of a page has a larger product with q's codes than the page's score says (both as whole codes and steps)."""
    rng = np.random.default_rng(3)
    k = torch.tensor(rng.normal(size=(6, 2, 16, 64)) * rng.uniform(0.1, 3, (1, 2, 1, 64)), dtype=torch.bfloat16)
    bounds, steps = plain.summaries((k, k, None, None), range(6), [16, 16, 1, 7, 16, 16])
    q = rng.normal(size=64)
    codes = np.rint(q * 127 / np.abs(q).max())
    x = k.double().numpy()
    for p, n in enumerate([16, 16, 1, 7, 16, 16]):
        for h in range(2):
            lo, hi = bounds[p, h].astype(np.float64) * float(steps[p, h])
            # outwards but for a rounding of the code itself (half a step of fp32 in hi * s, and the clamp at 127)
            slack = 127.5 * float(steps[p, h]) * 2.0 ** -22
            assert (x[p, h, :n] <= hi + slack).all() and (x[p, h, :n] >= lo - slack).all()
            assert (x[p, h, :n] @ codes).max() <= np.maximum(codes * lo, codes * hi).sum() + slack * np.abs(codes).sum()
