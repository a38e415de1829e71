"""How far a page's score bounds the products of its keys (CPU: the plain forms, which the kernels equal in every bit)."""
import numpy as np
import pytest
import torch

import serving_plain as plain


def page_of(kind, rng, n, D):
    """fp32 keys [n, D] and their steps [n] as an int8 cache holds them."""
    if kind == "one large dim":
        x = rng.normal(size=(n, D)) * 1e-3
        x[:, rng.integers(D)] = rng.uniform(0.1, 10) * rng.choice([-1, 1])
    elif kind == "equal":
        x = np.full((n, D), rng.uniform(0.01, 100) * rng.choice([-1, 1]))
    elif kind == "tiny":
        x = rng.normal(size=(n, D)) * 10.0 ** rng.uniform(-9, -5)
    else:
        x = rng.normal(size=(n, D)) * rng.uniform(0.01, 30, D)
    step = (np.abs(x).max(1).clip(1e-30) / 127).astype(np.float32)
    return np.clip(np.rint(x / step[:, None]), -127, 127).astype(np.int8), step


@pytest.mark.parametrize("kind", ["mixed", "one large dim", "equal", "tiny"])
@pytest.mark.parametrize("D", [16, 80, 256])
def test_no_product_is_above_the_score_but_for_roundings(kind, D):
    """sum_d c_d k_d (m / 127) <= score + 2^-21 m step sum_d |c_d|.

    A bound of a dim is short by three roundings (hi s, s and step) of at most 2^-24 of the page's largest value a each, so
    by 3 / 4 2^-22 a; acc step (m / 127) has three more of a sum that is at most a sum |c|.  Together 6 2^-24 (1 + 2^-20) of
    a sum |c| m / 127, with a = 127 step (1 + 2^-24): below 2^-21 m step sum |c|."""
    rng, above = np.random.default_rng(D), 0
    for _ in range(400):
        codes, steps = page_of(kind, rng, int(rng.integers(1, 17)), D)
        cache = (torch.tensor(codes)[None, None], None, torch.tensor(steps)[None, None], torch.zeros(1))
        (bounds,), (step,) = plain.summaries(cache, [0], [len(codes)])
        lower, upper, step = bounds[0, 0].astype(np.int64), bounds[0, 1].astype(np.int64), step[0]
        keys = (codes.astype(np.float32) * steps[:, None]).astype(np.float64)
        q = (keys[rng.integers(len(keys))] if rng.random() < 0.5 else rng.normal(size=D)).astype(np.float32)
        m = max(np.abs(q).max(), np.float32(1e-5))
        c = np.rint(q * (np.float32(127) / m)).astype(np.int64)
        acc = np.maximum(c * lower, c * upper).sum()
        score = (np.float32(acc) * step) * (m / np.float32(127))
        assert score.dtype == np.float32
        product = (keys @ c).max() * (float(m) / 127)
        above += product > float(score)
        assert product <= float(score) + 2.0 ** -21 * float(m) * float(step) * np.abs(c).sum()
    if kind in ("one large dim", "equal"):
        assert above > 0  # the roundings show: the score alone is no bound
