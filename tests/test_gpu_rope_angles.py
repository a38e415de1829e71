"""The angle of a rotation, as include/bitlinear.h bounds it: fast and slow pairs, near and far positions."""
import numpy as np
import pytest
import torch

import attention_plain as plain
import bitlinear_w1_a8_gb300 as bl

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("layout", [bl.ROPE_HALF, bl.ROPE_INTERLEAVED])
@pytest.mark.parametrize("low,high", [(1e-14, 1e-9), (1e-9, 1e-4), (1e-4, 1.0), (1.0, 1e3)])
def test_sine_and_cosine(low, high, layout):
    """The row (1, 0) of a pair becomes its cosine and sine: one product by 1, no sum that rounds."""
    n, T = 64, 4000
    rng = np.random.default_rng(int(-np.log10(low)) + 3)
    freq = np.exp(rng.uniform(np.log(low), np.log(high), n)) * rng.choice([1, 1, 1, -1], n)
    pos = np.concatenate([np.arange(1000), -np.arange(1000), rng.integers(-2 ** 31, 2 ** 31, 1000),
                          np.exp(rng.uniform(0, np.log(2.0 ** 31 - 1), 1000)).astype(np.int64)])
    x = torch.zeros(T, 1, 2 * n, device="cuda")
    a, b = (slice(0, n), slice(n, 2 * n)) if layout == bl.ROPE_HALF else (slice(0, None, 2), slice(1, None, 2))
    x[..., a] = 1.0
    bl.bitlinear_rope(x, torch.tensor(pos, dtype=torch.int32, device="cuda"), (torch.tensor(freq).cuda(), layout), x)
    angle = pos.astype(np.longdouble)[:, None] * freq.astype(np.longdouble)[None]
    got, off = x.double().cpu().numpy()[:, 0], np.abs(angle) * 2.0 ** -52 + np.abs(pos)[:, None] * 2.0 ** -62 + 2.0 ** -45
    for want, of in ((np.cos(angle), a), (np.sin(angle), b)):
        # half a step of fp32; the series' own 2^-40 makes the nearest value one of two in a border case
        bound = np.abs(want) * plain.U * (1 + 2.0 ** -10) + off * (1 + 2.0 ** -10)
        assert (np.abs(got[:, of] - want) <= bound).all()
