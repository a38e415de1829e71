"""What bitlinear_attention's rounding has in common for all logits of a call, which no average over tokens takes
out: a stretch of the logits.

Values that name their token (one 1, else 0) give the weights themselves; the slope of log(weight / exact weight)
against the exact logit is the stretch.  Each weight is off by some U (half a step of fp32, 2^-24) besides, so over
thousands of weights and a spread of several in the logits the slope is known to a hundredth of U."""
import math

import numpy as np
import pytest
import torch

import attention_plain as plain
import bitlinear_w1_a8_gb300 as bl

pytestmark = pytest.mark.gpu

U = plain.U


def cache_of(fmt, k, v, page):
    """k, v [pages, heads, page, D] quantised; -> the cache and the fp64 keys and values that it holds."""
    pages, heads, _, D = k.shape
    cache = plain.make_cache(fmt, pages, heads, page, D, 0)
    at = torch.arange(pages * page, device="cuda")
    rows = lambda x: x.transpose(1, 2).reshape(pages * page, heads, D).cuda()  # noqa: E731
    plain.fill_row(cache, fmt, at // page, at % page, rows(k), rows(v))
    return cache, plain.held(cache, "k"), plain.held(cache, "v")


def worst_scales(D):
    """Two fp32 scales whose products with log2(e), in fp32, are off by the most up and down (relative)."""
    s = np.float32(D ** -0.5) * np.float32(1 + 2.0 ** -10) ** np.arange(700, dtype=np.float32)
    off = (s * np.float32(math.log2(math.e))).astype(np.float64) / (s.astype(np.float64) * math.log2(math.e)) - 1
    lo, hi = int(off.argmin()), int(off.argmax())
    return [(float(s[i]), off[i]) for i in (lo, hi)]


class Weights:
    """A call whose outputs are its weights."""

    def __init__(self, fmt, D):
        page, self.B, self.Hk, self.G, g = 16, 32, 2, 8, torch.Generator().manual_seed(D)
        self.D = self.n = D
        k = torch.randn(D // page, self.Hk, page, D, generator=g)
        v = torch.eye(D).view(D // page, 1, page, D).expand(-1, self.Hk, -1, -1)
        self.cache, keys, _ = cache_of(fmt, k, v.contiguous(), page)
        self.keys = keys.transpose(1, 0, 2, 3).reshape(self.Hk, D, D)
        self.ones = np.ones((self.Hk, D))
        if fmt != "bf16":  # the value of a one is code * step, 1 but for the step's rounding
            self.cache[3].copy_(1 / self.cache[1].float().amax(-1).double())
            self.ones = (self.cache[1].double().amax(-1) * self.cache[3].double()).transpose(0, 1).reshape(self.Hk, D).cpu().numpy()
        self.q = (torch.randn(self.B, self.Hk * self.G, D, generator=g) * 1.5).cuda()
        self.table = torch.arange(D // page, dtype=torch.int32, device="cuda").expand(self.B, -1).contiguous()
        self.lengths = torch.full((self.B,), D, dtype=torch.int32, device="cuda")

    def stretch(self, scale):
        out = torch.empty_like(self.q)
        bl.bitlinear_attention(self.q, self.cache, self.table, self.lengths, out, scale=scale)
        shape = (self.B, self.Hk, self.G, self.n)
        x = scale * np.einsum("bhgd,htd->bhgt", self.q.double().cpu().numpy().reshape(shape), self.keys)
        p = np.exp(x - x.max(-1, keepdims=True))
        p /= p.sum(-1, keepdims=True)
        off = np.log(out.double().cpu().numpy().reshape(shape) / (p * self.ones[None, :, None]))
        keep = p > p.max(-1, keepdims=True) * 2.0 ** -12   # below that an 8-bit cache's weight has fewer bits
        above = np.where(keep, x - (x * keep).sum(-1, keepdims=True) / keep.sum(-1, keepdims=True), 0.0)
        return (above * np.where(keep, off, 0.0)).sum() / (above * above).sum()


@pytest.mark.parametrize("fmt", plain.FORMATS)
@pytest.mark.parametrize("D", [64, 80, 128])
def test_scale_is_not_rounded(fmt, D):
    """What else stretches a logit does so at two near scales alike, so it falls out of the difference."""
    w, (down, up) = Weights(fmt, D), worst_scales(D)
    assert up[1] - down[1] > 1.5 * U   # what the difference would be
    stretches = [w.stretch(scale) / U for scale, _ in (down, up)]
    assert abs(stretches[1] - stretches[0]) <= 0.25, stretches


@pytest.mark.parametrize("fmt", plain.FORMATS)
@pytest.mark.parametrize("D", [64, 80, 128, 256])
def test_a_logits_sum_is_cut_once_per_16_dims(fmt, D):
    """The MMA's adder may cut a sum toward zero, by half a unit on average: U 2^e of a sum m 2^e, U times the mean of
    1 / m over 1 <= m < 2, the logarithm of m even: U / (2 ln 2) = 0.72 U of it.  The S = D / 16 sums of a logit x are
    s / S x on average: 0.72 U (S + 1) / 2 of x in all, where each is cut once."""
    stretch = Weights(fmt, D).stretch(D ** -0.5) / U
    assert abs(stretch) <= 0.75 * (D // 16 + 1) / 2, stretch
