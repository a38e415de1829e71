"""The attention operators written out plainly in 64 bits (numpy), and the bounds their fp32 forms keep.

U = 2^-24 is half a step of fp32 relative to a value (eps / 2)."""
import numpy as np
import torch

U = 2.0 ** -24
FORMATS = {"int8": torch.int8, "fp8": torch.float8_e4m3fn, "bf16": torch.bfloat16}
TOP = {"int8": 127.0, "fp8": 448.0}


def rotate(x, positions, freq, layout, amplitude=1.0):
    """x [T, H, D] -> (rotated rows, bound of an fp32 rotation's error), float64."""
    x = np.asarray(x, np.float64)
    n = len(freq)
    angle = np.asarray(positions, np.float64)[:, None] * np.asarray(freq, np.float64)[None, :]
    c, s = (amplitude * np.cos(angle))[:, None], (amplitude * np.sin(angle))[:, None]
    a_at, b_at = (np.arange(n), np.arange(n) + n) if layout == 0 else (2 * np.arange(n), 2 * np.arange(n) + 1)
    y, bound = x.copy(), np.zeros_like(x)
    a, b = x[..., a_at], x[..., b_at]
    y[..., a_at], y[..., b_at] = a * c - b * s, b * c + a * s
    # cosine and sine rounded (U), times the amplitude (itself an fp32 value: U, and the product U), one
    # product (U) and the sum (U): 5 U of each of the two terms; the angle to 8 steps of fp64
    size = amplitude * (np.abs(a) + np.abs(b))
    bound[..., a_at] = bound[..., b_at] = size * (5 * U + 8 * 2.0 ** -53 * np.abs(angle)[:, None])
    return y, bound


def places(positions, seq, table, page_size):
    """(page, offset) of each row, page -1 where the row has none."""
    page, at = np.full(len(positions), -1), np.zeros(len(positions), np.int64)
    for i, p in enumerate(positions):
        s = i if seq is None else int(seq[i])
        if p < 0 or not 0 <= s < table.shape[0] or p // page_size >= table.shape[1]:
            continue
        page[i], at[i] = table[s, p // page_size], p % page_size
    return page, at


def held(cache, name):
    """fp64 values of a whole cache tensor (k, v, k_step, v_step on any device)."""
    k, v, ks, vs = cache
    x, step = (k, ks) if name == "k" else (v, vs)
    x = x.float().double()
    return (x if step is None else x * step.double()[..., None]).cpu().numpy()


def attend(q, cache, table, lengths, page_size, scale, window=0):
    """-> (out [B, Hq, D], bound) over the cache's exact values, in float64."""
    keys, values = held(cache, "k"), held(cache, "v")
    steps = None if cache[3] is None else cache[3].double().cpu().numpy()
    B, Hq, D = q.shape
    Hkv, G = keys.shape[1], Hq // keys.shape[1]
    out, bound = np.zeros((B, Hq, D)), np.zeros((B, Hq, D))
    for b in range(B):
        n = min(int(lengths[b]), table.shape[1] * page_size)
        first = max(0, n - window) if window else 0
        rows = [(table[b, t // page_size], t % page_size) for t in range(first, n)]
        rows = [(p, o) for p, o in rows if 0 <= p < keys.shape[0]]
        if not rows:
            continue
        p, o = (np.array(x) for x in zip(*rows))
        K, V = keys[p, :, o], values[p, :, o]  # [t, Hkv, D]
        for h in range(Hq):
            k, v, qq = K[:, h // G], V[:, h // G], np.asarray(q[b, h], np.float64)
            x = scale * (k @ qq)
            w = np.exp(x - x.max())
            out[b, h] = w @ v / w.sum()
            # A logit: D products and sums and a handful of roundings, each at most 2 U (an adder that
            # truncates) of sum |q k|; an exponential and its argument: 8 U and 2 U |x - max|.  Both
            # sums: a rounding of at most 2 U a token and 64 more for the joins.
            d = abs(scale) * (np.abs(k) @ np.abs(qq)) * 2 * U * (D + 16)
            rel = np.expm1(2 * (d.max() + 8 * U + 2 * U * (x.max() - x).clip(0, 100).max())) + 2 * U * (len(x) + 64)
            bound[b, h] = 2 * rel * (w @ np.abs(v)) / w.sum() + 1e-37
            # 8-bit codes are weighted by p * step as two fp16 parts, in units that make the largest such
            # weight 1 or more.  Below 2^-14 the first part is subnormal (off by 2^-25), what it leaves,
            # times 2^11, is again (off by 2^-25 / 2^11): 2^-36 of the largest weight a token, times its code.
            if steps is not None:
                s = steps[p, h // G, o]
                codes = np.abs(v) / np.where(s > 0, s, 1.0)[:, None]
                bound[b, h] += 2.0 ** -36 * (w * s).max() * codes.sum(0) / w.sum()
    return out, bound


def make_cache(fmt, pages, heads, page_size, D, seed, device="cuda"):
    """A cache holding garbage that must not be read: NaN values or NaN steps."""
    g = torch.Generator().manual_seed(seed)
    shape = (pages, heads, page_size, D)
    if fmt == "bf16":
        return tuple(torch.full(shape, float("nan"), dtype=torch.bfloat16, device=device) for _ in "kv") + (None, None)
    codes = [torch.randint(0, 256, shape, generator=g, dtype=torch.uint8) for _ in "kv"]
    codes = [c.view(FORMATS[fmt]).to(device) for c in codes]
    steps = [torch.full(shape[:3], float("nan"), device=device) for _ in "kv"]
    return codes[0], codes[1], steps[0], steps[1]


def fill_row(cache, fmt, page, at, k, v):
    """Writes fp32 rows [T, heads, D] at (page, at), quantised by torch."""
    for i, x in enumerate((k, v)):
        if fmt == "bf16":
            cache[i][page, :, at] = x.to(torch.bfloat16)
            continue
        top = x.abs().amax(-1).clamp(min=1e-5)
        y = x * (TOP[fmt] / top)[..., None]
        if fmt == "int8":
            cache[i][page, :, at] = y.round().clamp(-128, 127).to(torch.int8)
        else:
            cache[i].view(torch.uint8)[page, :, at] = y.clamp(-448, 448).to(torch.float8_e4m3fn).view(torch.uint8)
        cache[2 + i][page, :, at] = top / TOP[fmt]
