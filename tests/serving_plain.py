"""The operators of a serving step written out plainly (numpy, 64 bits or whole numbers), and the bounds their fp32 forms keep."""
from fractions import Fraction

import numpy as np

from attention_plain import U, held


def head(q, k, v, s, scale):
    """(out [D], bound) of one q head over tokens k, v [t, D] (fp64), s [t] the values' steps or None: the bound of
    attention_plain.attend, derived there."""
    D = len(q)
    if len(k) == 0:
        return np.zeros(D), np.zeros(D)
    x = scale * (k @ q)
    w = np.exp(x - x.max())
    out = w @ v / w.sum()
    d = abs(scale) * (np.abs(k) @ np.abs(q)) * 2 * U * (D + 16)
    rel = np.expm1(2 * (d.max() + 8 * U + 2 * U * (x.max() - x).clip(0, 100).max())) + 2 * U * (len(x) + 64)
    bound = 2 * rel * (w @ np.abs(v)) / w.sum() + 1e-37
    if s is not None:
        codes = np.abs(v) / np.where(s > 0, s, 1.0)[:, None]
        bound = bound + 2.0 ** -36 * (w * s).max() * codes.sum(0) / w.sum()
    return out, bound


def attend_blocks(q, cache, table, lengths, blocks, page, scale):
    """-> (out [B, Hq, D], bound): attention over the listed pages' tokens."""
    keys, values = held(cache, "k"), held(cache, "v")
    steps = None if cache[3] is None else cache[3].double().cpu().numpy()
    B, Hq, D = q.shape
    Hkv = keys.shape[1]
    out, bound = np.zeros((B, Hq, D)), np.zeros((B, Hq, D))
    for b in range(B):
        for hk in range(Hkv):
            rows = []
            for j in blocks[b, hk]:
                if not 0 <= j < table.shape[1] or not 0 <= table[b, j] < keys.shape[0]:
                    continue
                rows += [(table[b, j], o) for o in range(page) if j * page + o < lengths[b]]
            p, o = (np.array(x, np.int64) for x in zip(*rows)) if rows else (np.zeros(0, np.int64),) * 2
            s = None if steps is None else steps[p, hk, o]
            for h in range(hk * Hq // Hkv, (hk + 1) * Hq // Hkv):
                out[b, h], bound[b, h] = head(np.asarray(q[b, h], np.float64), keys[p, hk, o], values[p, hk, o], s, scale)
    return out, bound


def summaries(cache, page_ids, filled):
    """Bounds [n, heads, 2, D] (int8) and steps [n, heads] (fp32) of the first filled[i] tokens of pages page_ids[i]."""
    k = cache[0].float().cpu().numpy()
    x = k if cache[2] is None else k * cache[2].float().cpu().numpy()[..., None]  # one fp32 product
    assert x.dtype == np.float32
    bounds, steps = [], []
    for p, n in zip(page_ids, filled):
        lo, hi = x[p, :, :n].min(1), x[p, :, :n].max(1)
        top = np.maximum(np.maximum(np.abs(lo), np.abs(hi)).max(-1), np.float32(1e-5))
        s = (np.float32(127) / top)[:, None]
        bounds.append(np.stack([np.maximum(np.floor(lo * s), -127), np.minimum(np.ceil(hi * s), 127)], 1).astype(np.int8))
        steps.append(top / np.float32(127))
    return np.stack(bounds), np.stack(steps)


def choose(q, bounds, steps, table, length, page, keep_first, keep_last, count):
    """The columns [heads, count] that are chosen for one sequence's q [Hq, D] (fp32)."""
    Hkv = bounds.shape[1]
    G = q.shape[0] // Hkv
    n = max(0, min(int(length), len(table) * page))
    pages = -(-n // page)
    out = np.full((Hkv, count), -1)
    for hk in range(Hkv):
        scored = []
        for j in range(pages):
            p = table[j]
            if not 0 <= p < bounds.shape[0]:
                continue
            best = []
            for h in range(hk * G, (hk + 1) * G):
                top = max(np.abs(q[h]).max(), np.float32(1e-5))
                codes = np.rint(q[h] * (np.float32(127) / top)).astype(np.int64)
                lo, hi = bounds[p, hk].astype(np.int64)
                acc = np.maximum(codes * lo, codes * hi).sum()
                best.append((np.float32(acc) * steps[p, hk]) * (top / np.float32(127)))
            score = np.inf if j < keep_first or j >= pages - keep_last else max(best)
            scored.append((-float(score), j))
        chosen = sorted(j for _, j in sorted(scored)[:count])
        out[hk, :len(chosen)] = chosen
    return out


def softmax(y, temperature):
    """-> (p, bound), rows of logits in fp64."""
    y = np.asarray(y, np.float64)
    t = np.ones(len(y)) if temperature is None else np.asarray(temperature, np.float64)
    out, bound = np.zeros_like(y), np.zeros_like(y)
    for m in range(len(y)):
        top = y[m].max()
        if top == -np.inf:
            continue
        if not t[m] >= 1e-30:
            out[m, np.argmax(y[m])] = 1.0
            continue
        T = min(t[m], 1e30)
        z = (y[m] - top) / T
        e = np.exp(z)
        out[m] = e / e.sum()
        # The argument of a power of two: a difference, log2(e) / T (two roundings) and a product, 4 U of |z|, twice (a
        # warp's maximum lies between), and as much for the sum's largest terms; the power itself 2^-22 (4 U), three times; the
        # sums: a chain of at most 64 + V / 2^14 additions and 30 joins; a division and three products.  What is below 2^-126 of
        # a warp's largest is 0.
        near = np.where(np.isfinite(z), np.abs(z), 0.0)
        rel = U * (12 * near + 12 + 12 * (out[m] * near).sum() + 64 + len(z) / 2 ** 14 + 40)
        bound[m] = 1.01 * out[m] * rel + 2.0 ** -125
    return out, bound


def units(w):
    """Weights as whole numbers of 2^-s, s = 62 - ceil(log2 of how many)."""
    s = 62 - (len(w) - 1).bit_length()
    w = np.where(np.asarray(w) > 0, np.minimum(np.asarray(w, np.float32), np.float32(2)), np.float32(0))  # NaN: 0
    return [int(x) for x in np.rint(w.astype(np.float64) * 2.0 ** s)]


def draw(w, r):
    """The first index whose running sum is above r times the whole, or -1."""
    w = units(w)
    total, r = sum(w), Fraction(min(max(float(r), 0.0), 1 - 2.0 ** -24) if r == r else 0.0)
    upto = 0
    for v, x in enumerate(w):
        upto += x
        if x and upto > r * total:
            return v
    return -1


def verify(p, q, draft, uniform):
    """-> (tokens [B, K + 1], accepted [B]) of fp32 probabilities, exactly."""
    B, K1, V = p.shape
    K = K1 - 1
    tokens, accepted = np.full((B, K1), -1), np.zeros(B, np.int64)
    for b in range(B):
        n, refused = 0, False
        while n < K:
            x = draft[b, n]
            if not 0 <= x < V:
                break
            if not float(uniform[b, n]) * float(q[b, n, x]) < float(p[b, n, x]):  # the product of two fp32 is exact
                refused = True
                break
            n += 1
        w = p[b, n]
        if refused:
            rest = p[b, n] - q[b, n]
            if sum(units(rest)) > 0:
                w = rest
        tokens[b, :n] = draft[b, :n] if n else 0
        tokens[b, n] = draw(w, uniform[b, K])
        accepted[b] = n
    return tokens, accepted
