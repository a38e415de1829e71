"""Shared prefixes on the tensor cores with several tiles a CTA, against 64 bits: the rings of pages, operands and logits go
round, references move late, tiles end short, pages are missing."""
import numpy as np
import pytest
import torch

import attention_plain
import bitlinear_w1_a8_gb300 as bl
from harness import check_canary, guarded
from serving_ways import way, wide_tiles

pytestmark = pytest.mark.gpu

U = attention_plain.U
FP8 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def built():
    bl.load_library()


def ints(values):
    return torch.as_tensor(np.asarray(values), dtype=torch.int32, device="cuda")


def quantised(x, fmt):
    """fp32 rows [..., D] -> codes and steps as the cache holds them."""
    if fmt == "bf16":
        return x.to(torch.bfloat16), None
    top = x.abs().amax(-1).clamp(min=1e-5)
    y = x * (attention_plain.TOP[fmt] / top)[..., None]
    return (y.round().clamp(-127, 127).to(torch.int8) if fmt == "int8" else y.clamp(-448, 448).to(FP8)), top / attention_plain.TOP[fmt]


def long_case(fmt, groups, R, Hq, Hkv, D, shared, lengths, page, columns, seed, missing):
    """Cache, q and page table on the GPU: keys that grow along the prefix under q heads that follow them, turn away from them or
    do neither; what no row attends to is NaN.  missing: every fourth tile lacks a part (a third of pages as
    large as tiles)."""
    g, rng = torch.Generator(device="cuda").manual_seed(seed), np.random.default_rng(seed)
    B = groups * R
    used = [-(-max(1, int(n)) // page) for n in lengths]
    whole = [-(-int(s) // page) for s in shared]
    pages = sum(whole) + sum(max(0, u - whole[b // R]) for b, u in enumerate(used)) + 3
    ids = iter(rng.permutation(pages).tolist())
    table = np.full((B, columns), -1)
    for i in range(groups):
        table[i * R:(i + 1) * R, :whole[i]] = [next(ids) for _ in range(whole[i])]
    for b in range(B):
        for j in range(whole[b // R], used[b]):
            table[b, j] = next(ids)
    at, there = torch.zeros(pages, page), torch.zeros(pages, page, dtype=torch.bool)
    for b in range(B):
        n = max(0, int(lengths[b]))
        t = np.arange(n)
        at[table[b, t // page], t % page] = torch.tensor(t / float(max(shared)), dtype=torch.float32)
        there[table[b, t // page], t % page] = True
    if missing:
        first = np.arange(columns) * page
        gone = (first // 128 % 4 == 3) & (first % 128 >= 64) if page < 128 else np.arange(columns) % 3 == 1
        gone[max(0, int(max(shared)) // page):] = False
        table[:, gone] = np.where(rng.random(gone.sum()) < 0.5, -1, 10 ** 8)
    at, there = at.cuda(), there.cuda()
    parts = []
    for name in "kv":
        x = torch.randn(pages, Hkv, page, D, generator=g, device="cuda") * 0.7
        if name == "k":
            x += 12.0 * D ** -0.5 * at[:, None, :, None]
        codes, step = quantised(x, fmt)
        if fmt == "bf16":
            codes.masked_fill_(~there[:, None, :, None], float("nan"))
        else:
            garbage = torch.randint(0, 256, codes.shape, generator=g, dtype=torch.uint8, device="cuda")
            codes = torch.where(there[:, None, :, None], codes.view(torch.uint8), garbage).view(codes.dtype)
            step = torch.where(there[:, None], step, float("nan"))
        parts += [(codes, step)]
    (k, ks), (v, vs) = parts
    q = torch.randn(B, Hq, D, generator=g, device="cuda") * 1.5
    # logits that rise by 48 (69 bits) along the prefix, fall as much, or stay
    q += (torch.arange(Hq, device="cuda") % 3 - 1)[None, :, None] * 4.0
    return (k, v, ks, vs), q, table


def row_in_64_bits(q, cache, table, n, shared, page, scale):
    """attention_plain.attend of one row of length n, all heads at once on the GPU: (out, bound) [Hq, D].  shared: the
    tokens that its group shares and has."""
    k, v, ks, vs = cache
    Hkv, D = k.shape[1], k.shape[3]
    table = torch.as_tensor(table, device="cuda").long()

    def places(n):
        t = torch.arange(n, device="cuda")
        p = table[t // page]
        return (x[(p >= 0) & (p < k.shape[0])] for x in (t, p))

    t, p = places(n)
    if len(t) == 0:
        return torch.zeros_like(q, dtype=torch.float64), torch.zeros_like(q, dtype=torch.float64)
    take = lambda x: x.view(torch.uint8)[p, :, t % page].view(FP8).double() if x.dtype == FP8 else x[p, :, t % page].double()  # noqa: E731
    K, V = (take(x).transpose(0, 1) for x in (k, v))           # [Hkv, t, D]
    steps = None if ks is None else vs[p, :, t % page].double().T  # [Hkv, t]
    codes = V.abs()
    if steps is not None:
        K, V = K * ks[p, :, t % page].double().T[..., None], V * steps[..., None]
    qq = q.double().view(Hkv, -1, D)
    x = scale * (qq @ K.transpose(1, 2))
    top = x.amax(-1, keepdim=True)
    w = (x - top).exp()
    total = w.sum(-1, keepdim=True)
    out = w @ V / total
    d = abs(scale) * (qq.abs() @ K.abs().transpose(1, 2)) * 2 * U * (D + 16)
    rel = torch.expm1(2 * (d.amax(-1, keepdim=True) + 8 * U + 2 * U * (top - x).clamp(0, 100).amax(-1, keepdim=True))) + 2 * U * (len(t) + 64)
    bound = 2 * rel * (w @ V.abs()) / total + 1e-37
    if steps is not None:
        bound = bound + 2.0 ** -36 * (w * steps[:, None]).amax(-1, keepdim=True) * codes.sum(1)[:, None] / total
    else:  # a bf16 value is off by 2^-39 of the largest of its tile
        s, p = places(max(n, shared))
        tile, of_tile = t // 128, (s // 128).expand(Hkv, -1)
        largest = torch.zeros(Hkv, int(s.max()) // 128 + 1, dtype=torch.float64, device="cuda")
        largest = largest.scatter_reduce(1, of_tile, v[p, :, s % page].double().abs().amax(-1).T.contiguous(), "amax")
        bound = bound + 1.01 * 2.0 ** -39 * (w @ largest.gather(1, tile.expand(Hkv, -1))[..., None]) / total
    return out.view(q.shape), bound.view(q.shape)


CASES = {  # format-free sizes, and the fewest and most tiles a CTA that they give
    "a tile of q heads a row, equal runs": (dict(groups=5, R=24, Hq=64, Hkv=16, D=64, S=1300, own=20, page=64), 5, 12),
    "three, runs by the tokens": (dict(groups=2, R=33, Hq=64, Hkv=8, D=128, S=2609, own=9, page=32), 5, 9),
    "one group, twenty tiles": (dict(groups=1, R=16, Hq=280, Hkv=40, D=80, S=128 * 58 - 5, own=40, page=64), 20, 20),
    "pages of 16, a last tile of 16 q heads": (dict(groups=3, R=48, Hq=39, Hkv=13, D=112, S=641, own=17, page=16), 5, 6),
    "pages of 512": (dict(groups=4, R=30, Hq=80, Hkv=20, D=96, S=1281, own=5, page=512), 6, 11),
    "pages of 128, narrow heads": (dict(groups=2, R=26, Hq=160, Hkv=40, D=16, S=1535, own=3, page=128), 6, 12),
}


@pytest.mark.parametrize("fmt", attention_plain.FORMATS)
@pytest.mark.parametrize("missing", [False, True])
@pytest.mark.parametrize("name", CASES)
def test_many_tiles_a_cta(fmt, missing, name):
    c, fewest, most = CASES[name]
    groups, R, Hq, Hkv, D, S, own, page = (c[k] for k in ("groups", "R", "Hq", "Hkv", "D", "S", "own", "page"))
    rng = np.random.default_rng(S)
    shared = np.array([S] + [int(rng.integers(S * 3 // 4, S + 1)) for _ in range(groups - 1)])
    lengths = np.repeat(shared, R) + rng.integers(0, own + 1, groups * R)
    lengths[3::7] = rng.integers(1, S, len(lengths[3::7]))  # rows that do not have all of their group's tokens
    lengths[5] = 0
    columns = -(-(S + own) // page)
    assert way(fmt, groups, R, Hq, Hkv, D, columns, page) == "wide"
    tiles = wide_tiles(groups, R, Hq, Hkv, shared, columns, page)
    assert fewest <= max(tiles) <= most, tiles
    cache, q, table = long_case(fmt, groups, R, Hq, Hkv, D, shared, lengths, page, columns, S + missing, missing)
    out, full = guarded(q.numel(), torch.float32, 7.5)
    out = out.view(q.shape)
    ws, ws_full = guarded(bl.bitlinear_attention_shared_workspace(groups * R, Hq, Hkv, D, groups), torch.uint8, 0x5a)
    out.fill_(float("nan"))
    bl.bitlinear_attention_shared(q, cache, ints(table), ints(lengths), ints(shared), out, ws)
    torch.cuda.synchronize()
    check_canary(full, 7.5)
    check_canary(ws_full, 0x5a)
    assert torch.isfinite(out).all() and bl.bitlinear_device_status() == 0
    for b in range(groups * R):
        group = slice(b // R * R, b // R * R + R)
        has = min(int(shared[b // R]), int(lengths[group].max()))
        want, bound = row_in_64_bits(q[b], cache, table[b], int(lengths[b]), has, page, D ** -0.5)
        off = (out[b].double() - want).abs() - bound
        assert (off <= 0).all(), f"row {b} of length {lengths[b]}: worst by {off.max().item():.3g}, {(off > 0).sum().item()} of {off.numel()}"


@pytest.mark.parametrize("fmt", attention_plain.FORMATS)
@pytest.mark.parametrize("page,groups,R,D,S,columns", [(512, 2, 40, 128, 1300, 4), (32, 60, 130, 32, 130, 16), (16, 3, 70, 112, 300, 64)])
def test_tile_counts_of_short_prefixes(fmt, page, groups, R, D, S, columns):
    """Two groups by their tokens; many with one CTA a row; pages of 16: wider tables make the call take the tensor cores."""
    Hq, Hkv, own = 4, 2, 19
    rng = np.random.default_rng(page)
    shared = rng.integers(S // 2, S + 1, groups)
    shared[-1] = S
    lengths = np.repeat(shared, R) + rng.integers(0, own + 1, groups * R)
    if way(fmt, groups, R, Hq, Hkv, D, columns, page) == "alone":
        columns = 36_000_001 * 2 // (groups * R * page * Hkv * D * 2 * (2 if fmt == "bf16" else 1)) + 1
    assert way(fmt, groups, R, Hq, Hkv, D, columns, page) == "wide"
    cache, q, table = long_case(fmt, groups, R, Hq, Hkv, D, shared, lengths, page, columns, S, False)
    out = torch.full_like(q, float("nan"))
    ws = torch.empty(bl.bitlinear_attention_shared_workspace(groups * R, Hq, Hkv, D, groups), dtype=torch.uint8, device="cuda")
    bl.bitlinear_attention_shared(q, cache, ints(table), ints(lengths), ints(shared), out, ws)
    assert torch.isfinite(out).all() and bl.bitlinear_device_status() == 0
    for b in range(0, groups * R, max(1, groups * R // 200)):
        want, bound = row_in_64_bits(q[b], cache, table[b], int(lengths[b]), int(shared[b // R]), page, D ** -0.5)
        assert ((out[b].double() - want).abs() <= bound).all(), b


@pytest.mark.parametrize("fmt", attention_plain.FORMATS)
def test_many_tiles_do_not_depend_on_timing(fmt):
    """The same bits in calls that run beside copies of large buffers, which slow the cache's rows down."""
    c, _, _ = CASES["one group, twenty tiles"]
    groups, R, Hq, Hkv, D, S, own, page = (c[k] for k in ("groups", "R", "Hq", "Hkv", "D", "S", "own", "page"))
    lengths, shared, columns = S + np.arange(R) % own, np.array([S]), -(-(S + own) // page)
    cache, q, table = long_case(fmt, groups, R, Hq, Hkv, D, shared, lengths, page, columns, 5, True)
    ws = torch.empty(bl.bitlinear_attention_shared_workspace(R, Hq, Hkv, D, 1), dtype=torch.uint8, device="cuda")
    args = q, cache, ints(table), ints(lengths), ints(shared)
    alone, outs = torch.empty_like(q), [torch.empty_like(q) for _ in range(20)]
    bl.bitlinear_attention_shared(*args, alone, ws)
    large, other = torch.empty(1 << 28, device="cuda"), torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(other):
        for _ in range(12):
            large[1 << 27:].copy_(large[:1 << 27])
    for out in outs:
        bl.bitlinear_attention_shared(*args, out, ws)
    torch.cuda.synchronize()
    for out in outs:
        assert torch.equal(out, alone)
