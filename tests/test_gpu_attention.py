"""Rotary positions, the paged key-value cache and attention over it, on the GPU, against plain 64-bit forms."""
import math

import numpy as np
import pytest
import torch

import attention_plain as plain
import bitlinear_w1_a8_gb300 as bl
from harness import check_canary, guarded

pytestmark = pytest.mark.gpu

U = plain.U
LAYOUTS = {"half": bl.ROPE_HALF, "interleaved": bl.ROPE_INTERLEAVED}


@pytest.fixture(scope="module", autouse=True)
def built():
    bl.load_library()


def normal(shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g) * std


def ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def within(got, want, bound):
    got = got.double().cpu().numpy() if isinstance(got, torch.Tensor) else np.asarray(got, np.float64)
    assert np.isfinite(got).all()
    off = np.abs(got - want) - bound
    assert (off <= 0).all(), f"{(off > 0).sum()} of {off.size} beyond the bound, worst by {off.max():.3g}"


# ------------------------------------------------------------------ rotary positions


@pytest.mark.parametrize("layout", LAYOUTS)
@pytest.mark.parametrize("T,H,D,rot", [(1, 1, 4, 2), (1, 32, 80, 80), (3, 5, 128, 64), (7, 20, 128, 128), (130, 3, 96, 34),
                                       (2, 1, 256, 256), (5, 40, 64, 30), (1000, 2, 36, 36)])
def test_rope(T, H, D, rot, layout):
    x = normal((T, H, D), 10 + T)
    rng = np.random.default_rng(T + D)
    pos = rng.integers(0, 2 ** 31 - 1, T)
    pos[: T // 2] = rng.integers(0, 5000, T // 2)
    pos[-1] = 0 if T > 1 else 2047
    freq = bl.bitlinear_rope_frequencies(rot)
    y, full = guarded(T * H * D, torch.float32, 5.5)
    y = y.view(T, H, D)
    bl.bitlinear_rope(x.cuda(), ints(pos.tolist()), (freq.cuda(), LAYOUTS[layout], 1.25), y)
    want, bound = plain.rotate(x.numpy(), pos, freq.numpy(), LAYOUTS[layout], 1.25)
    within(y, want, bound)
    check_canary(full, 5.5)
    assert torch.equal(y[..., rot:].cpu(), x[..., rot:])


def test_rope_in_place_strided_and_back():
    T, H, D, rot = 37, 6, 80, 48
    wide = normal((T, 3 * H * D), 3).cuda()
    keep = wide.clone()
    x = wide[:, H * D:2 * H * D].unflatten(1, (H, D))  # the middle third of a wider row
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 911
    freq = bl.bitlinear_rope_frequencies(rot, scaling=bl.ROPE_SCALE_PARTS, factor=8.0, original_length=2048.0)
    spec = (freq.cuda(), bl.ROPE_HALF)
    bl.bitlinear_rope(x, pos, spec, x)
    want, bound = plain.rotate(keep[:, H * D:2 * H * D].unflatten(1, (H, D)).cpu().numpy(), pos.cpu().numpy(), freq.numpy(), 0)
    within(x, want, bound)
    assert torch.equal(wide[:, :H * D], keep[:, :H * D]) and torch.equal(wide[:, 2 * H * D:], keep[:, 2 * H * D:])
    # the gradient's rotation: by the negative position the rows come back
    bl.bitlinear_rope(x, -pos, spec, x)
    back = keep[:, H * D:2 * H * D].unflatten(1, (H, D)).cpu().numpy()
    _, again = plain.rotate(want, -pos.cpu().numpy(), freq.numpy(), 0)
    n = rot // 2
    carried = np.zeros_like(bound)
    carried[..., :n] = carried[..., n:rot] = bound[..., :n] + bound[..., n:rot]  # |c|, |s| <= 1
    within(x, back, again + carried)


@pytest.mark.parametrize("T,H,D,rot,layout", [(12001, 9, 80, 80, "half"), (10007, 33, 32, 16, "interleaved"), (11003, 5, 64, 20, "half")])
def test_rope_of_many_tokens(T, H, D, rot, layout):
    """Warps in several rounds, whose rows are asked for early: in place, rows apart, the last row at the end of its memory."""
    wide = normal((T * (H * D + 4) - 4,), T).cuda()
    x = wide.as_strided((T, H, D), (H * D + 4, D, 1))
    before, keep = x.cpu().numpy(), wide.clone()
    pos = torch.arange(T, dtype=torch.int32, device="cuda") * 7
    freq = bl.bitlinear_rope_frequencies(rot)
    y = torch.empty(T, H, D, device="cuda")
    bl.bitlinear_rope(x, pos, (freq.cuda(), LAYOUTS[layout]), y)
    want, bound = plain.rotate(before, pos.cpu().numpy(), freq.numpy(), LAYOUTS[layout])
    within(y, want, bound)
    assert torch.equal(wide, keep)
    bl.bitlinear_rope(x, pos, (freq.cuda(), LAYOUTS[layout]), x)
    assert torch.equal(x, y)
    between = torch.ones_like(wide, dtype=torch.bool)
    between.as_strided((T, H, D), (H * D + 4, D, 1)).fill_(False)
    assert torch.equal(wide[between], keep[between])


def test_rope_is_the_gradient_of_itself():
    """d/dx of sum(g * rope(x, p)) is rope(g, -p): against differences of the 64-bit form."""
    T, H, D = 2, 1, 8
    x, g = normal((T, H, D), 1).numpy().astype(np.float64), normal((T, H, D), 2)
    pos, freq = np.array([5, 977]), bl.bitlinear_rope_frequencies(D)
    dx = torch.empty(T, H, D, device="cuda")
    bl.bitlinear_rope(g.cuda(), ints((-pos).tolist()), (freq.cuda(), bl.ROPE_INTERLEAVED), dx)
    want, bound = plain.rotate(g.numpy(), -pos, freq.numpy(), 1)
    within(dx, want, bound)
    diff, h = np.zeros_like(x), 2.0 ** -10
    for i in np.ndindex(*x.shape):
        up, down = x.copy(), x.copy()
        up[i] += h
        down[i] -= h
        diff[i] = ((plain.rotate(up, pos, freq.numpy(), 1)[0] - plain.rotate(down, pos, freq.numpy(), 1)[0]) * g.numpy()).sum() / (2 * h)
    # linear in x: the differences are exact but for fp64 rounding of O(10) values over 2h
    within(dx, diff, bound + 64 * 2.0 ** -53 / h)


# ------------------------------------------------------------------ writing and reading the cache


def append_case(fmt, T, Hq, Hk, D, page, seed, rope=True, in_place=False):
    rng = np.random.default_rng(seed)
    num_seqs, max_pages = 5, 6
    table = rng.permutation(num_seqs * max_pages + 3)[: num_seqs * max_pages].reshape(num_seqs, max_pages)
    table[1, 2], table[2, 0], table[3, 1] = -1, 10 ** 6, num_seqs * max_pages + 3  # pages that do not exist
    all_places = [(s, p) for s in range(num_seqs) for p in range(max_pages * page)]
    picked = [all_places[i] for i in rng.choice(len(all_places), T, replace=False)]
    seq, pos = np.array([s for s, _ in picked]), np.array([p for _, p in picked])
    if T > 6:
        pos[1], seq[2], seq[3], pos[4] = -1, -1, num_seqs, max_pages * page  # padding and rows out of range
    cache = plain.make_cache(fmt, num_seqs * max_pages + 3, Hk, page, D, seed)
    before = [None if c is None else c.clone() for c in cache]
    q, k, v = normal((T, Hq, D), seed), normal((T, Hk, D), seed + 1), normal((T, Hk, D), seed + 2, 3.0)
    k[0], v[-1, 0] = 0.0, 1e-7  # a row of zeros, one below the floor of the step
    freq = bl.bitlinear_rope_frequencies(D - 16 if D > 32 else D)
    spec = (freq.cuda(), bl.ROPE_HALF) if rope else None
    qd = q.cuda()
    q_out = qd if in_place else torch.full_like(qd, -9.0)
    bl.bitlinear_kv_append(k.cuda(), v.cuda(), cache, ints(pos.tolist()), ints(table.tolist()), seq=ints(seq.tolist()),
                           q=qd if Hq else None, q_out=q_out if Hq else None, rope=spec)
    page_of, at = plain.places(pos, seq, table, page)
    ok = (page_of >= 0) & (page_of < num_seqs * max_pages + 3)
    assert ok.sum() < T or T <= 6
    n = freq.numpy() if rope else np.zeros(0)
    qr, q_bound = plain.rotate(q.numpy(), pos, n, 0)
    kr, k_bound = plain.rotate(k.numpy(), pos, n, 0)
    if Hq:
        within(q_out[ok], qr[ok], q_bound[ok])
        untouched = q if in_place else torch.full_like(q, -9.0)
        assert torch.equal(q_out[~ok].cpu(), untouched[~ok])
    # every byte of the cache outside the written rows is as it was
    mask = torch.zeros(cache[0].shape[0], page, dtype=torch.bool)
    mask[page_of[ok], at[ok]] = True
    mask = mask[:, None].expand(-1, Hk, -1).cuda()
    for now, was in zip(cache, before):
        if now is not None:
            raw = (lambda t: t.view(torch.uint8 if t.element_size() == 1 else torch.int16 if t.element_size() == 2 else torch.int32))
            assert torch.equal(raw(now)[~mask], raw(was)[~mask])
    for i, (x, bound) in enumerate(((kr, k_bound), (v.numpy().astype(np.float64), np.zeros(v.shape)))):
        x, bound = x[ok], bound[ok]
        got = cache[i].float()[page_of[ok], :, at[ok]].double().cpu().numpy()
        if fmt == "bf16":
            within(got, x, bound + (np.abs(x) + bound) * 2.0 ** -8 + 1e-38)
            continue
        top, slack = np.abs(x).max(-1, keepdims=True).clip(1e-5), bound.max(-1, keepdims=True)
        step = cache[2 + i][page_of[ok], :, at[ok]].double().cpu().numpy()[..., None]
        within(step, top / plain.TOP[fmt], (slack + 2 * U * top) / plain.TOP[fmt])
        y = x * plain.TOP[fmt] / top
        # scale and product rounded (2 U of it), the row's maximum and the value off by their rotations
        near = 3 * U * np.abs(y) + plain.TOP[fmt] / top * (bound + slack * np.abs(x) / top) * (1 + 4 * U)
        if fmt == "int8":
            within(got, y, 0.5 + near)
        else:  # half a step of e4m3: 2^-4 of a normal value, 2^-10 below 2^-6
            within(got, y, near + np.maximum((np.abs(y) + near) * 2.0 ** -4, 2.0 ** -10))
    return cache, table, ok


@pytest.mark.parametrize("fmt", plain.FORMATS)
@pytest.mark.parametrize("T,Hq,Hk,D,page", [(1, 32, 32, 80, 64), (9, 4, 1, 128, 16), (64, 0, 5, 96, 32), (150, 6, 3, 64, 128),
                                            (11, 2, 2, 256, 16), (8, 3, 3, 16, 4096), (33, 16, 2, 112, 16)])
def test_append(fmt, T, Hq, Hk, D, page):
    append_case(fmt, T, Hq, Hk, D, page, seed=T + D)


@pytest.mark.parametrize("fmt", plain.FORMATS)
def test_append_unrotated_and_in_place(fmt):
    append_case(fmt, 40, 4, 2, 80, 16, seed=5, rope=False)
    append_case(fmt, 40, 4, 2, 80, 16, seed=6, in_place=True)


@pytest.mark.parametrize("D", [64, 128, 192])
def test_int8_codes_follow_quant_act(D):
    """bit for bit the rule with s = 127 * (1 / a); quant_act's s is 127 / a, a step of fp32 away at most, so its
    codes differ only where x * s comes within 127 * 4 U of a border."""
    T, H = 6, 3
    cache = plain.make_cache("int8", 6, H, 16, D, 1)
    k, v = normal((T, H, D), 8).cuda(), normal((T, H, D), 9, 20.0).cuda()
    bl.bitlinear_kv_append(k, v, cache, ints([3] * T), ints([[i] for i in range(T)]))
    xq = torch.empty(T * H, D, dtype=torch.int8, device="cuda")
    sx = torch.empty(T * H, device="cuda")
    for i, x in enumerate((k, v)):
        codes = cache[i][:, :, 3]
        a = x.abs().amax(-1, keepdim=True).clamp(min=1e-5)
        assert torch.equal(codes, (x * (a.reciprocal() * 127)).round().clamp(-128, 127).to(torch.int8))
        np.testing.assert_array_equal(cache[2 + i][:, :, 3].cpu().numpy(), a[..., 0].cpu().numpy() / np.float32(127))
        bl.bitlinear_quant_act(x.view(T * H, D), xq, sx)
        other = codes != xq.view(T, H, D)
        y = x.double() * 127 / a.double()
        assert ((y - y.floor() - 0.5).abs()[other] <= 127 * 4 * U).all()


@pytest.mark.parametrize("fmt", plain.FORMATS)
@pytest.mark.parametrize("T,H,D,page", [(1, 1, 16, 16), (5, 32, 80, 64), (77, 5, 128, 16), (33, 2, 256, 32)])
def test_read(fmt, T, H, D, page):
    rng = np.random.default_rng(T)
    cache = plain.make_cache(fmt, 12, H, page, D, T)
    table = rng.permutation(12).reshape(3, 4)
    table[1, 1] = 12
    seq, pos = rng.integers(0, 3, T), rng.integers(0, 4 * page, T)
    if T > 4:
        pos[0], seq[1] = -5, 3
    page_of, at = plain.places(pos, seq, table, page)
    ok = (page_of >= 0) & (page_of < 12)
    for p, a in zip(page_of[ok], at[ok]):
        plain.fill_row(cache, fmt, p, a, normal((H, D), int(p) * 100 + int(a)).cuda(), normal((H, D), int(p) * 77 + int(a), 4.0).cuda())
    wide = torch.full((2, T, 2 * H * D + 4), 3.25, device="cuda")  # rows of another stride than their length
    outs = [w[:, 4:4 + H * D].unflatten(1, (H, D)) for w in wide]
    bl.bitlinear_kv_read(cache, ints(pos.tolist()), ints(table.tolist()), outs[0], outs[1], seq=ints(seq.tolist()))
    for i, out in enumerate(outs):
        codes = cache[i].float()[page_of[ok], :, at[ok]]
        want = codes if fmt == "bf16" else codes * cache[2 + i][page_of[ok], :, at[ok]][..., None]
        assert torch.equal(out[ok], want)                       # one fp32 product
        assert (out[~ok] == 3.25).all()
    assert (wide[:, :, :4] == 3.25).all() and (wide[:, :, 4 + H * D:] == 3.25).all()


def test_empty_calls_touch_nothing():
    cache = plain.make_cache("int8", 2, 2, 16, 64, 0)
    none, table = torch.empty(0, 2, 64, device="cuda"), ints([[0, 1]])
    bl.bitlinear_rope(none, ints([]), (torch.ones(32, dtype=torch.float64, device="cuda"), 0), none)
    bl.bitlinear_kv_append(none, none, cache, ints([]), table)
    bl.bitlinear_kv_read(cache, ints([]), table, none, none)
    bl.bitlinear_attention(none, cache, table[:0], ints([]), none)
    assert torch.isnan(cache[2]).all() and torch.isnan(cache[3]).all()


# ------------------------------------------------------------------ attention


def attend_case(fmt, Hq, Hk, D, page, lengths, window=0, seed=0, value_std=1.0, value_mean=0.0, workspace=False,
                bad_page=None, key_std=1.0, scale=None, spread_steps=False, columns=0):
    """A cache filled to each sequence's length, garbage everywhere else (and in the table's columns past
    the longest sequence, at least `columns` in all); -> the output."""
    B, width = len(lengths), max(1, -(-max(1, max(lengths)) // page)) + 1
    rng = np.random.default_rng(seed)
    pages = B * width + 2
    table = rng.permutation(pages)[: B * width].reshape(B, width)
    cache = plain.make_cache(fmt, pages, Hk, page, D, seed)
    g = torch.Generator(device="cuda").manual_seed(seed)
    for b, n in enumerate(lengths):
        n = max(0, n)
        k = torch.randn(n, Hk, D, generator=g, device="cuda") * key_std
        v = torch.randn(n, Hk, D, generator=g, device="cuda") * value_std + value_mean
        if spread_steps:
            v *= torch.exp(torch.randn(n, Hk, 1, generator=g, device="cuda") * 4)
        t = torch.arange(n, device="cuda")
        at = torch.tensor(table[b], device="cuda")[t // page]
        plain.fill_row(cache, fmt, at, t % page, k, v)
    if bad_page is not None:
        table[bad_page] = [-1, pages, 10 ** 9][seed % 3]
    if columns > width:
        table = np.concatenate([table, rng.integers(-2 ** 31, 2 ** 31 - 1, (B, columns - width))], 1)
    q = torch.randn(B, Hq, D, generator=g, device="cuda") * 1.5
    out, full = guarded(B * Hq * D, torch.float32, -7.0)
    out = out.view(B, Hq, D)
    need = bl.bitlinear_attention_workspace(B, Hq, Hk, D) if workspace else 0
    ws, ws_full = guarded(need, torch.uint8, 0x3C) if need else (None, None)
    bl.bitlinear_attention(q, cache, ints(table.tolist()), ints(lengths), out, workspace=ws, window=window, scale=scale)
    want, bound = plain.attend(q.cpu().numpy(), cache, table, lengths, page,
                               D ** -0.5 if scale is None else scale, window)
    within(out, want, bound)
    check_canary(full, -7.0)
    if need:
        check_canary(ws_full, 0x3C)
    return out


@pytest.mark.parametrize("fmt", plain.FORMATS)
@pytest.mark.parametrize("D", [16, 32, 48, 64, 80, 96, 112, 128, 144, 192, 256])
def test_attention_every_head_size(fmt, D):
    attend_case(fmt, 2, 2, D, 16, [1, 33, 0, 70], seed=D)


@pytest.mark.parametrize("fmt", plain.FORMATS)
@pytest.mark.parametrize("Hq,Hk", [(1, 1), (3, 1), (8, 2), (14, 2), (16, 2), (9, 1), (40, 5), (32, 1)])
def test_attention_shared_heads(fmt, Hq, Hk):
    attend_case(fmt, Hq, Hk, 64, 32, [45, 1, 130], seed=Hq)


@pytest.mark.parametrize("fmt", plain.FORMATS)
@pytest.mark.parametrize("page", [16, 64, 4096])
def test_attention_lengths_around_every_border(fmt, page):
    lengths = [0, 1, 2, 7, 8, 9, 15, 16, 17, 31, 32, 33, 47, 48, 63, 64, 65, 127, 128, 129, 255, 257, 511, 513, -3]
    attend_case(fmt, 4, 2, 80, page, lengths, seed=page)


@pytest.mark.parametrize("fmt", plain.FORMATS)
@pytest.mark.parametrize("window", [1, 15, 16, 33, 100, 10 ** 6])
def test_attention_window(fmt, window):
    attend_case(fmt, 4, 2, 96, 16, [1, 16, 17, 40, 99, 100, 101, 300], window=window, seed=window % 97)


@pytest.mark.parametrize("fmt", plain.FORMATS)
@pytest.mark.parametrize("seed", [0, 1, 2])
def test_attention_pages_out_of_range_are_masked(fmt, seed):
    out = attend_case(fmt, 4, 4, 64, 16, [100, 16, 40], bad_page=([0, 0, 1, 2], [0, 3, 0, 1]), seed=seed)
    assert (out[1] == 0).all()  # its only page is out of range


@pytest.mark.parametrize("fmt", plain.FORMATS)
def test_attention_long_and_ragged(fmt):
    attend_case(fmt, 8, 2, 128, 64, [5000, 3, 1025, 2048, 4097], seed=1, workspace=True)
    attend_case(fmt, 2, 1, 80, 16, [9001], seed=2, workspace=True)
    attend_case(fmt, 2, 1, 80, 16, [9001], seed=3)
    attend_case(fmt, 4, 4, 64, 32, [1 + 37 * i % 900 for i in range(70)], seed=4)


@pytest.mark.parametrize("fmt", plain.FORMATS)
@pytest.mark.parametrize("Hq,Hk,D,page,lengths,window", [
    (8, 1, 16, 16, [5000, 0, 3, 2049], 0), (1, 1, 256, 64, [2600], 0), (24, 3, 48, 32, [4000, 10], 0), (5, 5, 96, 16, [8000], 0),
    (32, 32, 80, 64, [4100], 0), (16, 2, 112, 4096, [9000], 2500), (7, 1, 128, 16, [0], 0), (4, 2, 64, 64, [4096, 4097, 4095, 1], 4096)])
def test_attention_one_cluster_a_row(fmt, Hq, Hk, D, page, lengths, window):
    """Long sequences of few heads without a workspace: the largest clusters."""
    attend_case(fmt, Hq, Hk, D, page, lengths, window=window, seed=Hq + D, columns=16384 // page)


# A table wide enough that a call with a workspace cuts one line through all sequences and heads.
WIDE = 1 << 16


@pytest.mark.parametrize("fmt", plain.FORMATS)
@pytest.mark.parametrize("Hq,Hk,D,page,lengths,window", [
    (4, 1, 128, 64, [3000], 0), (8, 8, 80, 16, [5], 0), (2, 2, 64, 32, [0, 0, 700, 0, 1, 33, 2050, 0], 0),
    (18, 2, 96, 16, [900, 0, 31, 32, 33, 1], 0), (5, 5, 112, 64, [1500, 64, 4097], 0), (4, 2, 256, 16, [513, 2000], 0),
    (4, 4, 80, 64, [4000, 3999, 17, 0, 250], 700), (8, 1, 32, 128, [9000, 100], 33), (2, 1, 64, 16, [0, 0], 0),
    (3, 1, 128, 4096, [10000, 1, 5000], 0)])
def test_attention_as_one_line(fmt, Hq, Hk, D, page, lengths, window):
    attend_case(fmt, Hq, Hk, D, page, lengths, window=window, seed=len(lengths) + D, workspace=True, columns=WIDE * 16 // page)


@pytest.mark.parametrize("fmt", plain.FORMATS)
def test_attention_as_one_line_of_many_short_rows(fmt):
    lengths = [(37 * i) % 90 for i in range(300)]
    attend_case(fmt, 4, 2, 64, 16, lengths, seed=1, workspace=True, columns=WIDE // 16)
    attend_case(fmt, 4, 4, 80, 16, lengths[:100], seed=2, workspace=True, columns=WIDE // 16,
                bad_page=([3, 3, 4, 99], [0, 1, 0, 2]))


@pytest.mark.parametrize("fmt", plain.FORMATS)
def test_attention_values_of_one_sign_and_peaked_rows(fmt):
    attend_case(fmt, 4, 1, 128, 64, [3000], seed=5, value_mean=10.0)             # long sums of one sign
    attend_case(fmt, 4, 1, 64, 16, [700, 90], seed=6, key_std=12.0)              # one token takes nearly all
    attend_case(fmt, 4, 1, 64, 16, [300, 31], seed=7, scale=0.0)                 # every token counts the same
    attend_case(fmt, 4, 1, 64, 16, [300, 31], seed=8, scale=-0.5)
    attend_case(fmt, 4, 1, 96, 16, [600, 100], seed=9, value_std=1e4, spread_steps=True)   # steps of many sizes
    attend_case(fmt, 4, 1, 96, 16, [600, 100], seed=10, value_std=1e-3, spread_steps=True)


@pytest.mark.parametrize("fmt", plain.FORMATS)
def test_attention_over_rows_of_zeros(fmt):
    """Rows never written in a cache of zeros: keys and values of 0 (steps of 0), which count in the sum."""
    B, H, D, page = 3, 2, 64, 16
    cache = tuple(None if c is None else torch.zeros_like(c) for c in plain.make_cache(fmt, 12, H, page, D, 0))
    table = np.arange(12).reshape(3, 4)
    t = torch.tensor([5, 40, 41], device="cuda")
    for b, rows in ((1, t[:1]), (2, t)):
        plain.fill_row(cache, fmt, torch.tensor(table[b], device="cuda")[rows // page], rows % page,
                       normal((len(rows), H, D), b).cuda() * 30, normal((len(rows), H, D), b + 5).cuda())
    q, out = normal((B, 2 * H, D), 3).cuda(), torch.full((B, 2 * H, D), -1.0, device="cuda")
    bl.bitlinear_attention(q, cache, ints(table.tolist()), ints([33, 60, 64]), out)
    want, bound = plain.attend(q.cpu().numpy(), cache, table, [33, 60, 64], page, D ** -0.5)
    within(out, want, bound)


def test_attention_length_beyond_the_table_counts_as_the_table():
    cache = plain.make_cache("int8", 4, 1, 16, 64, 0)
    t = torch.arange(32, device="cuda")
    table = ints([[2, 0]])
    plain.fill_row(cache, "int8", table[0].long()[t // 16], t % 16, normal((32, 1, 64), 1).cuda(), normal((32, 1, 64), 2).cuda())
    q, outs = normal((1, 2, 64), 3).cuda(), torch.empty(2, 1, 2, 64, device="cuda")
    bl.bitlinear_attention(q, cache, table, ints([32]), outs[0])
    bl.bitlinear_attention(q, cache, table, ints([2 ** 31 - 1]), outs[1])
    assert torch.isfinite(outs).all() and torch.equal(outs[0], outs[1])


def test_attention_strides_and_one_page_list_for_all_rows():
    """Causal rows of a prompt's end: rows of one page list with lengths n, n + 1, ..."""
    D, H, page, n, rows = 80, 4, 16, 61, 19
    cache = plain.make_cache("bf16", 8, H, page, D, 3)
    table = ints([[5, 1, 7, 0, 2]])
    t = torch.arange(n + rows, device="cuda")
    plain.fill_row(cache, "bf16", table[0].long()[t // page], t % page, normal((n + rows, H, D), 1).cuda(), normal((n + rows, H, D), 2).cuda())
    wide = normal((rows, 3 * H * D), 4).cuda()
    q = wide[:, H * D:2 * H * D].unflatten(1, (H, D))
    out_wide = torch.full((rows, H * D + 8), 2.5, device="cuda")
    out = out_wide[:, 4:4 + H * D].unflatten(1, (H, D))
    lengths = [n + 1 + i for i in range(rows)]
    bl.bitlinear_attention(q, cache[:2], table.expand(rows, 5), ints(lengths), out)
    want, bound = plain.attend(q.cpu().numpy(), cache, table.expand(rows, 5).cpu().numpy(), lengths, page, D ** -0.5)
    within(out, want, bound)
    assert (out_wide[:, :4] == 2.5).all() and (out_wide[:, 4 + H * D:] == 2.5).all()


@pytest.mark.parametrize("fmt", plain.FORMATS)
@pytest.mark.parametrize("B,H", [(77, 8), (127, 5), (128, 8), (129, 8)])
def test_attention_of_batches_that_start_with_the_longest(fmt, B, H):
    """More rows than fit at once, of equal, empty, negative and far too large lengths."""
    D, page, cols = 64, 16, 9
    n = cols * page
    cache = plain.make_cache(fmt, cols, H, page, D, B)
    table = ints([[3, 1, 8, 0, 2, 7, 5, 4, 6]])
    t = torch.arange(n, device="cuda")
    plain.fill_row(cache, fmt, table[0].long()[t // page], t % page, normal((n, H, D), 1).cuda(), normal((n, H, D), 2).cuda())
    rng = np.random.default_rng(B)
    lengths = rng.integers(0, n + 1, B)
    lengths[rng.permutation(B)[:40]] = [0, 2 ** 31 - 1, -5, n, 1 << 24, (1 << 24) + 1, -2 ** 31, 1] * 5
    q, (out, full) = normal((B, H, D), 3).cuda(), guarded(B * H * D, torch.float32, -7.0)
    out = out.view(B, H, D)
    bl.bitlinear_attention(q, cache, table.expand(B, cols), ints(lengths.tolist()), out)
    want, bound = plain.attend(q.cpu().numpy(), cache, table.expand(B, cols).cpu().numpy(), lengths, page, D ** -0.5)
    within(out, want, bound)
    check_canary(full, -7.0)


def test_cache_past_32_bit_offsets():
    """Codes at offsets above 2^32, in one page near a large cache's end."""
    page, H, D = 4096, 8, 128
    pages = (1 << 32) // (page * H * D) + 3
    k = torch.zeros(pages, H, page, D, dtype=torch.int8, device="cuda")
    cache = (k, torch.zeros_like(k), *(torch.ones(pages, H, page, device="cuda") for _ in "kv"))
    T = 40
    rows, vals = normal((T, H, D), 1).cuda(), normal((T, H, D), 2).cuda()
    table = ints([[pages - 1]])
    seq, pos = torch.zeros(T, dtype=torch.int32, device="cuda"), torch.arange(T, dtype=torch.int32, device="cuda")
    bl.bitlinear_kv_append(rows, vals, cache, pos, table, seq=seq)
    outs = torch.empty(2, T, H, D, device="cuda")
    bl.bitlinear_kv_read(cache, pos, table, outs[0], outs[1], seq=seq)
    top = torch.stack([rows, vals]).abs().amax(-1, keepdim=True)
    assert ((outs - torch.stack([rows, vals])).abs() <= top / 127 * (0.5 + 1e-4)).all()
    assert not cache[0][:-1].any() and not cache[1][:-1].any()
    q, out = normal((1, H, D), 3).cuda(), torch.empty(1, H, D, device="cuda")
    bl.bitlinear_attention(q, cache, table, ints([T]), out)
    small = tuple(c[-1:] for c in cache)
    want, bound = plain.attend(q.cpu().numpy(), small, np.array([[0]]), [T], page, D ** -0.5)
    within(out, want, bound)


# ------------------------------------------------------------------ used together


def decode_steps(fmt, B, Hq, Hk, D, page, steps, run):
    """`steps` decode steps from empty caches through `run(step)` -> (outs per step, 64-bit outs and bounds)."""
    width = -(-steps // page)
    st = dict(cache=plain.make_cache(fmt, B * width, Hk, page, D, 1),
              table=ints(np.random.default_rng(2).permutation(B * width).reshape(B, width).tolist()),
              positions=torch.zeros(B, dtype=torch.int32, device="cuda"), lengths=torch.ones(B, dtype=torch.int32, device="cuda"),
              freq=bl.bitlinear_rope_frequencies(D).cuda(), q=torch.empty(B, Hq, D, device="cuda"),
              k=torch.empty(B, Hk, D, device="cuda"), v=torch.empty(B, Hk, D, device="cuda"), out=torch.empty(B, Hq, D, device="cuda"))

    def step(flags=0, stream=None):
        bl.bitlinear_kv_append(st["k"], st["v"], st["cache"], st["positions"], st["table"], q=st["q"], q_out=st["q"],
                               rope=(st["freq"], bl.ROPE_HALF), flags=flags, stream=stream)
        bl.bitlinear_attention(st["q"], st["cache"], st["table"], st["lengths"], st["out"], flags=flags, stream=stream)

    one = run(step, st)
    for i in range(steps):
        for j, x in enumerate("qkv"):
            st[x].copy_(normal(st[x].shape, 1000 * j + i))
        one()
        torch.cuda.synchronize()
        want, bound = plain.attend(st["q"].cpu().numpy(), st["cache"],
                                   st["table"].cpu().numpy(), [i + 1] * B, page, D ** -0.5)
        within(st["out"], want, bound)
        st["positions"] += 1
        st["lengths"] += 1
    assert bl.bitlinear_device_status() == 0


@pytest.mark.parametrize("fmt", plain.FORMATS)
def test_decode_steps_eager(fmt):
    decode_steps(fmt, 3, 4, 2, 80, 16, 40, lambda step, st: step)


@pytest.mark.parametrize("fmt", plain.FORMATS)
def test_decode_steps_as_one_replayed_graph(fmt):
    def run(step, st):
        stream = torch.cuda.Stream()
        for x in "qkv":
            st[x].zero_()
        stream.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(stream):
            step(bl.FLAG_PDL, stream)
            torch.cuda.synchronize()
            g = torch.cuda.CUDAGraph()
            with torch.cuda.graph(g, stream=stream):
                step(bl.FLAG_PDL, stream)
        torch.cuda.synchronize()
        return g.replay
    decode_steps(fmt, 2, 8, 2, 128, 32, 35, run)


def test_results_repeat_bit_for_bit_and_streams_do_not_mix():
    B, Hq, Hk, D, page, n = 6, 8, 2, 80, 32, 1500
    width = -(-n // page)
    states = []
    for seed in (1, 2):
        cache = plain.make_cache("int8", B * width, Hk, page, D, seed)
        t = torch.arange(B * width * page, device="cuda")
        plain.fill_row(cache, "int8", t // page, t % page, normal((len(t), Hk, D), seed).cuda(), normal((len(t), Hk, D), seed + 9).cuda())
        states.append((normal((B, Hq, D), seed + 5).cuda(), cache, torch.arange(B * width, dtype=torch.int32, device="cuda").view(B, width),
                       ints([n - 100 * i for i in range(B)])))
    ws = [torch.empty(max(16, bl.bitlinear_attention_workspace(B, Hq, Hk, D)), dtype=torch.uint8, device="cuda") for _ in states]
    alone = []
    for s, w in zip(states, ws):
        out = torch.empty_like(s[0])
        bl.bitlinear_attention(*s, out, workspace=w)
        torch.cuda.synchronize()
        alone.append(out)
    streams = [torch.cuda.Stream() for _ in states]
    torch.cuda.synchronize()
    outs = [[torch.empty_like(s[0]) for _ in range(20)] for s in states]
    for i in range(20):
        for s, w, stream, out in zip(states, ws, streams, outs):
            bl.bitlinear_attention(*s, out[i], workspace=w, stream=stream)
    torch.cuda.synchronize()
    for want, got in zip(alone, outs):
        for o in got:
            assert torch.equal(want, o)


def test_binding_with_and_without_the_compiled_marshal(monkeypatch):
    if bl._marshal is None:
        pytest.skip("bitlinear_marshal.so was not built")
    T, Hq, Hk, D, page = 5, 6, 3, 80, 16
    for fmt in plain.FORMATS:
        results = []
        for marshal in (bl._marshal, None):
            monkeypatch.setattr(bl, "_marshal", marshal)
            cache = tuple(c if c is None else c.zero_() if c.dtype != torch.float8_e4m3fn else c.view(torch.uint8).zero_().view(c.dtype)
                          for c in plain.make_cache(fmt, 2 * T, Hk, page, D, 4))
            cache = cache[:2] if fmt == "bf16" else cache
            q, k, v = normal((T, Hq, D), 1).cuda(), normal((T, Hk, D), 2).cuda(), normal((T, Hk, D), 3).cuda()
            table, pos, freq = torch.arange(2 * T, dtype=torch.int32, device="cuda").view(T, 2), ints([3, 17, 0, 31, -1]), bl.bitlinear_rope_frequencies(64).cuda()
            y, q_out, ks, vs, out = torch.zeros_like(k), torch.zeros_like(q), torch.zeros_like(k), torch.zeros_like(v), torch.zeros_like(q)
            bl.bitlinear_rope(k, pos, (freq, bl.ROPE_INTERLEAVED, 1.5), y)
            bl.bitlinear_kv_append(k, v, cache, pos, table, q=q, q_out=q_out, rope=(freq, bl.ROPE_HALF))
            bl.bitlinear_kv_append(k, v, cache, pos - 1, table, seq=ints([1, 0, 2, 4, 3]), stream=torch.cuda.current_stream())
            bl.bitlinear_kv_read(cache, pos, table, ks, vs)
            bl.bitlinear_attention(q_out, cache, table, pos + 1, out, scale=0.3, window=9)
            bl.bitlinear_attention(q_out, cache, table, pos + 1, q, flags=bl.FLAG_PDL, stream=torch.cuda.current_stream().cuda_stream)
            results.append([y, q_out, ks, vs, out, q])
        for a, b in zip(*results):
            assert torch.isfinite(a).all() and a.abs().sum() > 0 and torch.equal(a, b)


@pytest.mark.parametrize("compiled", [True, False])
def test_binding_refusals(compiled, monkeypatch):
    if not compiled:
        monkeypatch.setattr(bl, "_marshal", None)
    cache = plain.make_cache("int8", 4, 2, 16, 64, 0)
    x, p, table = torch.zeros(2, 2, 64, device="cuda"), ints([0, 1]), ints([[0, 1], [2, 3]])
    freq = torch.ones(32, dtype=torch.float64, device="cuda")
    with pytest.raises(ValueError):
        bl.bitlinear_rope(x.transpose(0, 1), p, (freq, 0), x)                # heads not side by side
    with pytest.raises(TypeError):
        bl.bitlinear_rope(x, p.long(), (freq, 0), x)
    with pytest.raises(TypeError):
        bl.bitlinear_rope(x, p, (freq.float(), 0), x)
    with pytest.raises(bl.BitLinearError):
        bl.bitlinear_rope(x, p, (freq, 7), x)
    with pytest.raises(bl.BitLinearError):
        bl.bitlinear_rope(x, p, (torch.ones(33, dtype=torch.float64, device="cuda"), 0), x)
    with pytest.raises(ValueError):
        bl.bitlinear_kv_append(x, x, (cache[0], cache[1][:3], cache[2], cache[3]), p, table)
    with pytest.raises(TypeError):
        bl.bitlinear_kv_append(x, x, (cache[0], cache[1]), p, table)         # int8 without steps
    with pytest.raises(ValueError):
        bl.bitlinear_kv_append(x, x, cache, p, table, q_out=x)
    with pytest.raises(bl.BitLinearError):
        bl.bitlinear_kv_append(x, x, cache, p, table[:1])                    # two rows, one sequence, no seq
    with pytest.raises(ValueError):
        bl.bitlinear_attention(x, cache, table[:1], p, torch.empty_like(x))
    with pytest.raises(ValueError):
        bl.bitlinear_attention(x, cache, table.t(), p, torch.empty_like(x))
    with pytest.raises(bl.BitLinearError):
        bl.bitlinear_attention(torch.zeros(2, 3, 64, device="cuda"), cache, table, p, torch.zeros(2, 3, 64, device="cuda"))
    with pytest.raises(bl.BitLinearError):
        bl.bitlinear_attention(x, cache, table, p, torch.empty_like(x), scale=math.nan)
    with pytest.raises(ValueError):
        bl.bitlinear_attention(x, (cache[0].bfloat16(), cache[1].bfloat16(), cache[2], cache[3]), table, p, torch.empty_like(x))
