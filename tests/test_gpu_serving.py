"""The operators of a serving step on the GPU against plain forms in 64 bits or whole numbers."""
import numpy as np
import pytest
import torch

import attention_plain
import bitlinear_w1_a8_gb300 as bl
import serving_plain as plain
from harness import check_canary, guarded

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def built():
    bl.load_library()


def normal(shape, seed, std=1.0):
    g = torch.Generator().manual_seed(seed)
    return torch.randn(*shape, generator=g) * std


def ints(values):
    return torch.tensor(np.asarray(values), dtype=torch.int32, device="cuda")


def within(got, want, bound):
    got = got.double().cpu().numpy() if isinstance(got, torch.Tensor) else np.asarray(got, np.float64)
    assert np.isfinite(got).all()
    off = np.abs(got - want) - bound
    assert (off <= 0).all(), f"{(off > 0).sum()} of {off.size} beyond the bound, worst by {off.max():.3g}"


# ------------------------------------------------------------------ shared prefixes


def shared_case(fmt, groups, R, Hq, Hkv, D, shared, lengths, page, seed, one_list=False, spare=0):
    """A filled cache, q, the page table whose rows share their groups' pages (one_list: all of them), on the GPU.
    What no row attends to is NaN."""
    B, rng = groups * R, np.random.default_rng(seed)
    lengths = np.asarray(lengths)
    width = -(-int(max(lengths.max(), 1)) // page) + spare
    pages = B * width + 3
    cache = attention_plain.make_cache(fmt, pages, Hkv, page, D, seed)
    table = rng.permutation(pages)[:B * width].reshape(B, width)
    for b in range(B):
        first = b // R * R
        ends = width if one_list else -(-max(0, int(shared[b // R])) // page)
        table[b, :ends] = table[first, :ends]
    for b in range(B):
        n = int(lengths[b])
        if n <= 0:
            continue
        t = np.arange(n)
        where = torch.tensor(table[b, t // page].astype(np.int64), device="cuda"), torch.tensor(t % page, device="cuda")
        whose = (b // R * R if one_list else b)  # shared tokens are written by every row that has them: the same values
        k, v = (normal((width * page, Hkv, D), 1000 * i + whose)[:n] for i in (1, 2))
        s = min(n, width * page if one_list else max(0, int(shared[b // R])))
        for x, i in ((k, 3), (v, 4)):
            x[:s] = normal((width * page, Hkv, D), 1000 * i + b // R)[:s]
        attention_plain.fill_row(cache, fmt, where[0], where[1], k.cuda() * 1.3, v.cuda())
    q = normal((B, Hq, D), seed + 5, 1.5)
    return cache, q, table


def wide_table(table, cache):
    """The table with columns that no length reaches, as many as make the call share: over few columns it attends row by row."""
    pages, heads, page, D = cache[0].shape
    a_column = len(table) * page * heads * D * 2 * cache[0].element_size()
    wide = np.full((len(table), max(table.shape[1], 120_000_000 // a_column)), -1)
    wide[:, :table.shape[1]] = table
    return ints(wide)


def run_shared(fmt, groups, R, Hq, Hkv, D, shared, lengths, page=32, seed=0, one_list=False, scale=None, spare=0, flags=0):
    cache, q, table = shared_case(fmt, groups, R, Hq, Hkv, D, shared, lengths, page, seed, one_list, spare)
    out, full = guarded(q.numel(), torch.float32, 7.5)
    out = out.view(q.shape)
    need = bl.bitlinear_attention_shared_workspace(groups * R, Hq, Hkv, D, groups)
    ws, ws_full = guarded(max(need, 16), torch.uint8, 0x5a)
    want, bound = attention_plain.attend(q.numpy(), cache, table, lengths, page, D ** -0.5 if scale is None else scale)
    for columns in (ints(table), wide_table(table, cache)):
        out.fill_(float("nan"))
        bl.bitlinear_attention_shared(q.cuda(), cache, columns, ints(lengths), ints(shared), out, ws, scale=scale, flags=flags)
        torch.cuda.synchronize()
        within(out, want, bound)
        check_canary(full, 7.5)
        check_canary(ws_full, 0x5a)
    return out, (cache, q, table)


@pytest.mark.parametrize("fmt", attention_plain.FORMATS)
@pytest.mark.parametrize("groups,R,Hq,Hkv,D,S,own,page", [
    (1, 2, 2, 2, 64, 1, 1, 16), (1, 3, 8, 2, 80, 37, 5, 16), (2, 5, 4, 4, 96, 200, 33, 32), (1, 9, 4, 4, 112, 130, 64, 64),
    (3, 4, 14, 2, 128, 95, 17, 32), (1, 17, 8, 1, 16, 300, 20, 16), (2, 2, 16, 1, 256, 70, 40, 128), (1, 70, 3, 3, 80, 150, 9, 64),
    (1, 6, 60, 2, 64, 64, 16, 16), (5, 2, 1, 1, 48, 129, 1, 16), (1, 130, 2, 1, 128, 260, 3, 64), (1, 33, 16, 4, 128, 515, 30, 32)])
def test_shared(fmt, groups, R, Hq, Hkv, D, S, own, page):
    rng = np.random.default_rng(S)
    shared = rng.integers(max(1, S // 2), S + 1, groups)
    lengths = np.repeat(shared, R) + rng.integers(0, own + 1, groups * R)
    run_shared(fmt, groups, R, Hq, Hkv, D, shared, lengths, page, seed=S)


@pytest.mark.parametrize("fmt", attention_plain.FORMATS)
@pytest.mark.parametrize("groups,R,Hq,Hkv,D,S,own,page", [(1, 80, 4, 4, 48, 70, 30, 16), (2, 31, 10, 5, 80, 100, 700, 32), (5, 4, 48, 16, 128, 33, 400, 16),
                                                           (1, 40, 72, 8, 64, 50, 300, 64), (60, 5, 2, 1, 240, 20, 500, 16), (1, 1100, 1, 1, 16, 40, 20, 16)])
def test_shared_of_many_rows(fmt, groups, R, Hq, Hkv, D, S, own, page):
    """Enough rows that one CTA takes several of them: one, two or four warps a row, by the tokens of its own."""
    rng = np.random.default_rng(own)
    shared = rng.integers(max(1, S // 2), S + 1, groups)
    more = rng.integers(0, 20, groups * R)
    more[::7] = rng.integers(0, own + 1, len(more[::7]))
    run_shared(fmt, groups, R, Hq, Hkv, D, shared, np.repeat(shared, R) + more, page, seed=S)


@pytest.mark.parametrize("fmt", attention_plain.FORMATS)
@pytest.mark.parametrize("R,Hq,Hkv,D,n", [(5, 4, 4, 80, 100), (2, 8, 2, 128, 31), (9, 8, 1, 64, 47), (20, 4, 1, 96, 333)])
def test_drafted_rows_share_everything(fmt, R, Hq, Hkv, D, n):
    """Rows of one sequence that see one token more each; the longest sees all that is shared."""
    lengths = np.concatenate([m + 1 + np.arange(R) for m in (n, n // 3)])
    run_shared(fmt, 2, R, Hq, Hkv, D, [n + R, n // 3 + R], lengths, 16, seed=n, one_list=True)


@pytest.mark.parametrize("R,G", [(3, 1), (20, 4), (40, 1)])
def test_shared_borders(R, G):
    """Groups that share nothing, less than nothing, more than they have; rows without any token; lengths past the table."""
    page = 16
    shared = [0, -7, 40, 10 ** 6, 33]
    lengths = np.array([np.arange(R) % 50, 1 + np.arange(R) % 20, 40 + np.arange(R) % 9, 30 + np.arange(R) % 5, np.arange(R) % 2 * 40 + 33]).reshape(-1)
    lengths[0], lengths[R] = 0, -3
    one_list = np.repeat([False, False, False, True, False], R)
    cache, q, table = shared_case("int8", 5, R, 2 * G, 2, 64, [0, 0, 40, 0, 33], lengths, page, 9)
    for b in np.nonzero(one_list)[0]:
        table[b] = table[3 * R]
    t = np.arange(34)
    for b in (3 * R,):  # everything of the fourth group lies in its first row's pages
        x = [normal((34, 2, 64), 77 + i).cuda() for i in range(2)]
        attention_plain.fill_row(cache, "int8", torch.tensor(table[b, t // page].astype(np.int64), device="cuda"), torch.tensor(t % page, device="cuda"), *x)
    out = torch.full(q.shape, 3.0, device="cuda")
    ws = torch.empty(bl.bitlinear_attention_shared_workspace(5 * R, 2 * G, 2, 64, 5), dtype=torch.uint8, device="cuda")
    bl.bitlinear_attention_shared(q.cuda(), cache, wide_table(table, cache), ints(lengths), ints(shared), out, ws)
    want, bound = attention_plain.attend(q.numpy(), cache, table, lengths, page, 64 ** -0.5)
    within(out, want, bound)
    assert (out[lengths <= 0] == 0).all()


@pytest.mark.parametrize("R,G", [(4, 1), (32, 4)])
def test_shared_pages_out_of_range(R, G):
    page, S = 16, 100
    lengths = S + np.arange(R) % 30
    cache, q, table = shared_case("bf16", 1, R, 2 * G, 2, 80, [S], lengths, page, 11, spare=2)
    table[:, 2], table[:, 5] = 10 ** 6, -1   # shared pages that are nowhere
    table[1, 6:] = -1                        # a row without own pages (but for the shared one that it ends in)
    table[:, -2:] = 2 ** 31 - 1              # columns that no length reaches
    out = torch.empty(q.shape, device="cuda")
    ws = torch.empty(bl.bitlinear_attention_shared_workspace(R, 2 * G, 2, 80, 1), dtype=torch.uint8, device="cuda")
    table[1, 6] = table[0, 6]
    bl.bitlinear_attention_shared(q.cuda(), cache, wide_table(table, cache), ints(lengths), ints([S]), out, ws)
    want, bound = attention_plain.attend(q.numpy(), cache, table, lengths, page, 80 ** -0.5)
    within(out, want, bound)


def test_shared_strides_scales_and_agreement():
    """Slices of wider rows, a table of more columns, another scale and sign of it; rows alone give what attention gives."""
    R, Hq, Hkv, D, page, S = 6, 8, 4, 80, 32, 150
    lengths = S + np.arange(R) * 7
    cache, q, table = shared_case("fp8", 1, R, Hq, Hkv, D, [S], lengths, page, 21)
    wide_q, wide_out = torch.full((R, 3, Hq, D), float("nan"), device="cuda"), torch.full((R, 2, Hq, D), 4.0, device="cuda")
    wide_q[:, 1] = q.cuda()
    columns = wide_table(table, cache)
    padded = torch.full((R, columns.shape[1] + 5), -1, dtype=torch.int32, device="cuda")
    padded[:, :table.shape[1]] = ints(table)
    ws = torch.empty(bl.bitlinear_attention_shared_workspace(R, Hq, Hkv, D, 1), dtype=torch.uint8, device="cuda")
    for scale in (0.3, -0.2, 0.0):
        bl.bitlinear_attention_shared(wide_q[:, 1], cache, padded[:, :columns.shape[1]], ints(lengths), ints([S]), wide_out[:, 1], ws, scale=scale)
        want, bound = attention_plain.attend(q.numpy(), cache, table, lengths, page, scale)
        within(wide_out[:, 1], want, bound)
        assert (wide_out[:, 0] == 4.0).all()
    alone, plain_out = torch.empty(R, Hq, D, device="cuda"), torch.empty(R, Hq, D, device="cuda")
    bl.bitlinear_attention_shared(q.cuda(), cache, ints(table), ints(lengths), ints(np.zeros(R)), alone, None)
    bl.bitlinear_attention(q.cuda(), cache, ints(table), ints(lengths), plain_out)
    assert torch.equal(alone, plain_out)
    one = torch.empty(R, Hq, D, device="cuda")  # a table of stride 0: every row one list
    bl.bitlinear_attention_shared(q.cuda(), cache, wide_table(table, cache)[:1].expand(R, -1), ints(np.full(R, 120)), ints([120]), one, ws)
    want, bound = attention_plain.attend(q.numpy(), cache, np.repeat(table[:1], R, 0), np.full(R, 120), page, D ** -0.5)
    within(one, want, bound)


@pytest.mark.parametrize("R,G", [(4, 2), (64, 4)])
def test_shared_values_that_are_not_finite(R, G):
    """A NaN among shared tokens that count shows; one in a row's own tokens stays that row's; garbage behind the longest is not read."""
    S, page, D = 90, 16, 64
    lengths = S + 1 + np.arange(R) % 11
    cache, q, table = shared_case("bf16", 1, R, 2 * G, 2, D, [S], lengths, page, 31)
    ws = torch.empty(bl.bitlinear_attention_shared_workspace(R, 2 * G, 2, D, 1), dtype=torch.uint8, device="cuda")
    run = lambda: (bl.bitlinear_attention_shared(q.cuda(), cache, wide_table(table, cache), ints(lengths), ints([S]), out, ws), out.cpu())[1]  # noqa: E731
    out = torch.empty(q.shape, device="cuda")
    clean = run()
    assert torch.isfinite(clean).all()
    t = int(lengths[3]) - 1
    if t >= S and table[3, t // page] != table[0, t // page]:
        cache[1][table[3, t // page], 0, t % page] = float("nan")
        got = run()
        assert torch.isnan(got[3, :G]).all()
        keep = torch.ones(R, dtype=torch.bool)
        keep[3] = False
        assert torch.equal(got[keep], clean[keep]) and torch.equal(got[3, G:], clean[3, G:])
        cache[1][table[3, t // page], 0, t % page] = 0.5
    cache[0][table[0, 1], 1, 3] = float("nan")
    got = run()
    assert torch.isnan(got[:, G:]).all() and torch.isfinite(got[:, :G]).all()
    cache[0][table[0, 1], 1, 3] = 0.25
    q[2, 0, 5] = float("nan")
    got = run()
    assert torch.isnan(got[2, 0]).all() and torch.isfinite(got[2, 1:]).all() and torch.isfinite(got[:2]).all() and torch.isfinite(got[3:]).all()


@pytest.mark.parametrize("R,Hq,Hkv,D,S", [(8, 8, 8, 80, 700), (64, 8, 2, 128, 900)])
def test_shared_replayed_and_on_other_streams(R, Hq, Hkv, D, S):
    """Captured calls replayed with new lengths, calls on another stream and in a row on one workspace: the same bits."""
    page = 64
    lengths = S + 1 + np.arange(R) % 90
    cache, q, table = shared_case("int8", 1, R, Hq, Hkv, D, [S], lengths, page, 41)
    ws = torch.empty(bl.bitlinear_attention_shared_workspace(R, Hq, Hkv, D, 1), dtype=torch.uint8, device="cuda")
    q, table = q.cuda(), wide_table(table, cache)
    shared, n = ints([S]), ints(lengths)
    first, second, replayed = (torch.empty(q.shape, device="cuda") for _ in range(3))
    half, n_half = ints([S // 2]), ints(np.full(R, S // 2))
    for flags in (0, bl.FLAG_PDL):
        bl.bitlinear_attention_shared(q, cache, table, n, shared, first, ws, flags=flags)
        bl.bitlinear_attention_shared(q, cache, table, n_half, half, second, ws, flags=flags)
        stream = torch.cuda.Stream()
        torch.cuda.synchronize()
        with torch.cuda.stream(stream):
            graph = torch.cuda.CUDAGraph()
            length, share = n.clone(), shared.clone()
            torch.cuda.synchronize()
            with torch.cuda.graph(graph, stream=stream):
                bl.bitlinear_attention_shared(q, cache, table, length, share, replayed, ws, flags=flags)
        for _ in range(3):
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(replayed, first)
            length.copy_(n_half)
            share.copy_(half)
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(replayed, second)
            length.copy_(n)
            share.copy_(shared)
            torch.cuda.synchronize()


# ------------------------------------------------------------------ chosen blocks


def filled_cache(fmt, B, Hkv, D, lengths, page, seed):
    """A cache whose sequences are filled to their lengths, the rest NaN, and its page table."""
    rng = np.random.default_rng(seed)
    width = -(-max(1, int(np.max(lengths))) // page)
    pages = B * width + 2
    cache = attention_plain.make_cache(fmt, pages, Hkv, page, D, seed)
    table = rng.permutation(pages)[:B * width].reshape(B, width)
    for b in range(B):
        n = max(0, int(lengths[b]))
        if n:
            t = np.arange(n)
            drift = normal((width, Hkv, D), seed + b)[t // page] * 0.8
            attention_plain.fill_row(cache, fmt, torch.tensor(table[b, t // page].astype(np.int64), device="cuda"), torch.tensor(t % page, device="cuda"),
                                     (normal((n, Hkv, D), seed + 50 + b) + drift).cuda(), normal((n, Hkv, D), seed + 90 + b).cuda())
    return cache, table


def new_summary(cache):
    pages, heads, _, D = cache[0].shape
    return torch.full((pages, heads, 2, D), 99, dtype=torch.int8, device="cuda"), torch.full((pages, heads), 5.0, device="cuda")


@pytest.mark.parametrize("fmt", attention_plain.FORMATS)
@pytest.mark.parametrize("B,Hkv,D,lengths,page", [
    (1, 1, 16, [1], 16), (3, 4, 80, [37, 0, 200], 16), (2, 5, 128, [129, 64], 64), (2, 3, 96, [300, 31], 32), (1, 2, 112, [500], 128),
    (2, 2, 256, [70, 33], 16), (1, 3, 48, [1000], 512), (4, 2, 64, [5, 90, -2, 48], 16)])
def test_summarise(fmt, B, Hkv, D, lengths, page):
    cache, table = filled_cache(fmt, B, Hkv, D, lengths, page, 3 * B + D)
    bounds, step = new_summary(cache)
    bl.bitlinear_kv_summarise(cache, (bounds, step), ints(table), ints(np.zeros(B)), ints(lengths))
    want_b, want_s = np.full(bounds.shape, 99, np.int8), np.full(step.shape, 5.0, np.float32)
    ids = [(table[b, j], min(page, n - j * page)) for b, n in enumerate(lengths) for j in range(-(-max(n, 0) // page))]
    if ids:
        at = [i for i, _ in ids]
        want_b[at], want_s[at] = plain.summaries(cache, *zip(*ids))
    np.testing.assert_array_equal(bounds.cpu().numpy(), want_b)
    np.testing.assert_array_equal(step.cpu().numpy(), want_s)


def test_summarise_touches_only_the_pages_of_its_tokens():
    page, lengths, first = 16, [100, 64, 33], [99, 64, 15]   # the last page; none (no token); three
    cache, table = filled_cache("int8", 3, 2, 80, lengths, page, 5)
    bounds, step = new_summary(cache)
    wide = torch.full((3, table.shape[1] + 4), -5, dtype=torch.int32, device="cuda")
    wide[:, :table.shape[1]] = ints(table)
    wide[2, 1] = 10 ** 7                                     # one of them nowhere
    bl.bitlinear_kv_summarise(cache, (bounds, step), wide, ints(first), ints(lengths))
    touched = {table[0, 6]: 4, table[2, 0]: 16, table[2, 2]: 1}
    want_b, want_s = np.full(bounds.shape, 99, np.int8), np.full(step.shape, 5.0, np.float32)
    want_b[list(touched)], want_s[list(touched)] = plain.summaries(cache, list(touched), touched.values())
    np.testing.assert_array_equal(bounds.cpu().numpy(), want_b)
    np.testing.assert_array_equal(step.cpu().numpy(), want_s)
    bl.bitlinear_kv_summarise(cache, (bounds, step), wide, ints([-4, 200, 0]), ints([10 ** 9, 64, 0]))  # past the table: its pages
    ids = {table[0, j]: 16 for j in range(6)}
    want_b[list(ids)], want_s[list(ids)] = plain.summaries(cache, list(ids), ids.values())
    keep = [p for p in range(len(want_b)) if p != table[0, 6]]  # 16 tokens of it now, 12 of them garbage
    np.testing.assert_array_equal(bounds.cpu().numpy()[keep], want_b[keep])


def test_summarise_of_zeros_and_single_values():
    cache = tuple(torch.zeros(2, 1, 16, 32, dtype=torch.bfloat16, device="cuda") for _ in "kv")
    cache[0][1, 0, 3, 7] = -2.0
    bounds, step = new_summary(cache)
    bl.bitlinear_kv_summarise(cache, (bounds, step), ints([[0, 1]]), ints([0]), ints([32]))
    want_b, want_s = plain.summaries((*cache, None, None), [0, 1], [16, 16])
    np.testing.assert_array_equal(bounds.cpu().numpy(), want_b)
    np.testing.assert_array_equal(step.cpu().numpy(), want_s)
    assert bounds[1, 0, 0, 7] == -127 and step[0, 0] == np.float32(1e-5) / np.float32(127)


def random_summary(pages, heads, D, seed):
    rng = np.random.default_rng(seed)
    a, b = rng.integers(-127, 128, (2, pages, heads, D))
    return np.stack([np.minimum(a, b), np.maximum(a, b)], 2).astype(np.int8), rng.uniform(0.001, 0.05, (pages, heads)).astype(np.float32)


def run_select(q, bounds, step, table, lengths, page, keep_first, keep_last, count, flags=0):
    pages, heads, _, D = bounds.shape
    sizes = torch.empty(pages, heads, page, D, dtype=torch.bfloat16, device="cuda")  # its codes are not read
    B = len(lengths)
    blocks, full = guarded(B * heads * count, torch.int32, 12345)
    blocks = blocks.view(B, heads, count)
    bl.bitlinear_attention_select(torch.as_tensor(q).cuda(), (sizes, sizes), (torch.as_tensor(bounds).cuda(), torch.as_tensor(step).cuda()), ints(table),
                                  ints(lengths), blocks, keep_first=keep_first, keep_last=keep_last, flags=flags)
    torch.cuda.synchronize()
    check_canary(full, 12345)
    return blocks.cpu().numpy()


@pytest.mark.parametrize("B,Hq,Hkv,D,columns,count,keep", [
    (1, 1, 1, 16, 1, 1, (0, 0)), (2, 8, 2, 80, 40, 8, (1, 1)), (3, 4, 4, 128, 129, 64, (0, 0)), (1, 40, 2, 64, 700, 33, (2, 3)),
    (2, 3, 1, 256, 300, 4, (3, 3)), (1, 8, 8, 96, 2048, 64, (1, 1)), (1, 2, 1, 112, 5000, 500, (0, 7)), (20, 16, 16, 48, 90, 16, (1, 1)),
    (1, 34, 1, 32, 1500, 4096, (1, 1))])
def test_select(B, Hq, Hkv, D, columns, count, keep):
    page, rng = 16, np.random.default_rng(D + columns)
    q = normal((B, Hq, D), columns).numpy()
    bounds, step = random_summary(B * columns + 1, Hkv, D, columns)
    table = rng.permutation(B * columns + 1)[:B * columns].reshape(B, columns)
    lengths = rng.integers(1, columns * page + 1, B)
    lengths[0] = columns * page - (5 if columns > 1 else 0)
    table[rng.random(table.shape) < 0.03] = -1 if columns % 2 else 10 ** 8  # pages that are nowhere
    got = run_select(q, bounds, step, table, lengths, page, *keep, count)
    for b in range(B):
        np.testing.assert_array_equal(got[b], plain.choose(q[b], bounds, step, table[b], lengths[b], page, *keep, count))


def test_select_ties_and_borders():
    """Equal scores go to the earlier page, on both sides of every border between CTAs; no token, no page; more kept than wanted."""
    page, D, columns = 16, 64, 1000
    q = normal((6, 2, D), 1).numpy()
    bounds, step = np.repeat(random_summary(1, 1, D, 2)[0], 3, 0), np.array([[0.01], [0.01], [0.02]], np.float32)
    table = np.zeros((6, columns), np.int64)
    table[:, 7::3] = 1                      # another page of the same bounds and step
    table[1, 500], table[1, 999] = 2, 2     # two of twice the score (or its negative)
    lengths = [columns * page, columns * page, 0, -4, 1, 10 ** 9]
    for count, keep in ((1, (0, 0)), (130, (0, 0)), (999, (0, 1)), (1001, (1, 1)), (3, (2, 9)), (64, (0, 0))):
        got = run_select(q, bounds, step, table, lengths, page, *keep, count)
        for b in range(6):
            np.testing.assert_array_equal(got[b], plain.choose(q[b], bounds, step, table[b], lengths[b], page, *keep, count), err_msg=f"{count} {keep} {b}")


def test_select_scores_of_zero_and_nan():
    page, D = 16, 32
    q = np.zeros((1, 1, D), np.float32)     # every score 0 (of either sign)
    bounds, step = random_summary(50, 1, D, 4)
    table = np.arange(50)[None]
    assert run_select(q, bounds, step, table, [800], page, 0, 0, 5)[0, 0].tolist() == [0, 1, 2, 3, 4]
    q = normal((1, 1, D), 5).numpy()
    step[3], step[20] = np.nan, np.inf
    want = plain.choose(q[0], bounds, np.where(np.isnan(step), 0, step), table[0], 800, page, 0, 0, 50)[0]
    got = run_select(q, bounds, step, table, [800], page, 0, 0, 50)[0, 0]
    assert (got == want).all()              # all 50, the NaN among them
    assert 3 not in run_select(q, bounds, step, table, [800], page, 0, 0, 49)[0, 0]


@pytest.mark.parametrize("columns,heads,B", [(131072, 1, 1), (70000, 2, 2), (30000, 8, 3)])
def test_select_of_many_pages(columns, heads, B):
    """As many pages as a row may have, all of them in one summary that the table repeats."""
    page, D, count = 16, 16, 100
    rng = np.random.default_rng(columns)
    q = normal((B, heads, D), 6).numpy()
    bounds, step = random_summary(4096, heads, D, 7)
    table = rng.integers(0, 4096, (B, columns))
    lengths = [columns * page - 3 * b for b in range(B)]
    got = run_select(q, bounds, step, table, lengths, page, 1, 1, count)
    for b in range(B):
        for h in range(heads):
            top = np.abs(q[b, h]).max()
            codes = np.rint(q[b, h] * (np.float32(127) / top)).astype(np.int64)
            acc = np.maximum(codes * bounds[:, h, 0].astype(np.int64), codes * bounds[:, h, 1].astype(np.int64)).sum(-1)
            score = ((acc.astype(np.float32) * step[:, h]) * (top / np.float32(127)))[table[b]]
            score[0] = score[-1] = np.inf
            np.testing.assert_array_equal(got[b, h], np.sort(np.argsort(-score, kind="stable")[:count]))


@pytest.mark.parametrize("fmt", attention_plain.FORMATS)
@pytest.mark.parametrize("B,Hq,Hkv,D,page,L,count", [
    (1, 1, 1, 64, 16, 1, 1), (3, 8, 2, 80, 16, 200, 5), (2, 4, 4, 128, 32, 333, 4), (1, 14, 2, 96, 64, 900, 9), (2, 20, 2, 112, 16, 300, 12),
    (1, 2, 1, 256, 16, 100, 3), (9, 4, 2, 16, 128, 700, 2), (1, 8, 8, 80, 64, 2000, 31), (40, 8, 8, 64, 16, 90, 4)])
def test_attention_over_blocks(fmt, B, Hq, Hkv, D, page, L, count):
    rng = np.random.default_rng(L)
    lengths = rng.integers(max(1, L // 3), L + 1, B)
    cache, table = filled_cache(fmt, B, Hkv, D, lengths, page, L)
    q = normal((B, Hq, D), 8, 1.5)
    columns = table.shape[1]
    blocks = np.full((B, Hkv, count), -1)
    for b in range(B):
        for h in range(Hkv):
            n = rng.integers(1, min(count, columns) + 1)
            some = rng.permutation(columns)[:n]       # in no order, some of them past the length
            blocks[b, h, rng.permutation(count)[:n]] = some
    out, full = guarded(q.numel(), torch.float32, 2.5)
    out = out.view(q.shape)
    bl.bitlinear_attention_blocks(q.cuda(), cache, ints(table), ints(lengths), ints(blocks), out)
    want, bound = plain.attend_blocks(q.numpy(), cache, table, lengths, blocks, page, D ** -0.5)
    within(out, want, bound)
    check_canary(full, 2.5)


def test_blocks_that_are_none_or_listed_twice():
    B, Hkv, D, page = 4, 2, 80, 16
    lengths = [100, 70, 0, 33]
    cache, table = filled_cache("int8", B, Hkv, D, lengths, page, 13)
    wide = np.full((B, table.shape[1] + 2), 10 ** 9)
    wide[:, :table.shape[1]] = table
    wide[0, 1] = -1                                                   # a page that is nowhere
    blocks = np.full((B, Hkv, 6), -1)
    blocks[0] = [[0, 1, 0, 6, 10 ** 9, 2 ** 31 - 1], [3, 3, 3, -2 ** 31, 5, 1]]
    blocks[1] = [[-1, -1, -1, -1, -1, 4], [5, 6, 7, 8, 9, -9]]        # the second: none of its tokens
    q, out = normal((B, 4, D), 14), torch.full((B, 4, D), 9.0, device="cuda")
    bl.bitlinear_attention_blocks(q.cuda(), cache, ints(wide), ints(lengths), ints(blocks), out, scale=0.2)
    want, bound = plain.attend_blocks(q.numpy(), cache, wide, lengths, blocks, page, 0.2)
    within(out, want, bound)
    assert (out[2] == 0).all() and (out[3] == 0).all() and (out[1, 2:] == 0).all() and (out[1, :2] != 0).any()


def test_all_blocks_are_attention():
    """Every page listed in order: what bitlinear_attention gives, to both bounds."""
    B, Hq, Hkv, D, page, L = 2, 8, 2, 128, 32, 700
    cache, table = filled_cache("fp8", B, Hkv, D, [L, L - 90], page, 15)
    q = normal((B, Hq, D), 16, 1.5)
    blocks = np.tile(np.arange(table.shape[1]), (B, Hkv, 1))
    out = torch.empty(B, Hq, D, device="cuda")
    bl.bitlinear_attention_blocks(q.cuda(), cache, ints(table), ints([L, L - 90]), ints(blocks), out)
    want, bound = attention_plain.attend(q.numpy(), cache, table, [L, L - 90], page, D ** -0.5)
    within(out, want, bound)


# ------------------------------------------------------------------ probabilities


@pytest.mark.parametrize("M,V", [(1, 1), (2, 3), (3, 7), (5, 129), (1, 2048), (2, 4097), (1, 50000), (3, 50001), (2, 65534), (1, 131075), (2, 300007)])
@pytest.mark.parametrize("warm", [False, True])
def test_softmax(M, V, warm):
    y = normal((M, V), V, 3.0)
    t = torch.tensor([1.0, 0.3, 7.0, 0.0, 1e-20, 2e30][:M] if M < 6 else [1.0] * M) if warm else None
    if warm and M == 1:
        t = torch.tensor([0.7])
    if V > 5:
        y[0, 2] = y[-1, V - 1] = -np.inf
    p, full = guarded(M * V, torch.float32, 4.5)
    p = p.view(M, V)
    bl.bitlinear_softmax(y.cuda(), p, None if t is None else t.cuda())
    want, bound = plain.softmax(y.numpy(), None if t is None else t.numpy())
    within(p, want, bound)
    check_canary(full, 4.5)
    inplace = y.cuda()
    bl.bitlinear_softmax(inplace, inplace, None if t is None else t.cuda())
    assert torch.equal(inplace, p)


def test_softmax_borders():
    V = 5003
    y = normal((8, V), 1, 2.0)
    y[0] = -np.inf                                   # masked whole
    y[1] = -np.inf
    y[1, 4000] = -3.0                                # one left
    y[2] = 5.0                                       # all equal
    y[3, 17] = y[3, 4999] = 50.0                     # two maxima, temperature 0
    y[4, 9] = np.nan
    y[5, 9] = np.inf
    y[6] *= 1e30                                     # far apart
    y[7] = torch.finfo(torch.float32).min            # masked with the type's lowest value, but for two
    y[7, :2] = 1.0
    t = torch.tensor([1.0, 1.0, 2.0, 0.0, 1.0, 1.0, 1.0, 0.5])
    p = torch.empty_like(y, device="cuda")
    bl.bitlinear_softmax(y.cuda(), p, t.cuda())
    p = p.cpu()
    assert (p[0] == 0).all() and p[1, 4000] == 1 and p[1].sum() == 1
    assert torch.isnan(p[4]).all() and torch.isnan(p[5]).all()
    assert p[3, 17] == 1 and p[3].sum() == 1 and p[7, 0] == p[7, 1] == 0.5 and (p[7, 2:] == 0).all()
    for m in (1, 2, 3, 6, 7):
        want, bound = plain.softmax(y[m:m + 1].numpy(), t[m:m + 1].numpy())
        within(p[m:m + 1], want, bound)
    zero = torch.zeros(8, device="cuda")
    bl.bitlinear_softmax(y.cuda(), q := torch.empty_like(y, device="cuda"), zero)
    assert (q[0] == 0).all()                         # no maximum to choose
    for m in (1, 2, 3, 6, 7):
        assert q[m].argmax().item() == y[m].argmax().item() and q[m].sum() == 1
    y[3, :] = -0.0
    y[3, 11] = 0.0                                   # equal to the others
    bl.bitlinear_softmax(y.cuda(), q, zero)
    assert q[3, 0] == 1


def test_softmax_of_many_rows():
    y = normal((70001, 5), 2, 2.0)
    p = torch.empty_like(y, device="cuda")
    bl.bitlinear_softmax(y.cuda(), p)
    want = torch.softmax(y.double(), -1).numpy()
    within(p, want, want * 2.0 ** -18 + 2.0 ** -125)  # |z| below 24: (12 * 24 * 2 + 120) U


# ------------------------------------------------------------------ drafted tokens


def probabilities(shape, seed, std=2.0):
    return torch.softmax(normal(shape, seed, std).double(), -1).float()


def run_verify(p, q, draft, uniform, flags=0):
    B, K1, V = p.shape
    tokens, full = guarded(B * K1, torch.int32, 777)
    accepted, full2 = guarded(B, torch.int32, 778)
    tokens = tokens.view(B, K1)
    cuda = lambda t: None if t is None else t.cuda()  # noqa: E731
    bl.bitlinear_verify(p.cuda(), cuda(q), cuda(draft), uniform.cuda(), tokens, accepted, flags=flags)
    torch.cuda.synchronize()
    check_canary(full, 777)
    check_canary(full2, 778)
    want = plain.verify(p.numpy(), None if q is None else q.numpy(), None if draft is None else draft.numpy(), uniform.numpy())
    np.testing.assert_array_equal(accepted.cpu().numpy(), want[1])
    np.testing.assert_array_equal(tokens.cpu().numpy(), want[0])
    return want


@pytest.mark.parametrize("B,K,V", [(1, 1, 1), (3, 2, 5), (7, 4, 1000), (2, 33, 257), (1, 70, 100), (5, 3, 4099), (2, 4, 50000), (1, 2, 131073), (40, 1, 600)])
def test_verify(B, K, V):
    p, g = probabilities((B, K + 1, V), V), torch.Generator().manual_seed(V)
    q = torch.softmax(p[:, :K].log().double() + 0.4 * normal((B, K, V), V + 1), -1).float()
    draft = torch.multinomial(q.view(B * K, V), 1, generator=g).view(B, K).int()
    uniform = torch.rand(B, K + 1, generator=g)
    run_verify(p, q, draft, uniform)
    run_verify(p, q, draft, uniform * 0.01)              # most are taken
    run_verify(p, p[:, :K].contiguous(), draft, uniform)  # the same distribution: all are taken
    draft[0, K // 2] = -1                                # drafts that end early, by a number out of range too
    draft[-1, -1] = V
    run_verify(p, q, draft, uniform)


@pytest.mark.parametrize("V", [1, 9, 2047, 50001])
def test_a_token_drawn(V):
    """No drafts: the token at a fraction of the whole, at its ends and at each border between tokens."""
    B = 12
    p, u = probabilities((B, 1, V), V, 1.0), torch.rand(B, 1, generator=torch.Generator().manual_seed(V))
    u[0], u[1], u[2], u[3], u[4], u[5] = 0.0, 1 - 2.0 ** -24, 1.0, -1.0, float("nan"), 2.0 ** -24
    p[6, 0, :V // 2] = 0.0
    u[6] = 0.0                                           # the first with any weight
    p[7] = 0.0                                           # none has
    p[8, 0, -1] = 0.0
    u[8] = 1 - 2.0 ** -24
    p[9] = 1.0                                           # not normalised
    p[10, 0, 0] = float("nan")
    p[11, 0, 0] = -5.0
    tokens = run_verify(p, None, None, u)[0]
    assert tokens[7, 0] == -1


def test_a_token_drawn_at_exact_borders():
    """Weights of 1/8: u = i/8 is the first fraction that belongs to token i."""
    p = torch.full((17, 1, 8), 0.125)
    u = torch.tensor([i / 8 for i in range(8)] + [i / 8 - 2.0 ** -24 for i in range(1, 9)] + [0.5 + 2.0 ** -24])[:, None]
    assert run_verify(p, None, None, u)[0][:, 0].tolist() == list(range(8)) + list(range(8)) + [4]


def test_verify_residuals_and_refusals():
    V, K = 3000, 3
    p, q = torch.zeros(5, K + 1, V), torch.zeros(5, K, V)
    p[:, :, 10], q[:, :, 20] = 1.0, 1.0                  # nothing in common: the first is refused, the rest is p
    p[1, 0], q[1, 0] = 0.0, 0.0                          # no weight at all
    q[2, 0] = 0.0
    q[2, 0, 10] = 2.0                                    # refused (u q >= p), and nothing is left of p - q: p itself
    draft, u = torch.full((5, K), 20, dtype=torch.int32), torch.full((5, K + 1), 0.75)
    draft[2, 0], draft[3, 0] = 10, 10                    # the fourth: q = 0 there, p = 1: taken whatever the number
    u[4, 0] = float("nan")                               # no number: refused
    p[4, 0, 20] = 1.0
    tokens, accepted = run_verify(p, q, draft, u)
    assert tokens[:, 0].tolist() == [10, -1, 10, 10, 10] and accepted.tolist() == [0, 0, 0, 1, 0]
    assert tokens[3].tolist() == [10, 10, -1, -1]


def test_verify_of_many_sequences():
    B, V = 70000, 4
    p, q = probabilities((B, 2, V), 1), probabilities((B, 1, V), 2)
    g = torch.Generator().manual_seed(3)
    draft, u = torch.randint(0, V, (B, 1), generator=g, dtype=torch.int32), torch.rand(B, 2, generator=g)
    tokens, accepted = (torch.empty(B, 2, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda"))
    bl.bitlinear_verify(p.cuda(), q.cuda(), draft.cuda(), u.cuda(), tokens, accepted)
    some = torch.arange(0, B, 997)
    some[-1] = B - 1
    want = plain.verify(p[some].numpy(), q[some].numpy(), draft[some].numpy(), u[some].numpy())
    np.testing.assert_array_equal(tokens.cpu()[some].numpy(), want[0])
    np.testing.assert_array_equal(accepted.cpu()[some].numpy(), want[1])


def test_verified_tokens_are_distributed_as_the_targets():
    """Drafts from q, verified against p: the first token's counts are p's, to six deviations."""
    V, n = 6, 60000
    p, q = torch.tensor([0.05, 0.3, 0.1, 0.25, 0.0, 0.3]), torch.tensor([0.3, 0.1, 0.1, 0.2, 0.2, 0.1])
    g = torch.Generator().manual_seed(4)
    draft = torch.multinomial(q, n, replacement=True, generator=g).int().view(n, 1)
    tokens, accepted = (torch.empty(n, 2, dtype=torch.int32, device="cuda"), torch.empty(n, dtype=torch.int32, device="cuda"))
    bl.bitlinear_verify(p.expand(n, 2, V).contiguous().cuda(), q.expand(n, 1, V).contiguous().cuda(), draft.cuda(), torch.rand(n, 2, generator=g).cuda(), tokens, accepted)
    counts = torch.bincount(tokens[:, 0].cpu(), minlength=V).double().numpy()
    want = p.double().numpy() * n
    assert (np.abs(counts - want) <= 6 * np.sqrt(want + 1e-9)).all()


# ------------------------------------------------------------------ the binding


@pytest.mark.parametrize("compiled", [True, False])
def test_the_binding_with_and_without_the_compiled_marshal(compiled, monkeypatch):
    if compiled and bl._marshal is None:
        pytest.skip("bitlinear_marshal was not built")
    if not compiled:
        monkeypatch.setattr(bl, "_marshal", None)
    test_shared("int8", 2, 5, 4, 4, 96, 200, 33, 32)
    test_summarise("fp8", 3, 4, 80, [37, 0, 200], 16)
    test_select(2, 8, 2, 80, 40, 8, (1, 1))
    test_attention_over_blocks("bf16", 3, 8, 2, 80, 16, 200, 5)
    test_softmax(3, 50001, True)
    test_verify(7, 4, 1000)
    x, i = torch.zeros(2, 2, 64, device="cuda"), ints([1, 1])
    cache = tuple(torch.zeros(4, 2, 16, 64, dtype=torch.int8, device="cuda") for _ in "kv") + tuple(torch.zeros(4, 2, 16, device="cuda") for _ in "kv")
    table, s = ints([[0, 1], [2, 3]]), (torch.zeros(4, 2, 2, 64, dtype=torch.int8, device="cuda"), torch.zeros(4, 2, device="cuda"))
    blocks = torch.zeros(2, 2, 1, dtype=torch.int32, device="cuda")
    with pytest.raises(bl.BitLinearError):
        bl.bitlinear_attention_shared(x, cache, table, i, i[:1], x.clone())          # no workspace
    with pytest.raises(bl.BitLinearError):
        bl.bitlinear_attention_select(x, cache, s, table, i, blocks, keep_first=-1)
    for call in (lambda: bl.bitlinear_attention_shared(x, cache, table, i, table, x.clone()),
                 lambda: bl.bitlinear_attention_shared(x, cache, table, i[:1], i, x.clone()),
                 lambda: bl.bitlinear_kv_summarise(cache, (s[0][:3], s[1]), table, i, i),
                 lambda: bl.bitlinear_kv_summarise(cache, s, table, i[:1], i),
                 lambda: bl.bitlinear_attention_select(x, cache, s, table, i, blocks[:1]),
                 lambda: bl.bitlinear_attention_blocks(x, cache, table, i, blocks[:, :1], x.clone()),
                 lambda: bl.bitlinear_softmax(x, x), lambda: bl.bitlinear_softmax(x[0], x[0, :1]),
                 lambda: bl.bitlinear_softmax(x[0], x[0].clone(), torch.ones(3, device="cuda")),
                 lambda: bl.bitlinear_verify(x, x, i, x[:, 0], i, i)):
        with pytest.raises(ValueError):
            call()
    for call in (lambda: bl.bitlinear_attention_blocks(x, cache, table, i, blocks.long(), x.clone()), lambda: bl.bitlinear_softmax(x[0].half(), x[0]),
                 lambda: bl.bitlinear_kv_summarise(cache, (s[0].float(), s[1]), table, i, i)):
        with pytest.raises(TypeError):
            call()


# ------------------------------------------------------------------ ranges of values, and of addresses


@pytest.mark.parametrize("D", [128, 64])
def test_shared_bf16_values_of_many_magnitudes(D):
    """Tiles of 128 tokens on the tensor cores whose values are 2^40 apart, one of zeros, one of a single large value.

    A value loses 2^-39 of its tile's largest at most, beside the bound of all formats: weighted as the values are."""
    R, G, Hkv, S, page = 40, 2, 2, 900, 64
    lengths = S + np.arange(R) % 7
    cache, q, table = shared_case("bf16", 1, R, G * Hkv, Hkv, D, [S], lengths, page, 71)
    size = np.ones(960)
    size[128:256], size[256:384], size[384:512], size[512:640] = 2.0 ** 20, 0.0, 2.0 ** -20, 2.0 ** -90
    largest = np.zeros((Hkv, 960))
    for t in range(S):
        cache[1][table[0, t // page], :, t % page] *= size[t]
    cache[1][table[0, 700 // page], :, 700 % page, 5] = 3e4
    want, bound = attention_plain.attend(q.numpy(), cache, table, lengths, page, D ** -0.5)
    held = attention_plain.held(cache, "v")
    for t0 in range(0, S, 128):
        rows = [(table[0, t // page], t % page) for t in range(t0, min(S, t0 + 128))]
        largest[:, t0:t0 + 128] = np.max([np.abs(held[p, :, o]).max(-1) for p, o in rows], 0)[:, None]
    keys = attention_plain.held(cache, "k")
    for b in range(R):
        for h in range(G * Hkv):
            k = np.stack([keys[table[b, t // page], h // G, t % page] for t in range(lengths[b])])
            w = np.exp((x := D ** -0.5 * (k @ q[b, h].double().numpy())) - x.max())
            bound[b, h] += 1.01 * 2.0 ** -39 * (w @ largest[h // G, :lengths[b]]) / w.sum()
    out = torch.empty(q.shape, device="cuda")
    ws = torch.empty(bl.bitlinear_attention_shared_workspace(R, G * Hkv, Hkv, D, 1), dtype=torch.uint8, device="cuda")
    bl.bitlinear_attention_shared(q.cuda(), cache, wide_table(table, cache), ints(lengths), ints([S]), out, ws)
    within(out, want, bound)


@pytest.mark.parametrize("fmt", ["bf16", "fp8"])
@pytest.mark.parametrize("R,G", [(4, 2), (64, 4)])
def test_shared_values_that_are_infinite(fmt, R, G):
    """An infinity among shared values: no finite number where it counts, the other key head as before; in a step likewise."""
    S, page, D = 300, 16, 64
    lengths = S + 1 + np.arange(R) % 11
    cache, q, table = shared_case(fmt, 1, R, 2 * G, 2, D, [S], lengths, page, 31)
    ws = torch.empty(bl.bitlinear_attention_shared_workspace(R, 2 * G, 2, D, 1), dtype=torch.uint8, device="cuda")
    out, columns = torch.empty(q.shape, device="cuda"), wide_table(table, cache)
    run = lambda: (bl.bitlinear_attention_shared(q.cuda(), cache, columns, ints(lengths), ints([S]), out, ws), out.cpu())[1]  # noqa: E731
    clean = run()
    assert torch.isfinite(clean).all()
    if fmt == "bf16":
        cache[1][table[0, 5], 1, 3, 7] = float("inf")
        got = run()
        assert not torch.isfinite(got[:, G:, 7]).any()
        others = torch.arange(D) != 7
        same = (got[:, G:] == clean[:, G:]) | torch.isnan(got[:, G:])
        assert same[:, :, others].all()
    else:
        cache[3][table[0, 5], 1, 3] = float("inf")
        assert not torch.isfinite(run()[:, G:]).any()
    assert torch.equal(run()[:, :G], clean[:, :G])


def test_garbage_behind_the_tokens_is_not_met():
    """The largest finite values where no token is, in the tile that shared tokens end in."""
    R, G, Hkv, S, page, D = 64, 2, 2, 333, 64, 96
    lengths = S + np.arange(R) % 3
    cache, q, table = shared_case("bf16", 1, R, G * Hkv, Hkv, D, [S], lengths, page, 77)
    for c in cache[:2]:
        c[torch.isnan(c)] = 3e38
    out = torch.empty(q.shape, device="cuda")
    ws = torch.empty(bl.bitlinear_attention_shared_workspace(R, G * Hkv, Hkv, D, 1), dtype=torch.uint8, device="cuda")
    bl.bitlinear_attention_shared(q.cuda(), cache, wide_table(table, cache), ints(lengths), ints([S]), out, ws)
    want, bound = attention_plain.attend(q.numpy(), cache, table, lengths, page, D ** -0.5)
    within(out, want, bound)


@pytest.mark.parametrize("fmt", attention_plain.FORMATS)
def test_caches_of_more_than_4_gib(fmt):
    """The same pages at the end of a cache whose codes pass 2^32 bytes: the same bits from every operator."""
    Hkv, G, D, page, S = 8, 4, 128, 64, 512  # whole pages: in one that rows share, all have as many tokens
    a_page = Hkv * page * D * (2 if fmt == "bf16" else 1)
    for R in (6, 64):  # the tensor cores' path among them
        lengths = S + 1 + np.arange(R) % 90
        cache, q, table = shared_case(fmt, 1, R, Hkv * G, Hkv, D, [S], lengths, page, 81)
        pages = cache[0].shape[0]
        first = (1 << 32) // a_page + 5
        large = tuple(None if c is None else torch.empty(first + pages, *c.shape[1:], dtype=c.dtype, device="cuda") for c in cache)
        for big, c in zip(large, cache):
            if big is not None:
                big[first:] = c
        ws = torch.empty(bl.bitlinear_attention_shared_workspace(R, Hkv * G, Hkv, D, 1), dtype=torch.uint8, device="cuda")
        columns, n, share, q = wide_table(table, cache), ints(lengths), ints([S]), q.cuda()
        got = []
        for c, t in ((cache, columns), (large, torch.where(columns >= 0, columns + first, columns))):
            out, listed = torch.empty(q.shape, device="cuda"), torch.empty(q.shape, device="cuda")
            summary = new_summary(c)
            blocks = torch.empty(R, Hkv, 4, dtype=torch.int32, device="cuda")
            bl.bitlinear_attention_shared(q, c, t, n, share, out, ws)
            bl.bitlinear_kv_summarise(c, summary, t, torch.zeros_like(n), n)
            bl.bitlinear_attention_select(q, c, summary, t[:, :table.shape[1]], n, blocks)
            bl.bitlinear_attention_blocks(q, c, t, n, blocks, listed)
            torch.cuda.synchronize()
            got.append((out, blocks, listed, summary[0][-pages:], summary[1][-pages:]))
        for a, b in zip(*got):
            assert torch.equal(a, b)


# ------------------------------------------------------------------ the compiled marshal


@pytest.fixture
def stand_ins():
    import ctypes
    lib = bl.load_library()
    if bl._marshal is None:
        pytest.skip("bitlinear_marshal was not built")
    address = lambda f: ctypes.cast(f, ctypes.c_void_p).value  # noqa: E731
    yield lambda f: bl._marshal.bind_serving(*[address(f)] * len(bl._SERVING))
    bl._marshal.bind_serving(*(address(getattr(lib, "bitlinear_" + n)) for n in bl._SERVING))


def serving_calls():
    x, i = torch.zeros(2, 2, 64, device="cuda"), ints([1, 1])
    cache = tuple(torch.zeros(4, 2, 16, 64, dtype=torch.int8, device="cuda") for _ in "kv") + tuple(torch.zeros(4, 2, 16, device="cuda") for _ in "kv")
    table, s = ints([[0, 1], [2, 3]]), (torch.zeros(4, 2, 2, 64, dtype=torch.int8, device="cuda"), torch.zeros(4, 2, device="cuda"))
    blocks, two = torch.zeros(2, 2, 1, dtype=torch.int32, device="cuda"), torch.zeros(2, 2, device="cuda")
    m = bl._marshal
    return {"attention_shared": m.attention_shared(x, cache, table, i, i[:1], x.clone(), None, None, 0, None),
            "kv_summarise": m.kv_summarise(cache, s, table, i, i, 0, None),
            "attention_select": m.attention_select(x, cache, s, table, i, blocks, 1, 1, 0, None),
            "attention_blocks": m.attention_blocks(x, cache, table, i, blocks, x.clone(), None, 0, None),
            "softmax": m.softmax(two, two, None, 0, None),
            "verify": m.verify(x, x[:, :1].clone(), i.view(2, 1), two, ints([[0, 0], [0, 0]]), i, 0, None)}


def test_the_marshal_returns_the_librarys_status_and_lets_other_threads_run(stand_ins):
    """Stand-ins for the entry points: nothing is launched."""
    import ctypes
    status = bl.load_library().bitlinear_abi_version
    stand_ins(status)
    assert serving_calls() == dict.fromkeys(bl._SERVING, status())
    stand_ins(ctypes.pythonapi.PyGILState_Check)
    assert serving_calls() == dict.fromkeys(bl._SERVING, 0)
    assert ctypes.pythonapi.PyGILState_Check() == 1


# ------------------------------------------------------------------ largest sizes, and calls at the same time


@pytest.mark.parametrize("fmt", attention_plain.FORMATS)
def test_pages_of_4096_tokens(fmt):
    lengths, page = [5000, 4096, 1], 4096
    cache, table = filled_cache(fmt, 3, 1, 16, lengths, page, 8)
    bounds, step = new_summary(cache)
    bl.bitlinear_kv_summarise(cache, (bounds, step), ints(table), ints([0, 0, 0]), ints(lengths))
    ids = [(table[b, j], min(page, n - j * page)) for b, n in enumerate(lengths) for j in range(-(-n // page))]
    want_b, want_s = plain.summaries(cache, *zip(*ids))
    at = [i for i, _ in ids]
    np.testing.assert_array_equal(bounds.cpu().numpy()[at], want_b)
    np.testing.assert_array_equal(step.cpu().numpy()[at], want_s)
    q = normal((3, 2, 16), 9)
    blocks = ints([[[1, 0]], [[0, -1]], [[0, 1]]])
    out = torch.empty(q.shape, device="cuda")
    bl.bitlinear_attention_blocks(q.cuda(), cache, ints(table), ints(lengths), blocks, out)
    want, bound = plain.attend_blocks(q.numpy(), cache, table, lengths, blocks.cpu().numpy(), page, 0.25)
    within(out, want, bound)


def test_as_many_blocks_as_there_may_be():
    """4096 of a row's columns in any order, most of them none."""
    page, L, rng = 16, 3000, np.random.default_rng(3)
    cache, table = filled_cache("int8", 2, 2, 80, [L, 40], page, 12)
    blocks = np.where(rng.random((2, 2, 4096)) < 0.02, rng.integers(0, table.shape[1], (2, 2, 4096)), rng.choice([-1, -2 ** 31, 2 ** 31 - 1, 10 ** 5], (2, 2, 4096)))
    q = normal((2, 6, 80), 13)
    out = torch.empty(q.shape, device="cuda")
    bl.bitlinear_attention_blocks(q.cuda(), cache, ints(table), ints([L, 40]), ints(blocks), out)
    want, bound = plain.attend_blocks(q.numpy(), cache, table, [L, 40], blocks, page, 80 ** -0.5)
    within(out, want, bound)


def test_as_many_drafts_as_there_may_be():
    K, V = 65535, 8
    p = probabilities((1, K + 1, V), 5)
    q, uniform = p[:, :K].clone(), torch.rand(1, K + 1, generator=torch.Generator().manual_seed(6))
    draft = torch.randint(0, V, (1, K), dtype=torch.int32, generator=torch.Generator().manual_seed(7))
    for refused in (None, 65000):
        if refused is not None:
            q[0, refused], uniform[0, refused] = 1.0, 0.999
        tokens, accepted = torch.empty(1, K + 1, dtype=torch.int32, device="cuda"), torch.empty(1, dtype=torch.int32, device="cuda")
        bl.bitlinear_verify(p.cuda(), q.cuda(), draft.cuda(), uniform.cuda(), tokens, accepted)
        want_tokens, want_accepted = plain.verify(p.numpy(), q.numpy(), draft.numpy(), uniform.numpy())
        np.testing.assert_array_equal(tokens.cpu().numpy(), want_tokens)
        assert accepted.item() == want_accepted[0] == (K if refused is None else refused)


def test_calls_at_the_same_time():
    """Two streams, each with calls of its own on its own workspace, beside matrix products on the tensor cores: the bits of each alone."""
    cases = [("bf16", 1, 64, 32, 8, 128, [700]), ("int8", 4, 10, 16, 16, 80, [900, 500, 40, 333])]
    runs = []
    for i, (fmt, groups, R, Hq, Hkv, D, shared) in enumerate(cases):
        lengths = np.repeat(shared, R) + np.random.default_rng(i).integers(1, 60, groups * R)
        cache, q, table = shared_case(fmt, groups, R, Hq, Hkv, D, shared, lengths, 32, 60 + i)
        ws = torch.empty(bl.bitlinear_attention_shared_workspace(groups * R, Hq, Hkv, D, groups), dtype=torch.uint8, device="cuda")
        y = torch.randn(40, 50000, device="cuda")
        args = q.cuda(), cache, wide_table(table, cache), ints(lengths), ints(shared)
        alone = torch.empty(q.shape, device="cuda"), torch.empty_like(y)
        bl.bitlinear_attention_shared(*args, alone[0], ws)
        bl.bitlinear_softmax(y, alone[1])
        runs.append((args, ws, y, alone, torch.cuda.Stream()))
    W = torch.randn(1024, 1024, device="cuda")
    packed, sw = torch.empty(bl.bitlinear_packed_bytes(1024, 1024), dtype=torch.uint8, device="cuda"), torch.empty(1, device="cuda")
    bl.bitlinear_quantize_weights(W, packed, sw, torch.empty(bl.bitlinear_quantize_weights_workspace(1024, 1024), dtype=torch.uint8, device="cuda"))
    x, third = torch.randn(512, 1024, device="cuda"), torch.cuda.Stream()
    xq, sx, y0, y1 = torch.empty(512, 1024, dtype=torch.int8, device="cuda"), torch.empty(512, device="cuda"), torch.empty(512, 1024, device="cuda"), torch.empty(512, 1024, device="cuda")
    bl.bitlinear_linear(x, [(packed, sw, y0)], xq, sx)
    torch.cuda.synchronize()
    got = [[(torch.empty_like(alone[0]), torch.empty_like(alone[1])) for _ in range(6)] for _, _, _, alone, _ in runs]
    torch.cuda.synchronize()
    for turn in range(6):
        for (args, ws, y, _, stream), outs in zip(runs, got):
            with torch.cuda.stream(stream):
                bl.bitlinear_attention_shared(*args, outs[turn][0], ws, flags=bl.FLAG_PDL)
                bl.bitlinear_softmax(y, outs[turn][1], flags=bl.FLAG_PDL)
        with torch.cuda.stream(third):
            bl.bitlinear_linear(x, [(packed, sw, y1)], xq, sx)
    torch.cuda.synchronize()
    for (_, _, _, alone, _), outs in zip(runs, got):
        for o in outs:
            assert torch.equal(o[0], alone[0]) and torch.equal(o[1], alone[1])
    assert torch.equal(y0, y1)
    assert bl.bitlinear_device_status() == 0


@pytest.mark.parametrize("columns", [1, 31, 32, 33, 63, 64, 65])
@pytest.mark.parametrize("count", [1, 32, 256, 257])
def test_select_of_few_pages(columns, count):
    """Both sides of the borders between what a warp ranks and what bins find, with ties, absent pages and short rows."""
    page, D, B, rng = 16, 80, 6, np.random.default_rng(columns + count)
    q = normal((B, 4, D), columns).numpy()
    bounds, step = random_summary(9, 2, D, count)  # few pages that the tables repeat: ties
    table = rng.integers(0, 9, (B, columns))
    table[rng.random(table.shape) < 0.1] = -1
    lengths = [columns * page, columns * page - 9, 1, 0, rng.integers(1, columns * page + 1), 10 ** 6]
    for keep in ((0, 0), (1, 1), (3, 40)):
        got = run_select(q, bounds, step, table, lengths, page, *keep, count)
        for b in range(B):
            np.testing.assert_array_equal(got[b], plain.choose(q[b], bounds, step, table[b], lengths[b], page, *keep, count), err_msg=f"{keep} {b}")


@pytest.mark.parametrize("fmt", attention_plain.FORMATS)
@pytest.mark.parametrize("page,groups,R,D,S", [(128, 1, 40, 96, 700), (512, 2, 24, 128, 1300), (4096, 1, 70, 64, 5000), (16, 3, 50, 112, 300), (32, 60, 24, 32, 130)])
def test_shared_on_the_tensor_cores_of_any_page_size(fmt, page, groups, R, D, S):
    """A tile's part of a page: from 16 tokens to the whole tile; one group in equal runs, a few by their tokens, many with as many CTAs as fit."""
    rng = np.random.default_rng(page)
    shared = rng.integers(S // 2, S + 1, groups)
    shared[-1] = S
    run_shared(fmt, groups, R, 4, 2, D, shared, np.repeat(shared, R) + rng.integers(0, 20, groups * R), page, seed=page)
