"""bitlinear_attention's way with a workspace, rows shared out over the whole GPU and joined by a second launch:
windows, many sequences, pages out of range, and calls that follow one another.  Every call here asserts that its
workspace was written, which no other way does."""
import numpy as np
import pytest
import torch

import attention_plain as plain
import bitlinear_w1_a8_gb300 as bl
from harness import check_canary, guarded

pytestmark = pytest.mark.gpu

POOL = 230   # pages, each filled; a sequence's table names them in an order of its own


def ints(values):
    return torch.tensor(np.asarray(values), dtype=torch.int32, device="cuda")


def within(got, want, bound):
    got = got.double().cpu().numpy()
    assert np.isfinite(got).all()
    off = np.abs(got - want) - bound
    assert (off <= 0).all(), f"{(off > 0).sum()} of {off.size} beyond the bound, worst by {off.max():.3g}"


class Case:
    def __init__(self, fmt, Hq, Hk, D, page, lengths, columns, window=0, seed=0, no_page=0.0):
        self.page, self.window, self.lengths = page, window, list(lengths)
        B, g, rng = len(lengths), torch.Generator(device="cuda").manual_seed(seed), np.random.default_rng(seed)
        self.cache = plain.make_cache(fmt, POOL, Hk, page, D, seed)
        t = torch.arange(POOL * page, device="cuda")
        plain.fill_row(self.cache, fmt, t // page, t % page, *(torch.randn(len(t), Hk, D, generator=g, device="cuda") for _ in "kv"))
        own = min(columns, -(-max(1, max(lengths)) // page))
        self.table = rng.integers(-2 ** 31, 2 ** 31 - 1, (B, columns))   # past the longest sequence: anything
        self.table[:, :own] = rng.integers(0, POOL, (B, own))
        if no_page:
            gone = rng.random((B, own)) < no_page
            self.table[:, :own][gone] = rng.choice([-1, POOL, 2 ** 31 - 1], int(gone.sum()))
        self.own = own
        self.q = torch.randn(B, Hq, D, generator=g, device="cuda") * 1.5
        self.device_table, self.device_lengths = ints(self.table), ints(self.lengths)
        self.out, self.out_full = guarded(B * Hq * D, torch.float32, -7.0)
        self.out = self.out.view(B, Hq, D)
        need = bl.bitlinear_attention_workspace(B, Hq, Hk, D)
        assert need > 0
        self.ws, self.ws_full = guarded(need, torch.uint8, 0x3C)

    def call(self, ws=None, out=None, q=None, lengths=None, **kw):
        bl.bitlinear_attention(self.q if q is None else q, self.cache, self.device_table,
                               self.device_lengths if lengths is None else lengths, self.out if out is None else out,
                               workspace=self.ws if ws is None else ws, window=self.window, **kw)

    def took_the_way(self):
        assert (self.ws != 0x3C).any()
        check_canary(self.ws_full, 0x3C)
        check_canary(self.out_full, -7.0)

    def exact(self, q=None, lengths=None):
        q = self.q if q is None else q
        return plain.attend(q.cpu().numpy(), self.cache, self.table[:, :self.own], self.lengths if lengths is None else lengths,
                            self.page, q.shape[-1] ** -0.5, self.window)

    def check(self):
        self.call()
        self.took_the_way()
        within(self.out, *self.exact())


@pytest.mark.parametrize("fmt", plain.FORMATS)
@pytest.mark.parametrize("Hq,Hk,D,page,lengths,window", [
    (2, 1, 64, 64, [40017, 3, 0, 33000, 52000], 40000),          # 16 CTAs a row: 64 warps
    (4, 2, 80, 256, [52000, 52001], 33333), (2, 2, 128, 256, [50001, 33, 1], 34001), (9, 1, 96, 256, [45000, 1], 33000)])
def test_windows(fmt, Hq, Hk, D, page, lengths, window):
    """Wide enough for this way, with sequences that begin inside it, at it and inside a step."""
    Case(fmt, Hq, Hk, D, page, lengths, 65536 // page, window=window, seed=D).check()


@pytest.mark.parametrize("fmt", plain.FORMATS)
@pytest.mark.parametrize("B,Hk,columns,window,no_page", [(150, 1, 2048, 0, 0.0), (33, 4, 2048, 0, 0.2), (65, 2, 2048, 0, 0.0),
                                                         (100, 1, 2048, 9000, 0.0), (150, 1, 4096, 0, 0.5)])
def test_many_sequences(fmt, B, Hk, columns, window, no_page):
    """Several sequences a lane in the search for a CTA's row; most short, some empty, a few long."""
    rng = np.random.default_rng(B)
    lengths = rng.integers(0, 90, B)
    lengths[rng.permutation(B)[:B // 5]] = 0
    lengths[rng.permutation(B)[:4]] = [12000, 5000, 9001, 700]
    lengths[rng.permutation(B)[:2]] = [-4, 1]
    c = Case(fmt, 2 * Hk, Hk, 64, 16, lengths, columns, window=window, seed=B, no_page=no_page)
    c.check()
    assert (c.out[torch.tensor(np.array(c.lengths) <= 0)] == 0).all()


@pytest.mark.parametrize("fmt", plain.FORMATS)
def test_rows_whose_every_page_is_gone(fmt):
    c = Case(fmt, 4, 2, 80, 16, [3000, 40, 3000], 65536 // 16, seed=3)
    c.table[0] = c.table[1] = -1
    c.device_table = ints(c.table)
    c.check()
    assert (c.out[:2] == 0).all() and (c.out[2] != 0).any()


def variants(c, n):
    """n calls' q and lengths: of every mix of long, short and empty sequences."""
    g, rng = torch.Generator(device="cuda").manual_seed(9), np.random.default_rng(9)
    top = max(c.lengths)
    return [(torch.randn(*c.q.shape, generator=g, device="cuda"),
             ints(rng.choice([0, 1, 17, top // 3, top - 1, top], len(c.lengths)))) for _ in range(n)]


def fresh(c):
    """Each variant's output by a call of its own with a workspace of its own, checked against 64 bits."""
    def one(q, lengths):
        out, ws = torch.full_like(q, -7.0), torch.full_like(c.ws, 0x3C)
        c.call(ws=ws, out=out, q=q, lengths=lengths)
        torch.cuda.synchronize()
        if (lengths > 0).any():
            assert (ws != 0x3C).any()
        within(out, *c.exact(q, lengths.tolist()))
        return out
    return one


@pytest.mark.parametrize("fmt", plain.FORMATS)
def test_calls_in_a_row_share_one_workspace(fmt):
    """Programmatic launches back to back: each call's parts are written while the last call's join may read its own."""
    c = Case(fmt, 8, 2, 80, 64, [6000, 700, 33, 2500], 65536 // 64, seed=1)
    calls = variants(c, 8)
    want = [fresh(c)(q, n) for q, n in calls]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(10):
        got = [torch.full_like(o, -7.0) for o in want]
        torch.cuda.synchronize()
        for (q, n), o in zip(calls, got):
            c.call(out=o, q=q, lengths=n, flags=bl.FLAG_PDL, stream=stream)
        torch.cuda.synchronize()
        for a, b in zip(got, want):
            assert torch.equal(a, b)
    c.took_the_way()


@pytest.mark.parametrize("fmt", plain.FORMATS)
def test_one_replayed_graph(fmt):
    """Two calls on one workspace in a graph, whose q and lengths change between replays."""
    c = Case(fmt, 8, 2, 128, 64, [6000, 700, 33, 2500], 65536 // 64, seed=2)
    calls = variants(c, 6)
    want = [fresh(c)(q, n) for q, n in calls]
    q, n = [c.q.clone() for _ in "ab"], [c.device_lengths.clone() for _ in "ab"]
    outs = [torch.full_like(c.q, -7.0) for _ in "ab"]
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            for i in range(2):
                c.call(out=outs[i], q=q[i], lengths=n[i], flags=bl.FLAG_PDL, stream=stream)
    for first in (0, 2, 4, 1, 3):
        for i in range(2):
            q[i].copy_(calls[first + i][0])
            n[i].copy_(calls[first + i][1])
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        for i in range(2):
            assert torch.equal(outs[i], want[first + i])
    c.took_the_way()


def test_streams_with_a_workspace_each_and_repeats():
    cases = [Case("int8", 8, 2, 80, 64, [6000, 700, 33, 2500], 65536 // 64, seed=4),
             Case("bf16", 4, 1, 128, 64, [14000], 131072 // 64, seed=5)]
    want = []
    for c in cases:
        c.check()
        want.append(c.out.clone())
    streams = [torch.cuda.Stream() for _ in cases]
    outs = [[torch.full_like(w, -7.0) for _ in range(25)] for w in want]
    torch.cuda.synchronize()
    for i in range(25):
        for c, s, o in zip(cases, streams, outs):
            c.call(out=o[i], stream=s, flags=bl.FLAG_PDL * (i % 2))
    torch.cuda.synchronize()
    for w, o in zip(want, outs):
        for x in o:
            assert torch.equal(x, w)


@pytest.mark.parametrize("fmt", plain.FORMATS)
def test_decode_steps_with_a_wide_table(fmt):
    """Cache writes and attention of one graph, both programmatic, a token further each replay."""
    B, Hq, Hk, D, page, start, steps = 3, 8, 2, 64, 16, 2000, 12
    c = Case(fmt, Hq, Hk, D, page, [start] * B, 65536 // page, seed=6)
    own = -(-(start + steps) // page)
    table = np.full_like(c.table, -1)
    table[:, :own] = np.random.default_rng(7).permutation(B * own).reshape(B, own)
    cache = plain.make_cache(fmt, B * own, Hk, page, D, 8)
    for i in range(len(cache)):   # the first tokens from the pool
        if cache[i] is not None:
            raw = cache[i].view(torch.uint8) if cache[i].element_size() == 1 else cache[i]
            src = c.cache[i].view(torch.uint8) if cache[i].element_size() == 1 else c.cache[i]
            raw.copy_(src[torch.arange(B * own, device="cuda") % POOL])
    c.cache, c.table, c.own, c.device_table = cache, table, own, ints(table)
    q, k, v = (torch.empty(B, h, D, device="cuda") for h in (Hq, Hk, Hk))
    positions, lengths = ints([start] * B), ints([start + 1] * B)
    rope = (bl.bitlinear_rope_frequencies(D).cuda(), bl.ROPE_HALF)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.stream(stream):
        with torch.cuda.graph(graph, stream=stream):
            bl.bitlinear_kv_append(k, v, cache, positions, c.device_table, q=q, q_out=q, rope=rope, flags=bl.FLAG_PDL, stream=stream)
            c.call(q=q, lengths=lengths, flags=bl.FLAG_PDL, stream=stream)
    g = torch.Generator(device="cuda").manual_seed(1)
    for i in range(steps):
        for x in (q, k, v):
            x.copy_(torch.randn(*x.shape, generator=g, device="cuda"))
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        within(c.out, *c.exact(q, [start + 1 + i] * B))
        positions += 1
        lengths += 1
    c.took_the_way()
    assert bl.bitlinear_device_status() == 0
