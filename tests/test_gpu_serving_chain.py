"""The operators of a serving step as they are used, in captured graphs with programmatic dependent launch:

    several drafted tokens of each sequence:
    x -> RMSNorm + [q || k || v] -> rotate, write the cache -> attention of rows that share -> o -> LM head -> softmax -> verify
    one token of each sequence of a long context:
    x -> [q || k || v] -> rotate, write the cache -> summarise its page -> choose pages -> attention over them -> o

Every operator's output is checked against its plain form of what the GPU itself handed to it, after every replay:
an ordering fault between any two launches shows as a mismatch."""
import numpy as np
import pytest
import torch

import attention_plain
import bitlinear_w1_a8_gb300 as bl
import oracle
import serving_plain as plain
from bitlinear_w1_a8_gb300 import synth
from test_gpu_attention_chain import DIM, HEAD, HEADS, quantised
from test_gpu_serving import ints, wide_table, within

pytestmark = pytest.mark.gpu


def f32(*shape):
    return torch.empty(*shape, device="cuda")


def captured(step, restore):
    """The step in a graph, after one eager run whose writes `restore` undoes."""
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        step(stream)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step(stream)
    torch.cuda.synchronize()
    restore()
    torch.cuda.synchronize()
    return graph


def filled(fmt, kv_heads, table, start, page, seed):
    cache = attention_plain.make_cache(fmt, int(table.max()) + 1, kv_heads, page, HEAD, seed)
    g = torch.Generator().manual_seed(seed)
    for b in range(len(start)):
        t = torch.arange(int(start[b]), device="cuda")
        k, v = (torch.randn(len(t), kv_heads, HEAD, generator=g).cuda() for _ in "kv")
        attention_plain.fill_row(cache, fmt, torch.tensor(table[b], device="cuda").long()[t // page], t % page, k, v)
    return cache


def o_is_right(out, oq, so, acc, o_w):
    rows = out.reshape(-1, DIM).cpu().numpy()
    codes, scales = oracle.act_quant(rows)
    np.testing.assert_array_equal(oq.cpu().numpy(), codes)
    np.testing.assert_array_equal(so.cpu().numpy(), scales)
    want, _ = oracle.forward(codes, scales, o_w[0].cpu().numpy(), float(o_w[1]), DIM, DIM)
    np.testing.assert_array_equal(acc.cpu().numpy(), want)


@pytest.mark.parametrize("fmt", attention_plain.FORMATS)
@pytest.mark.parametrize("B,K,kv_heads,start", [(2, 4, 8, [40, 93]), (3, 2, 2, [0, 30, 250]), (1, 20, 4, [200]), (2, 60, 8, [70, 300])])
def test_drafted_tokens_from_logits_to_tokens(fmt, B, K, kv_heads, start):
    bl.load_library()
    page, R, V, steps = 16, K + 1, 320, 3
    M = B * R
    width = -(-(max(start) + (steps + 1) * R) // page)
    q_w, k_w, v_w, o_w, head_w = (quantised(n, DIM, 50 + i) for i, n in enumerate((DIM, kv_heads * HEAD, kv_heads * HEAD, DIM, V)))
    gamma = synth.uniform((DIM,), 0.5, 1.5, 60).cuda()
    x, q, k, v, out, y, logits, p = f32(M, DIM), f32(M, DIM), f32(M, kv_heads * HEAD), f32(M, kv_heads * HEAD), f32(M, HEADS, HEAD), f32(M, DIM), f32(M, V), f32(M, V)
    acc = torch.empty(M, DIM, dtype=torch.int32, device="cuda")
    xq, sx, oq, so, yq, sy = (t for _ in range(3) for t in (torch.empty(M, DIM, dtype=torch.int8, device="cuda"), f32(M)))
    g = torch.Generator().manual_seed(9)
    own = np.random.default_rng(1).permutation(B * width).reshape(B, width)
    cache = filled(fmt, kv_heads, own, start, page, 7)
    # a row is a drafted token; those of a sequence have its pages
    table_rows = np.repeat(own, R, 0)
    table = wide_table(table_rows, cache)  # of as many columns as make the rows share
    position = np.concatenate([s + np.arange(R) for s in start])
    positions, lengths, shared = ints(position), ints(position + 1), ints(np.asarray(start) + R)
    rope = (bl.bitlinear_rope_frequencies(HEAD).cuda(), bl.ROPE_HALF)
    ws = torch.empty(bl.bitlinear_attention_shared_workspace(M, HEADS, kv_heads, HEAD, B), dtype=torch.uint8, device="cuda")
    temperature = torch.rand(M, generator=g).cuda() + 0.5
    temperature[0] = 0.0
    drafted = torch.softmax(torch.randn(B, K, V, generator=g) * 0.5, -1).cuda()
    draft, uniform = torch.randint(0, V, (B, K), generator=g, dtype=torch.int32).cuda(), torch.rand(B, R, generator=g).cuda()
    tokens, accepted = torch.empty(B, R, dtype=torch.int32, device="cuda"), torch.empty(B, dtype=torch.int32, device="cuda")
    rows = lambda a: a.view(M, -1, HEAD)  # noqa: E731

    def step(stream):
        pdl = dict(flags=bl.FLAG_PDL, stream=stream)
        bl.bitlinear_linear(x, [(*q_w, q), (*k_w, k), (*v_w, v)], xq, sx, rms_weight=gamma, **pdl)
        bl.bitlinear_kv_append(rows(k), rows(v), cache, positions, table, q=rows(q), q_out=rows(q), rope=rope, **pdl)
        bl.bitlinear_attention_shared(rows(q), cache, table, lengths, shared, out, ws, **pdl)
        bl.bitlinear_linear(out.view(M, DIM), [(*o_w, y, acc)], oq, so, **pdl)
        bl.bitlinear_linear(y, [(*head_w, logits)], yq, sy, **pdl)
        bl.bitlinear_softmax(logits, p, temperature, **pdl)
        bl.bitlinear_verify(p.view(B, R, V), drafted, draft, uniform, tokens, accepted, **pdl)

    before = [None if c is None else c.clone() for c in cache]
    first = synth.activations(M, DIM, 70).cuda()
    x.copy_(first)
    graph = captured(step, lambda: [now.copy_(was) for now, was in zip(cache, before) if now is not None])
    taken = 0
    for _ in range(steps):
        graph.replay()
        torch.cuda.synchronize()
        want, bound = attention_plain.attend(rows(q).cpu().numpy(), cache, table_rows, lengths.cpu().numpy(), page, HEAD ** -0.5)
        within(out, want, bound)
        o_is_right(out, oq, so, acc, o_w)
        want, bound = plain.softmax(logits.cpu().numpy(), temperature.cpu().numpy())
        within(p, want, bound)
        want_tokens, want_accepted = plain.verify(p.view(B, R, V).cpu().numpy(), drafted.cpu().numpy(), draft.cpu().numpy(), uniform.cpu().numpy())
        np.testing.assert_array_equal(tokens.cpu().numpy(), want_tokens)
        np.testing.assert_array_equal(accepted.cpu().numpy(), want_accepted)
        # every sequence goes on behind what was taken of its drafts; the rest is written again
        on = accepted + 1
        taken += int(on.sum())
        positions += on.repeat_interleave(R)
        lengths += on.repeat_interleave(R)
        shared += on
        x.copy_(y + first)
        uniform.copy_(torch.rand(B, R, generator=g))
        torch.cuda.synchronize()
    assert taken >= steps * B
    assert bl.bitlinear_device_status() == 0


@pytest.mark.parametrize("fmt", attention_plain.FORMATS)
@pytest.mark.parametrize("B,kv_heads,start,count,window", [(1, 8, [30], 2, (1, 1)), (3, 2, [61, 0, 300], 6, (1, 2)), (2, 4, [500, 95], 8, (0, 0))])
def test_long_contexts_over_chosen_pages(fmt, B, kv_heads, start, count, window):
    bl.load_library()
    page, steps = 16, 4
    width = -(-(max(start) + steps) // page)
    q_w, k_w, v_w, o_w = (quantised(n, DIM, 50 + i) for i, n in enumerate((DIM, kv_heads * HEAD, kv_heads * HEAD, DIM)))
    x, q, k, v, out, y = f32(B, DIM), f32(B, DIM), f32(B, kv_heads * HEAD), f32(B, kv_heads * HEAD), f32(B, HEADS, HEAD), f32(B, DIM)
    acc = torch.empty(B, DIM, dtype=torch.int32, device="cuda")
    xq, sx, oq, so = (t for _ in range(2) for t in (torch.empty(B, DIM, dtype=torch.int8, device="cuda"), f32(B)))
    own = np.random.default_rng(2).permutation(B * width).reshape(B, width)
    cache, table = filled(fmt, kv_heads, own, start, page, 11), ints(own)
    pages = cache[0].shape[0]
    summary = torch.full((pages, kv_heads, 2, HEAD), 55, dtype=torch.int8, device="cuda"), torch.full((pages, kv_heads), 3.0, device="cuda")
    bl.bitlinear_kv_summarise(cache, summary, table, ints(np.zeros(B)), ints(start))  # the prompts' pages
    positions, lengths = ints(start), ints(np.asarray(start) + 1)
    blocks = torch.empty(B, kv_heads, count, dtype=torch.int32, device="cuda")
    rope = (bl.bitlinear_rope_frequencies(HEAD).cuda(), bl.ROPE_HALF)
    rows = lambda a: a.view(B, -1, HEAD)  # noqa: E731

    def step(stream):
        pdl = dict(flags=bl.FLAG_PDL, stream=stream)
        bl.bitlinear_linear(x, [(*q_w, q), (*k_w, k), (*v_w, v)], xq, sx, **pdl)
        bl.bitlinear_kv_append(rows(k), rows(v), cache, positions, table, q=rows(q), q_out=rows(q), rope=rope, **pdl)
        bl.bitlinear_kv_summarise(cache, summary, table, positions, lengths, **pdl)
        bl.bitlinear_attention_select(rows(q), cache, summary, table, lengths, blocks, *window, **pdl)
        bl.bitlinear_attention_blocks(rows(q), cache, table, lengths, blocks, out, **pdl)
        bl.bitlinear_linear(out.view(B, DIM), [(*o_w, y, acc)], oq, so, **pdl)

    kept = [None if c is None else c.clone() for c in (*cache, *summary)]
    first = synth.activations(B, DIM, 71).cuda()
    x.copy_(first)
    graph = captured(step, lambda: [now.copy_(was) for now, was in zip((*cache, *summary), kept) if now is not None])
    for _ in range(steps):
        graph.replay()
        torch.cuda.synchronize()
        n = lengths.cpu().numpy()
        bounds, scales = (s.cpu().numpy() for s in summary)
        for b in range(B):
            columns = -(-n[b] // page)
            want_bounds, want_scales = plain.summaries(cache, own[b, :columns], [min(page, n[b] - page * j) for j in range(columns)])
            np.testing.assert_array_equal(bounds[own[b, :columns]], want_bounds)
            np.testing.assert_array_equal(scales[own[b, :columns]], want_scales)
            chosen = plain.choose(rows(q)[b].cpu().numpy(), bounds, scales, own[b], n[b], page, *window, count)
            np.testing.assert_array_equal(blocks[b].cpu().numpy(), chosen)
        want, bound = plain.attend_blocks(rows(q).cpu().numpy(), cache, own, n, blocks.cpu().numpy(), page, HEAD ** -0.5)
        within(out, want, bound)
        o_is_right(out, oq, so, acc, o_w)
        positions += 1
        lengths += 1
        x.copy_(y + first)
        torch.cuda.synchronize()
    assert bl.bitlinear_device_status() == 0


def test_two_graphs_share_a_workspace():
    """Captured calls of different shapes on one workspace, replayed in turn: each writes all that it reads of it."""
    from test_gpu_serving import shared_case
    cases = [("int8", 1, 40, 8, 8, 80, [300]), ("bf16", 1, 64, 8, 2, 128, [200]), ("fp8", 4, 6, 8, 8, 64, [90, 40, 0, 33])]
    calls, need = [], 0
    for i, (fmt, groups, R, Hq, Hkv, D, shared) in enumerate(cases):
        lengths = np.repeat(shared, R) + np.random.default_rng(i).integers(1, 40, groups * R)
        cache, q, table = shared_case(fmt, groups, R, Hq, Hkv, D, shared, lengths, 16, 90 + i)
        need = max(need, bl.bitlinear_attention_shared_workspace(groups * R, Hq, Hkv, D, groups))
        calls.append((cache, q.cuda(), table, lengths, ints(lengths), ints(shared), torch.empty(q.shape, device="cuda"), wide_table(table, cache)))
    ws = torch.full((need,), 0xff, dtype=torch.uint8, device="cuda")
    graphs = []
    for cache, q, _, _, n, shared, out, columns in calls:
        bl.bitlinear_attention_shared(q, cache, columns, n, shared, out, ws)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            bl.bitlinear_attention_shared(q, cache, columns, n, shared, out, ws, flags=bl.FLAG_PDL)
        graphs.append(graph)
    for order in ((0, 1, 2), (2, 0, 1), (1, 0, 2, 1)):
        for call in calls:
            call[6].fill_(float("nan"))
        for i in order:
            graphs[i].replay()
        torch.cuda.synchronize()
        for cache, q, table, lengths, _, _, out, _ in calls:
            want, bound = attention_plain.attend(q.cpu().numpy(), cache, table, lengths, 16, q.shape[-1] ** -0.5)
            within(out, want, bound)
