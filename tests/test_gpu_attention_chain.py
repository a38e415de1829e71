"""The attention of a block as a decode step uses it, one captured graph replayed for several tokens:

    x -> RMSNorm + [q || k || v] -> rotate, write the cache -> attention -> o -> the next token's x

with programmatic dependent launch throughout, positions and lengths advanced between replays.  After every
replay the attention of that step is checked against the 64-bit form over the GPU's own cache, the written rows
against the GPU's own k and v, and the o call's int8 activations and accumulators against the oracle's of the
attention's output: an ordering fault between any two launches shows as a mismatch."""
import numpy as np
import pytest
import torch

import attention_plain as plain
import bitlinear_w1_a8_gb300 as bl
import oracle
from bitlinear_w1_a8_gb300 import synth

pytestmark = pytest.mark.gpu

HEADS, HEAD = 8, 80
DIM = HEADS * HEAD


def quantised(N, K, seed):
    W = synth.weight(N, K, seed)
    packed = torch.empty(bl.bitlinear_packed_bytes(N, K), dtype=torch.uint8, device="cuda")
    sw = torch.empty(1, device="cuda")
    ws = torch.empty(bl.bitlinear_quantize_weights_workspace(N, K), dtype=torch.uint8, device="cuda")
    bl.bitlinear_quantize_weights(W.cuda(), packed, sw, ws)
    return packed, sw


@pytest.mark.parametrize("fmt", plain.FORMATS)
@pytest.mark.parametrize("M,kv_heads,start,window", [(1, 8, 0, 0), (3, 2, 61, 0), (20, 8, 130, 100)])
def test_decode_steps_with_attention_in_one_graph(fmt, M, kv_heads, start, window):
    bl.load_library()
    page, steps = 16, 5
    width = -(-(start + steps) // page)
    q_w, k_w, v_w, o_w = (quantised(n, DIM, 50 + i) for i, n in enumerate((DIM, kv_heads * HEAD, kv_heads * HEAD, DIM)))
    gamma = synth.uniform((DIM,), 0.5, 1.5, 60).cuda()
    f32 = lambda *s: torch.empty(*s, device="cuda")  # noqa: E731
    x, q, k, v, out, y = f32(M, DIM), f32(M, DIM), f32(M, kv_heads * HEAD), f32(M, kv_heads * HEAD), f32(M, HEADS, HEAD), f32(M, DIM)
    acc = torch.empty(M, DIM, dtype=torch.int32, device="cuda")
    xq, sx, oq, so = torch.empty(M, DIM, dtype=torch.int8, device="cuda"), f32(M), torch.empty(M, DIM, dtype=torch.int8, device="cuda"), f32(M)
    cache = plain.make_cache(fmt, M * width, kv_heads, page, HEAD, 7)
    table = torch.tensor(np.random.default_rng(1).permutation(M * width).reshape(M, width), dtype=torch.int32, device="cuda")
    t = torch.arange(start, device="cuda")
    g = torch.Generator().manual_seed(8)
    for b in range(M):
        plain.fill_row(cache, fmt, table[b].long()[t // page], t % page, torch.randn(start, kv_heads, HEAD, generator=g).cuda(),
                       torch.randn(start, kv_heads, HEAD, generator=g).cuda())
    before = [None if c is None else c.clone() for c in cache]
    positions = torch.full((M,), start, dtype=torch.int32, device="cuda")
    lengths = positions + 1
    rope = (bl.bitlinear_rope_frequencies(HEAD).cuda(), bl.ROPE_HALF)
    need = bl.bitlinear_attention_workspace(M, HEADS, kv_heads, HEAD)
    ws = torch.empty(need, dtype=torch.uint8, device="cuda") if need else None
    rows = lambda a: a.view(M, -1, HEAD)  # noqa: E731

    def step(stream):
        pdl = dict(flags=bl.FLAG_PDL, stream=stream)
        bl.bitlinear_linear(x, [(*q_w, q), (*k_w, k), (*v_w, v)], xq, sx, rms_weight=gamma, **pdl)
        bl.bitlinear_kv_append(rows(k), rows(v), cache, positions, table, q=rows(q), q_out=rows(q), rope=rope, **pdl)
        bl.bitlinear_attention(rows(q), cache, table, lengths, out, workspace=ws, window=window, **pdl)
        bl.bitlinear_linear(out.view(M, DIM), [(*o_w, y, acc)], oq, so, **pdl)

    first = synth.activations(M, DIM, 70).cuda()
    x.copy_(first)
    stream = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(stream):
        step(stream)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            step(stream)
    torch.cuda.synchronize()
    for now, was in zip(cache, before):  # the eager step wrote the first token: start again
        if now is not None:
            now.copy_(was)
    packed, scale = o_w[0].cpu().numpy(), float(o_w[1])
    for i in range(steps):
        graph.replay()
        torch.cuda.synchronize()
        n = lengths.cpu().numpy()
        assert (n == start + 1 + i).all()
        want, bound = plain.attend(rows(q).cpu().numpy(), cache, table.cpu().numpy(), n, page, HEAD ** -0.5, window)
        off = np.abs(out.double().cpu().numpy() - want) - bound
        assert (off <= 0).all(), off.max()
        page_of, at = plain.places(positions.cpu().numpy(), None, table.cpu().numpy(), page)
        held_v = plain.held(cache, "v")[page_of, :, at]
        top = np.abs(rows(v).cpu().numpy()).max(-1, keepdims=True)
        half = {"int8": top / 127 * 0.5, "fp8": np.maximum(np.abs(held_v) * 2.0 ** -4, top / 448 * 2.0 ** -10), "bf16": np.abs(held_v) * 2.0 ** -8}[fmt]
        assert (np.abs(held_v - rows(v).double().cpu().numpy()) <= half * 1.07 + top * 2.0 ** -20).all()
        oq_o, so_o = oracle.act_quant(out.view(M, DIM).cpu().numpy())
        np.testing.assert_array_equal(oq.cpu().numpy(), oq_o)
        np.testing.assert_array_equal(so.cpu().numpy(), so_o)
        acc_o, _ = oracle.forward(oq_o, so_o, packed, scale, DIM, DIM)
        np.testing.assert_array_equal(acc.cpu().numpy(), acc_o)
        x.copy_(y + first)
        positions += 1
        lengths += 1
        torch.cuda.synchronize()
    assert bl.bitlinear_device_status() == 0
