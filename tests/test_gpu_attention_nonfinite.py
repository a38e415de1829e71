"""What a NaN or an infinity does to bitlinear_attention's outputs: the heads that meet it show it, the others are
bit for bit as without it.  On each of the ways that a row's parts meet: one CTA, a cluster, shared out with a
workspace."""
import numpy as np
import pytest
import torch

import attention_plain as plain
import bitlinear_w1_a8_gb300 as bl
from harness import guarded

pytestmark = pytest.mark.gpu

NAN, INF = float("nan"), float("inf")
PAGE, HK, GROUP, D = 16, 2, 4, 64
# lengths, columns of the table, workspace
PATHS = {"one CTA": ([70, 33] * 200, 5, False), "cluster": ([900, 250], 64, False), "shared out": ([900, 250, 0], 4096, True)}


def case(fmt, path):
    lengths, cols, workspace = PATHS[path]
    B, n = len(lengths), max(lengths)
    own = -(-n // PAGE)
    pages = 2 * own
    cache = plain.make_cache(fmt, pages, HK, PAGE, D, 1)
    g = torch.Generator(device="cuda").manual_seed(2)
    t = torch.arange(pages * PAGE, device="cuda")
    plain.fill_row(cache, fmt, t // PAGE, t % PAGE, torch.randn(len(t), HK, D, generator=g, device="cuda"),
                   torch.randn(len(t), HK, D, generator=g, device="cuda"))
    table = torch.full((B, cols), -1, dtype=torch.int32)
    table[:, :own] = torch.arange(own)
    table[0, :own] += own   # the first sequence has pages of its own
    need = bl.bitlinear_attention_workspace(B, GROUP * HK, HK, D) if workspace else 0
    assert bool(need) == workspace
    ws, full = guarded(need, torch.uint8, 0x3C) if need else (None, None)
    q = torch.randn(B, GROUP * HK, D, generator=g, device="cuda")

    def run():
        out = torch.full_like(q, -7.0)
        if ws is not None:
            ws.fill_(0x3C)
        bl.bitlinear_attention(q, cache, table.cuda(), torch.tensor(lengths, dtype=torch.int32, device="cuda"), out, workspace=ws)
        if ws is not None:
            assert (ws != 0x3C).any()   # the workspace's path was taken
        return out

    return q, cache, own, run


def check(clean, got, poisoned):
    """`poisoned` [B, heads] of the outputs are not finite in any dim, the rest as before."""
    assert torch.isfinite(clean).all()
    assert torch.equal(got[~poisoned], clean[~poisoned])
    assert not torch.isfinite(got[poisoned]).any()


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("fmt", plain.FORMATS)
def test_q(fmt, path):
    q, cache, own, run = case(fmt, path)
    clean = run()
    poisoned = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
    for (b, h, d), x in {(0, 1, 5): NAN, (1, 6, 63): NAN, (1, 0, 0): INF, (0, 7, 33): -INF}.items():
        q[b, h, d] = x
        poisoned[b, h] = True
    check(clean, run(), poisoned)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("fmt", plain.FORMATS)
@pytest.mark.parametrize("at", [0, 37, 69])
def test_keys_and_values(fmt, path, at):
    """Of the first sequence's token `at` (69: the last of 70, in a step that is not whole), one key head."""
    for which, x in ((0, NAN), (1, NAN), (1, INF)):
        q, cache, own, run = case(fmt, path)
        clean = run()
        page, head = own + at // PAGE, 1
        held = cache[which][page, head, at % PAGE]
        if fmt == "bf16":
            held.fill_(x)
        else:
            cache[2 + which][page, head, at % PAGE] = x
            if fmt == "fp8":
                held.view(torch.uint8).fill_(0x38)  # 1: an infinity times a code of 0 aside
            else:
                held.fill_(1)
        poisoned = torch.zeros(q.shape[:2], dtype=torch.bool, device="cuda")
        poisoned[0, GROUP * head:GROUP * (head + 1)] = True
        check(clean, run(), poisoned)


@pytest.mark.parametrize("path", PATHS)
@pytest.mark.parametrize("fmt", plain.FORMATS)
def test_a_row_without_tokens_is_zeros_whatever_q_is(fmt, path):
    lengths, cols, workspace = PATHS[path]
    B = len(lengths)
    cache = plain.make_cache(fmt, 4, HK, PAGE, D, 1)
    q = torch.full((B, GROUP * HK, D), NAN, device="cuda")
    table = torch.full((B, cols), 9, dtype=torch.int32, device="cuda")   # no such page
    out = torch.full_like(q, -7.0)
    ws = torch.empty(bl.bitlinear_attention_workspace(B, GROUP * HK, HK, D), dtype=torch.uint8, device="cuda") if workspace else None
    n = torch.tensor(np.where(np.arange(B) % 2, 0, lengths), dtype=torch.int32, device="cuda")
    bl.bitlinear_attention(q, cache, table, n, out, workspace=ws)
    assert (out == 0).all()
