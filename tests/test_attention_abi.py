"""Refusals and host-side results of the attention entry points (CPU only: every call fails, or
returns for an empty batch, before it touches a GPU)."""
import ctypes
import math

import numpy as np
import pytest

import bitlinear_w1_a8_gb300 as bl
from bitlinear_w1_a8_gb300 import build as blbuild

A, U = 0x10000, 0x10004   # fake addresses, never dereferenced: 16-byte aligned and not
NULL, SHAPE, ALIGN, UNSUPPORTED, WORKSPACE = -1, -2, -3, -4, -7


@pytest.fixture(scope="module")
def lib():
    blbuild.build()
    return bl.load_library()


def pages(**kw):
    d = dict(k=A, v=A, k_step=A, v_step=A, num_pages=4, num_heads=2, page_size=16, head_dim=64, format=bl.KV_INT8)
    d.update(kw)
    return bl.BitLinearKVPages(*[d[f[0]] for f in bl.BitLinearKVPages._fields_])


def spec(**kw):
    d = dict(freq=A, rot_dim=64, layout=0, amplitude=1.0)
    d.update(kw)
    return bl.BitLinearRopeSpec(*[d[f[0]] for f in bl.BitLinearRopeSpec._fields_])


ROPE = dict(x=A, x_stride=128, T=3, H=2, D=64, positions=A, rope=spec(), y=A + 4096, y_stride=128, flags=0)
ROWS = dict(T=3, positions=A, seq=A, table=A, table_stride=5, num_seqs=2, max_pages=5)
APPEND = dict(q=A, q_stride=256, Hq=4, q_out=A, q_out_stride=256, k=A, k_stride=128, v=A, v_stride=128, **ROWS,
              rope=spec(), cache=pages(), flags=0)
READ = dict(cache=pages(), **ROWS, k_out=A, k_stride=128, v_out=A, v_stride=128, flags=0)
ATTEND = dict(q=A, q_stride=256, B=3, Hq=4, cache=pages(), table=A, table_stride=5, max_pages=5, lengths=A, window=0,
              scale=0.125, out=A, out_stride=256, workspace=None, workspace_bytes=0, flags=0)

BAD_PAGES = [(dict(k=None), NULL), (dict(v=None), NULL), (dict(k_step=None), NULL), (dict(v_step=None), NULL),
             (dict(k=U), ALIGN), (dict(v_step=U), ALIGN), (dict(num_pages=0), SHAPE), (dict(num_pages=1 << 31), SHAPE),
             (dict(num_heads=0), SHAPE), (dict(num_heads=4097), SHAPE), (dict(page_size=8), SHAPE),
             (dict(page_size=48), SHAPE), (dict(page_size=8192), SHAPE), (dict(head_dim=8), SHAPE),
             (dict(head_dim=72), SHAPE), (dict(head_dim=272), SHAPE), (dict(format=3), UNSUPPORTED),
             (dict(num_pages=1 << 30, num_heads=64, page_size=64, head_dim=64), SHAPE)]
BAD_ROPE = [(dict(freq=None), NULL), (dict(freq=U), ALIGN), (dict(rot_dim=0), SHAPE), (dict(rot_dim=63), SHAPE),
            (dict(rot_dim=66), SHAPE), (dict(layout=2), UNSUPPORTED), (dict(amplitude=math.nan), SHAPE)]
BAD_ROWS = [(dict(T=-1), SHAPE), (dict(T=(1 << 30) + 1), SHAPE), (dict(positions=None), NULL), (dict(table=None), NULL),
            (dict(positions=A + 2), ALIGN), (dict(seq=A + 2), ALIGN), (dict(table=A + 2), ALIGN),
            (dict(num_seqs=0), SHAPE), (dict(max_pages=0), SHAPE), (dict(table_stride=4), SHAPE),
            (dict(table_stride=-1), SHAPE), (dict(seq=None), SHAPE)]   # no seq: 3 rows of 2 sequences
BAD_KV = [(dict(k_stride=124), SHAPE), (dict(v_stride=130), SHAPE), (dict(flags=2), UNSUPPORTED)]


def refusals(fn, good, bad):
    for change, want in bad:
        assert fn(*{**good, **change}.values(), None) == want, change


def test_rope_refusals(lib):
    f = lib.bitlinear_rope
    refusals(f, ROPE, [(dict(x=None), NULL), (dict(y=None), NULL), (dict(positions=None), NULL), (dict(rope=None), NULL),
                       (dict(x=U), ALIGN), (dict(y=U), ALIGN), (dict(positions=A + 1), ALIGN), (dict(T=-1), SHAPE),
                       (dict(H=0), SHAPE), (dict(H=4097), SHAPE), (dict(D=66), SHAPE), (dict(D=260), SHAPE),
                       (dict(x_stride=124), SHAPE), (dict(y_stride=129), SHAPE), (dict(y=A, y_stride=132), SHAPE),
                       (dict(flags=2), UNSUPPORTED)])
    refusals(f, ROPE, [(dict(rope=spec(**c)), w) for c, w in BAD_ROPE])
    assert f(*{**ROPE, "T": 0, "x": None, "y": None, "positions": None, "y_stride": 128}.values(), None) == 0


def test_append_refusals(lib):
    f = lib.bitlinear_kv_append
    refusals(f, APPEND, [(dict(cache=pages(**c)), w) for c, w in BAD_PAGES])
    refusals(f, APPEND, [(dict(rope=spec(**c)), w) for c, w in BAD_ROPE])
    refusals(f, APPEND, BAD_ROWS + BAD_KV)
    refusals(f, APPEND, [(dict(q=None), NULL), (dict(q_out=None), NULL), (dict(k=None), NULL), (dict(v=None), NULL),
                         (dict(q=U), ALIGN), (dict(k=U), ALIGN), (dict(Hq=-1), SHAPE), (dict(Hq=4097), SHAPE),
                         (dict(Hq=0), SHAPE), (dict(q_stride=252), SHAPE), (dict(q_stride=260), SHAPE),
                         (dict(cache=None), NULL)])
    assert f(*{**APPEND, "T": 0}.values(), None) == 0


def test_read_refusals(lib):
    f = lib.bitlinear_kv_read
    refusals(f, READ, [(dict(cache=pages(**c)), w) for c, w in BAD_PAGES])
    refusals(f, READ, BAD_ROWS + BAD_KV)
    refusals(f, READ, [(dict(k_out=None), NULL), (dict(v_out=None), NULL), (dict(k_out=U), ALIGN), (dict(cache=None), NULL)])
    assert f(*{**READ, "T": 0}.values(), None) == 0


def test_attention_refusals(lib):
    f = lib.bitlinear_attention
    refusals(f, ATTEND, [(dict(cache=pages(**c)), w) for c, w in BAD_PAGES])
    refusals(f, ATTEND, [(dict(q=None), NULL), (dict(out=None), NULL), (dict(table=None), NULL), (dict(lengths=None), NULL),
                         (dict(cache=None), NULL), (dict(q=U), ALIGN), (dict(out=U), ALIGN), (dict(lengths=A + 2), ALIGN),
                         (dict(B=-1), SHAPE), (dict(Hq=0), SHAPE), (dict(Hq=3), SHAPE), (dict(Hq=4098), SHAPE),
                         (dict(q_stride=252), SHAPE), (dict(out_stride=258), SHAPE), (dict(window=-1), SHAPE),
                         (dict(scale=math.inf), SHAPE), (dict(scale=math.nan), SHAPE), (dict(max_pages=0), SHAPE),
                         (dict(table_stride=3), SHAPE), (dict(flags=2), UNSUPPORTED)])
    assert f(*{**ATTEND, "B": 0}.values(), None) == 0
    need = bl.bitlinear_attention_workspace(3, 4, 2, 64)
    if need:
        assert f(*{**ATTEND, "workspace": A, "workspace_bytes": need - 1}.values(), None) == WORKSPACE
        assert f(*{**ATTEND, "workspace": U, "workspace_bytes": need}.values(), None) == ALIGN
    for bad in ((0, 4, 2, 64), (3, 3, 2, 64), (3, 4, 0, 64), (3, 4, 2, 60), (3, 4, 2, 512)):
        assert bl.bitlinear_attention_workspace(*bad) == 0


def test_frequencies_values(lib):
    for rot in (2, 20, 80, 128, 256):
        i = np.arange(0, rot, 2)
        theta = 10000.0 ** (-i / rot)
        # pow is within a step or two of fp64; a handful for the scalings' own roundings
        close = lambda got, want: np.testing.assert_allclose(got.numpy(), want, rtol=8 * 2.0 ** -52, atol=0)  # noqa: E731
        close(bl.bitlinear_rope_frequencies(rot), theta)
        close(bl.bitlinear_rope_frequencies(rot, 500.0), 500.0 ** (-i / rot))
        close(bl.bitlinear_rope_frequencies(rot, scaling=bl.ROPE_SCALE_LINEAR, factor=4.0), theta / 4)
        g = ((4096 * theta / (2 * math.pi) - 1) / 31).clip(0, 1)
        np.testing.assert_allclose(bl.bitlinear_rope_frequencies(rot, scaling=bl.ROPE_SCALE_PARTS, factor=16.0,
                                                                 original_length=4096.0).numpy(),
                                   theta * (g + (1 - g) / 16), rtol=1e-13)
        if rot > 2:
            by_base = bl.bitlinear_rope_frequencies(rot, scaling=bl.ROPE_SCALE_BASE, factor=8.0).numpy()
            assert by_base[0] == 1.0
            np.testing.assert_allclose(by_base[-1], theta[-1] / 8, rtol=1e-13)   # the slowest pair: exactly by factor


def test_frequencies_refusals(lib):
    f, out = lib.bitlinear_rope_frequencies, ctypes.addressof((ctypes.c_double * 128)())
    good = dict(rot=64, base=1e4, scaling=0, factor=2.0, length=4096.0, low=1.0, high=32.0, out=out)
    for change, want in [(dict(out=None), NULL), (dict(rot=1), SHAPE), (dict(rot=0), SHAPE), (dict(rot=63), SHAPE),
                         (dict(rot=258), SHAPE), (dict(base=0.0), SHAPE), (dict(base=math.inf), SHAPE),
                         (dict(scaling=4), UNSUPPORTED), (dict(scaling=-1), UNSUPPORTED),
                         (dict(scaling=1, factor=0.0), SHAPE), (dict(scaling=2, rot=2), SHAPE),
                         (dict(scaling=2, factor=math.nan), SHAPE), (dict(scaling=3, length=0.0), SHAPE),
                         (dict(scaling=3, high=1.0), SHAPE)]:
        assert f(*{**good, **change}.values()) == want, change


def test_binding_refuses_cpu_tensors():
    import torch
    x, p, f = torch.zeros(2, 3, 64), torch.zeros(2, dtype=torch.int32), torch.zeros(32, dtype=torch.float64)
    k = torch.zeros(4, 3, 16, 64, dtype=torch.bfloat16)
    with pytest.raises(TypeError):
        bl.bitlinear_rope(x, p, (f, 0), x)
    with pytest.raises(TypeError):
        bl.bitlinear_kv_append(x, x, (k, k), p, torch.zeros(2, 4, dtype=torch.int32))
    with pytest.raises(TypeError):
        bl.bitlinear_kv_read((k, k), p, torch.zeros(2, 4, dtype=torch.int32), x, x)
    with pytest.raises(TypeError):
        bl.bitlinear_attention(x, (k, k), torch.zeros(2, 4, dtype=torch.int32), p, x)
