"""Which way bitlinear_attention_shared takes for given sizes, by the library's own rules (csrc/shares.h, compiled here)."""
import ctypes
import functools
import os
import subprocess
import tempfile

from bitlinear_w1_a8_gb300 import build as blbuild

SMS = 152
SOURCE = '''#include "shares.h"
using namespace bitlinear;
extern "C" {
int alone(int64_t B, int64_t tokens, int kv_heads, int head_dim, int code, int heads) { return faster_alone(B, tokens, kv_heads, head_dim, code, heads); }
int wide(int64_t heads, int64_t tokens, int head_dim, int code) { return wide_wins(heads, tokens, head_dim, code); }
int splits(int64_t groups, int64_t rows, int64_t steps, int sms) { return wide_splits(groups, rows, steps, sms); }
int share(int total, int spare, int least) { return share_of_steps(total, spare, least); }
int64_t pages(int64_t max_pages, int64_t heads, int64_t resident) { return page_shares(max_pages, heads, resident); }
int q_heads() { return kPrefixWide; }
int tile() { return kPrefixTile; }
}
'''


@functools.cache
def rules():
    with tempfile.TemporaryDirectory() as at:
        src, lib = os.path.join(at, "ways.cpp"), os.path.join(at, "ways.so")
        with open(src, "w") as f:
            f.write(SOURCE)
        subprocess.run(["g++", "-O1", "-fwrapv", "-fPIC", "-shared", "-I", blbuild.CSRC, src, "-o", lib], check=True)
        lib = ctypes.CDLL(lib)
    i64, i = ctypes.c_int64, ctypes.c_int
    lib.alone.argtypes, lib.wide.argtypes, lib.splits.argtypes = [i64, i64, i, i, i, i], [i64, i64, i, i], [i64, i64, i64, i]
    lib.pages.argtypes, lib.pages.restype = [i64, i64, i64], i64
    return lib


def way(fmt, groups, R, Hq, Hkv, D, columns, page, sms=SMS):
    """"alone" (row by row), "eight" (q heads a CTA) or "wide" (the tensor cores) for a table of `columns`."""
    code, tokens, G = 2 if fmt == "bf16" else 1, columns * page, Hq // Hkv
    if R == 1 or rules().alone(groups * R, tokens, Hkv, D, code, G):
        return "alone"
    return "wide" if rules().wide(R * G, tokens, D, code) else "eight"


def wide_tiles(groups, R, Hq, Hkv, shared, columns, page, sms=SMS):
    """The most tiles that a CTA has of each group, on the tensor cores."""
    up = lambda a, b: -(-a // b)  # noqa: E731
    lib, tile = rules(), rules().tile()
    a_group = Hkv * up(R * Hq // Hkv, lib.q_heads())
    steps = [up(max(0, min(int(s), columns * page)), tile) for s in shared]
    splits = lib.splits(groups, groups * a_group, up(columns * page, tile), sms)
    if splits:
        return [up(n, splits) for n in steps]
    share = lib.share(a_group * sum(steps), sms - a_group * sum(n > 0 for n in steps), 1)
    return [n and up(n, up(n, share)) for n in steps]
