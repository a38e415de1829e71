"""How the attention shares rows out over CTAs (csrc/shares.h, compiled here): every row has all of its steps,
and the CTAs of all rows fit the grid, up to the largest lengths that the call takes."""
import ctypes
import random
import subprocess

import pytest

from bitlinear_w1_a8_gb300 import build as blbuild

LEAST, TOKENS = 8, 16   # steps of a CTA at least; tokens of a short step


@pytest.fixture(scope="module")
def shares(tmp_path_factory):
    at = tmp_path_factory.mktemp("shares")
    (at / "shares.cpp").write_text('#include "shares.h"\n'
                                   'extern "C" int share(int total, int spare, int least) { return bitlinear::share_of_steps(total, spare, least); }\n'
                                   'extern "C" int fit(int64_t rows, int64_t steps) { return bitlinear::steps_fit(rows, steps); }\n')
    lib = str(at / "shares.so")
    # -fwrapv: an overflow would wrap, as it does on the GPU
    subprocess.run(["g++", "-O1", "-fwrapv", "-fPIC", "-shared", "-I", blbuild.CSRC, str(at / "shares.cpp"), "-o", lib], check=True)
    lib = ctypes.CDLL(lib)
    lib.fit.argtypes = [ctypes.c_int64, ctypes.c_int64]
    return lib


def check(shares, steps, rows_a_seq, ctas):
    """`steps` of each sequence, as find_part reads them."""
    rows, total = rows_a_seq * sum(n > 0 for n in steps), rows_a_seq * sum(steps)
    assert total <= 2 ** 31 - 1
    share = shares.share(total, ctas - rows, LEAST)
    assert share >= LEAST
    used = rows_a_seq * sum(-(-n // share) for n in steps)
    assert used <= ctas, (steps, rows_a_seq, ctas, share, used)


@pytest.mark.parametrize("ctas", [608, 456, 304])
@pytest.mark.parametrize("rows_a_seq", [1, 2, 16, 32, 101])
def test_the_longest_sequences_fit_the_grid(shares, ctas, rows_a_seq):
    """Sequences that share one page list: nothing but the table bounds their lengths."""
    for B in (1, 2, 3, 6, 12, 100):
        rows = B * rows_a_seq
        if rows > ctas // 3:
            continue
        most = (2 ** 31 - 1) // rows            # what the host lets through
        assert shares.fit(rows, most) and not shares.fit(rows, most + 1)
        longest = min(most, (2 ** 31 - 1 + TOKENS - 1) // TOKENS)  # what a length can be
        for short in (0, 1, 2, 599, 600, 1000):
            check(shares, [max(1, longest - short)] * B, rows_a_seq, ctas)
        check(shares, [longest] + [1] * (B - 1), rows_a_seq, ctas)


def test_any_lengths_fit_the_grid(shares):
    rng = random.Random(3)
    for _ in range(3000):
        ctas, B = rng.choice([608, 456, 304]), rng.randint(1, 200)
        rows_a_seq = rng.randint(1, max(1, ctas // 3 // B))
        if B * rows_a_seq > ctas // 3:
            continue
        top = int(2 ** rng.uniform(0, 26)) // (B * rows_a_seq) + 1
        check(shares, [rng.choice([0, 1, rng.randint(0, top), top]) for _ in range(B)], rows_a_seq, ctas)
