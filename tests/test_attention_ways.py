"""The rules by which attention of rows that share a prefix chooses its way and its CTAs (csrc/shares.h, compiled here)."""
import random

import pytest

from serving_ways import SMS, rules, way, wide_tiles


@pytest.mark.parametrize("fmt,groups,R,Hq,Hkv,D,tokens,want", [
    ("int8", 1, 2, 16, 16, 128, 38, "alone"), ("int8", 8, 5, 32, 32, 80, 2048, "eight"), ("int8", 1, 64, 32, 32, 80, 2300, "eight"),
    ("bf16", 1, 64, 32, 8, 128, 16484, "wide"), ("int8", 1, 64, 32, 8, 128, 16484, "wide"), ("fp8", 1, 64, 32, 8, 256, 16484, "eight"),
    ("bf16", 4, 1, 32, 8, 128, 16484, "alone")])
def test_the_way_of_a_served_batch(fmt, groups, R, Hq, Hkv, D, tokens, want):
    page = 64
    assert way(fmt, groups, R, Hq, Hkv, D, -(-tokens // page), page) == want


def test_a_document_gives_a_cta_many_tiles():
    assert wide_tiles(1, 64, 32, 8, [16384], 258, 64) == [15]


@pytest.mark.parametrize("sms", [152, 148, 16])
def test_parts_have_their_places(sms):
    """As many CTAs as the workspace has places for: one a row, or as many as there are SMs."""
    for groups in (1, 2, 5, 60, 1025):
        for a_group in (1, 3, 8, 16, 40, 96, 200):
            for steps in (1, 2, 7, 129, 1 << 20, 1 << 30):
                rows = groups * a_group
                splits = rules().splits(groups, rows, steps, sms)
                if splits == 0:
                    assert groups > 1 and rows < sms and rows * steps < 1 << 31
                else:
                    assert rows * splits <= max(rows, sms) <= max(rows, SMS)


def test_summaries_are_shared_out_up_to_the_largest_sizes():
    """Equal rounds of resident CTAs; sizes whose product passes 64 bits (one page list for all rows) as well."""
    rng = random.Random(1)
    sizes = [(1 << 30, 1 << 34), (1 << 30, 1 << 42), (1 << 30, 1), (1, 1 << 42), (1, 1), (1 << 30, 1215), (1 << 30, 1216)]
    sizes += [(int(2 ** rng.uniform(0, 30)), int(2 ** rng.uniform(0, 42))) for _ in range(2000)]
    for pages, heads in sizes:
        for resident in (1216, 1184, 128):
            rounds = -(-pages * heads // resident)
            assert rules().pages(pages, heads, resident) == -(-pages // rounds), (pages, heads, resident)
