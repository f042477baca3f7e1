"""Every form of cache_attention's kernels: each class of head sizes, whole blocks of 64 or not, rows of
a key head, and type of the cache, against the 64-bit formula and bounds of test_zz_ops_cache."""
from __future__ import annotations

import itertools

import pytest
import torch

from test_zz_ops_cache import FP8, check_attention, gen, gpu, random_cache, randn, tables

SIZES = [48, 64, 112, 128, 176, 192, 208, 256]     # of each block of 64, partly there and whole
# rows of a key head, on average, up to which a kernel serves; new rows of a long sequence and a
# short one with five query heads to a key head
ROWS = {16: (4, 1), 32: (7, 4), 64: (14, 10), None: (29, 3)}


def kind_of(T, G, B):
    return next((k for k in (16, 32, 64) if T * G <= k * B), None)


def test_the_rows_are_of_each_kind():
    for kind, new in ROWS.items():
        assert kind_of(sum(new), 5, 2) == kind
    assert {(d + 63) // 64 for d in SIZES} == {1, 2, 3, 4}
    assert all({d % 64 == 0 for d in SIZES if (d + 63) // 64 == c} == {True, False}
               for c in (1, 2, 3, 4))


@gpu
@pytest.mark.parametrize("kind", [torch.int8, FP8], ids=["int8", "e4m3"])
@pytest.mark.parametrize("rows", ROWS, ids=lambda r: f"rows{r}")
@pytest.mark.parametrize("D", SIZES)
def test_form(D, rows, kind):
    """Lengths that are no multiple of 64, one of enough pages that its tiles are joined from
    several parts (whatever the rows, parts have 16 pages at most here); with a window too."""
    new = ROWS[rows]
    lens = [1537, 75]
    g = gen(81, D, rows)
    P = 30
    cache = random_cache(g, P, 1, D, kind)
    starts = [0, *itertools.accumulate(new)]
    q = randn(g, sum(new), 5, D, std=1.5)
    table = tables(g, P, lens)
    check_attention(q, cache, table, lens, starts)
    check_attention(q, cache, table, lens, starts, window=1100)
