"""Pages that a row of fork_pages lacks, over several steps: every step says so."""
from __future__ import annotations

import pytest
import torch

import split_bf16_gemm_amd as sbg
from test_zz_ops_cache import I32, PAGE, by_token, check_attention, gen, gpu, ints, random_cache, \
    randn


def forked(cache, table, lens, parents=None, reserve=1, **kw):
    R, W = table.shape
    return sbg.fork_pages(cache, table, lens, parents, reserve=reserve,
                          workspace=sbg.make_pages_workspace(R, W, cache.k.shape[0]), **kw)


@gpu
@pytest.mark.parametrize("large", [False, True])
def test_a_pool_that_runs_out(large):
    """Two rows, three pages, and later four: the row that gets none is counted until its lost page
    is full, although there are free pages again, and sees no tokens of it; then it goes on.  (The
    large pool, most of it held, takes the path of several launches.)"""
    g = gen(71, large)
    P, W, H, D = (5000 if large else 4), 4, 1, 32
    cache = random_cache(g, P, H, D)
    held = torch.ones(P, dtype=I32, device="cuda")
    held[:3] = 0
    table = torch.full((2, W), -1, dtype=I32, device="cuda")
    table[0, 0], table[1, 0] = 0, 1
    lens, other = ints([PAGE, PAGE]), None
    for step in range(PAGE):
        if step == 10:
            held[3] = 0      # a page is given back
        table, lens, refs, missing = forked(cache, table, lens, held=held)
        assert missing.item() == 1
        assert table.tolist() == [[0, 2, -1, -1], [1, -1, -1, -1]]
        if other is None:
            other = [x[3:].clone() for x in cache]
        lens = lens + 1
        k = randn(g, 2, H, D)
        before = [x[1].clone() for x in cache]
        sbg.cache_append(k, k, cache, table, lens)
        assert all(torch.equal(x[1], y) for x, y in zip(cache, before))
    # what the row sees: its first page alone
    q = randn(g, 2, 2, D)
    check_attention(q, cache, table, lens.tolist(), [0, 1, 2], rs=None)
    # the lost page is full: a new one is reserved, and taken from the lowest (row 0 goes first)
    held[4:6] = 0
    table, lens, refs, missing = forked(cache, table, lens, held=held)
    want = [[0, 2, 3, -1], [1, -1, 4, -1]] if large else [[0, 2, 3, -1], [1, -1, -1, -1]]
    assert table.tolist() == want and missing.item() == (0 if large else 1)
    assert all(torch.equal(x[3:], y) for x, y in zip(cache, other))


@gpu
def test_a_copy_that_could_not_be_made():
    """Two rows from one with an unfinished page and no free page: the second is counted at each
    step, alone, and its parent's page stays as it is."""
    g = gen(72)
    cache = random_cache(g, 1, 1, 16)
    table, lens, refs, missing = forked(cache, ints([[0], [-1]]), ints([10, 0]), ints([0, 0]))
    for step in range(3):
        assert table.tolist() == [[0], [-1]] and missing.item() == 1 and refs.tolist() == [1]
        lens = lens + 1
        kb, vb = (x.clone() for x in by_token(cache))
        sbg.cache_append(*[randn(g, 2, 1, 16, std=0.01)] * 2, cache, table, lens)
        for x, y in zip(by_token(cache), (kb, vb)):
            keep = [t for t in range(PAGE) if t != 10 + step]
            assert torch.equal(x[0, keep], y[0, keep])
        table, lens, refs, missing = forked(cache, table, lens)
    # its end is no lack
    table, lens, refs, missing = forked(cache, table, lens, ints([0, -1]))
    assert lens.tolist() == [13, 0] and missing.item() == 0


@gpu
def test_a_row_that_ends_and_begins_anew():
    g = gen(73)
    cache = random_cache(g, 4, 1, 16)
    table, lens, refs, missing = forked(cache, ints([[0, 1], [2, -1]]), ints([70, 5]),
                                        ints([0, -1]))
    assert table.tolist() == [[0, 1], [-1, -1]] and lens.tolist() == [70, 0]
    assert refs.tolist() == [1, 1, 0, 0] and missing.item() == 0
    # with a length of 0 it gets its first page
    again = forked(cache, table, lens)
    assert again[0].tolist() == [[0, 1], [2, -1]] and again[3].item() == 0
    # counted one further than it was, its token has no page, and every call says so
    lens = lens + 1
    for _ in range(2):
        table, lens, refs, missing = forked(cache, table, lens)
        assert lens.tolist() == [71, 1] and table[1].tolist() == [-1, -1]
        assert missing.item() == 1
    # entries of an unfinished last page that are no page at all
    table = ints([[0, 1], [99, -1]])
    assert forked(cache, table, lens)[3].item() == 1
