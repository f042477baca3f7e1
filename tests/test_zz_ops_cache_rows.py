"""Bounds of the paged cache's rows that reach past the call's rows: those that are there stand where
the bounds, as they are given, put them (position of row r: lens[b] - row_starts[b + 1] + r).

The references are the operators themselves with bounds that end at the last row and lengths less by
the rows that are not there, which put every row at the same position, and for the attention the
64-bit formula with its derived bounds."""
from __future__ import annotations

import pytest
import torch

import split_bf16_gemm_amd as sbg
from test_zz_ops_cache import (BF16, FP8, HALF, attention_reference, gen, gpu, ints, logical,
                               random_cache, randn)

# lens, row_starts, T
BOUNDS = [
    ([100], [0, 4], 2), ([100], [-3, 40], 5), ([70, 130], [0, 3, 90], 50),
    ([300, 200, 64], [0, 70, 200, 300], 100), ([2, 5], [0, 4, 9], 6), ([1, 40], [0, 1, 1 << 30], 3),
    ([64, 10, 7], [0, 5, 5, 9], 5), ([(1 << 31) - 1], [0, (1 << 31) - 1], 3),
]
ids = lambda c: f"t{c[2]}_{c[1][-1]}"  # noqa: E731


def as_if_cut(lens, starts, T):
    """The same rows' lengths and bounds, those past T gone."""
    cut = [n - max(0, hi - T) for n, hi in zip(lens, starts[1:])]
    return [max(0, n) for n in cut], [min(max(x, 0), T) for x in starts]


def setting(case, H, D, kind=torch.int8):
    lens, starts, T = case
    g = gen(51, *starts, T)
    cache = random_cache(g, 5 * len(lens), H, D, kind)
    table = torch.randperm(5 * len(lens), generator=g).view(len(lens), 5).int().cuda()
    return g, cache, table


@gpu
@pytest.mark.parametrize("case", BOUNDS, ids=ids)
def test_append_and_read_of_rows_past_the_last(case):
    lens, starts, T = case
    H, D = 2, 32
    g, cache, table = setting(case, H, D)
    other = type(cache)(*(x.clone() for x in cache))
    k, v = randn(g, T, H, D), randn(g, T, H, D)
    cut_lens, cut_starts = as_if_cut(*case)
    sbg.cache_append(k, v, cache, table, ints(lens), row_starts=ints(starts))
    sbg.cache_append(k, v, other, table, ints(cut_lens), row_starts=ints(cut_starts))
    assert all(torch.equal(x, y) for x, y in zip(cache, other))
    outs = [torch.full((T, H, D), 9.0, dtype=BF16, device="cuda") for _ in "kv"]
    sbg.cache_read(cache, table, ints(lens), row_starts=ints(starts), k_out=outs[0], v_out=outs[1])
    for got, full in zip(outs, logical(cache)):
        want = torch.full((T, H, D), 9.0, dtype=BF16)
        for b, n in enumerate(lens):
            for r in range(max(0, starts[b]), min(T, starts[b + 1])):
                pos = n - starts[b + 1] + r
                if 0 <= pos < 5 * 64:
                    want[r] = full[int(table[b, pos // 64]), pos % 64].float().to(BF16)
        assert torch.equal(got.cpu(), want)


@gpu
@pytest.mark.parametrize("G", [1, 6, 24])
@pytest.mark.parametrize("case", BOUNDS[:-1], ids=ids)
def test_attention_of_rows_past_the_last(case, G):
    lens, starts, T = case
    H, D = 2, 64
    g, cache, table = setting(case, H, D, FP8)
    q = randn(g, T, H * G, D)
    cut_lens, cut_starts = as_if_cut(*case)
    for window in (0, 20):
        out = torch.full((T, H * G, D), 7.0, dtype=BF16, device="cuda")
        lse = torch.full((T, H * G), 7.0, device="cuda")
        sbg.cache_attention(q, cache, table, ints(lens), row_starts=ints(starts), window=window,
                            workspace=sbg.make_cache_attention_workspace(T, H * G, H, D), out=out,
                            lse_out=lse)
        ref, rl, err, lerr = attention_reference(q, cache, table, cut_lens, cut_starts, D ** -0.5,
                                                 window)
        got, gl = out.double().cpu(), lse.double().cpu()
        none, empty = torch.isnan(rl), torch.isneginf(rl)
        some = ~none & ~empty
        assert (got[none] == 7).all() and (gl[none] == 7).all()
        assert (got[empty] == 0).all() and torch.isneginf(gl[empty]).all()
        bound = err + (ref.abs() + err) * HALF[BF16]
        assert bool(((got - ref).abs() <= bound)[some].all())
        assert bool(((gl - rl).abs() <= lerr)[some].all())


def test_read_with_bounds_needs_the_number_of_rows():
    """How many rows row_starts counts is on the GPU: one row a sequence would be a guess, and a
    silent one, as rows past the last are left out.  (Refused before any tensor is looked at.)"""
    c = sbg.make_kv_cache(4, 1, 16, device="cpu")
    table, lens, starts = ints([[0], [1]], "cpu"), ints([9, 9], "cpu"), ints([0, 3, 7], "cpu")
    with pytest.raises(ValueError, match="rows"):
        sbg.cache_read(c, table, lens, row_starts=starts)
    out = torch.empty(7, 1, 16, dtype=BF16)
    for given in (dict(rows=7), dict(k_out=out), dict(v_out=out)):
        with pytest.raises(ValueError, match="GPU"):
            sbg.cache_read(c, table, lens, row_starts=starts, **given)
