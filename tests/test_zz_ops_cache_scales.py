"""Attention over pages whose value scales lie anywhere in fp32's range, against 64 bits.

The bound, with U = 2^-24, w a token's weight, s its page's value scale, b its byte's value:

  weights    fp16 holds w s to 2^-11 of itself, or to 2^-32 of M = max w s over the tokens that the
             row sees: the errors of a row's element sum to 2^-11 sum w |v| + 2^-32 M sum |b|.
  exponents  the logarithms of two scales (up to 149 each) and the reference they are taken from
             are each within 2^-16, six roundings of that size at most: relative 6 2^-16 log 2 < 2^-13,
             and the factor that brings the sums back to their scale is two more of them.
  scores     as in test_zz_ops_cache: E each, relative 2 E, and n U for the sums.
  out        one rounding to bf16, half a step: 2^-8 relative, or half of bf16's least, 2^-134."""
from __future__ import annotations

import itertools
import math

import pytest
import torch

import split_bf16_gemm_amd as sbg
from test_zz_ops_cache import BF16, F64, FP8, PAGE, U, gen, gpu, ints, logical, random_cache, randn


def reference(q, cache, table, lens, starts, scale, window=0):
    lk, lv = logical(cache)
    T, Hq, D = q.shape
    H = lk.shape[2]
    out, lse = torch.zeros(T, Hq, D, dtype=F64), torch.full((T, Hq), -math.inf, dtype=F64)
    err, lerr = torch.zeros_like(out), torch.zeros_like(lse)
    q = q.double().cpu()
    vs = cache.v_scale.double().cpu()
    for b, end in enumerate(lens):
        ids = torch.tensor(table[b])
        K, V = lk[ids].reshape(-1, H, D), lv[ids].reshape(-1, H, D)
        S = vs[ids].repeat_interleave(PAGE, 0)
        at = torch.arange(len(K))
        for j in range(starts[b + 1] - starts[b]):
            t, pos = starts[b] + j, end - (starts[b + 1] - starts[b]) + j
            sees = (at <= pos) & ((at > pos - window) if window else (at >= 0))
            if not sees.any():
                continue
            for h in range(Hq):
                k, v, s = (x[sees][:, h // (Hq // H)] for x in (K, V, S))
                x = scale * (k @ q[t, h])
                lse[t, h] = torch.logsumexp(x, 0)
                w = torch.exp(x - lse[t, h])
                out[t, h] = w @ v
                E = abs(scale) * (D + 3) * U * (k.abs() @ q[t, h].abs())
                E = E + 4 * U * (x.max() - x) + 4 * U * x.abs()
                n = (64 + len(ids) * 4 + 16) * U
                off = 2 * E + w @ E + 2.0 ** -11 + 2.0 ** -13 + 2.0 ** -14 + n
                bytes_ = torch.where(s[:, None] > 0, v / s[:, None], 0).abs().sum(0)
                err[t, h] = (w * off) @ v.abs() + 2.0 ** -32 * (w * s).max() * bytes_
                lerr[t, h] = E.max() + n + 8 * U * (1 + lse[t, h].abs()) + 2.0 ** -15
    return out, lse, err, lerr


def check(q, cache, table, lens, starts, scale=None, window=0):
    T, Hq, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    ws = sbg.make_cache_attention_workspace(T, Hq, cache.k.shape[1], D)
    out, lse = sbg.cache_attention(q, cache, ints(table), ints(lens), row_starts=ints(starts),
                                   scale=scale, window=window, workspace=ws,
                                   lse_out=torch.empty(T, Hq, device="cuda"))
    ref, rl, err, lerr = reference(q, cache, table, lens, starts, scale, window)
    got = out.double().cpu()
    assert torch.isfinite(got).all()
    bound = err + (ref.abs() + err) * 2.0 ** -8 + 2.0 ** -134
    assert bool(((got - ref).abs() <= bound).all()), ((got - ref).abs() / bound).max().item()
    some = torch.isfinite(rl)
    assert bool(((lse.double().cpu() - rl).abs() <= lerr)[some].all())


# v_scale of a sequence's pages, one after another
SCALES = [
    (1e2, 1e-37), (1e-37, 1e2), (10.0, 1e-37), (1e-20, 1e18), (1e20, 1e-20), (1e-20, 1e20),
    (2e-38, 10.0), (5.0, 1.2e-38), (1e-12, 1.0, 1e-12), (1.0, 1e-12, 1e13, 1e-25, 1.0),
    (1e-40, 1e-39, 1e-41), (1e-40, 1e30), (1e33, 1e-40), (0.0, 1e-37, 1e2), (1e2, 0.0, 1e-37),
    (1e-37, 0.0, 0.0, 1e2, 1e-37, 0.0), (0.0, 0.0, 1e-39), (3e33, 1e33), (1e33, 1e-37, 2e33),
]
# rows of a key head and of a sequence, by the kernel that they take
KINDS = [(1, 1), (5, 4), (4, 15), (10, 30)]


@gpu
@pytest.mark.parametrize("G,n", KINDS, ids=lambda x: str(x))
@pytest.mark.parametrize("kind", [torch.int8, FP8])
def test_values_of_any_size(kind, G, n):
    """Values up to bf16's largest: their sums are larger than fp32 holds.  Short sequences, and
    such whose parts are joined."""
    g = gen(60, G)
    H, D, P = 1, 64, 150
    cache = random_cache(g, P, H, D, kind)
    q = randn(g, n, H * G, D, std=3.0)
    top = 127 if kind == torch.int8 else 448
    for value in (3.3e38, 1e37, 1e32, 1e25):
        cache.v_scale.copy_(value / top * torch.exp(-0.5 * torch.rand(P, 1, generator=g)))
        for pages in (2, 9, P):
            check(q, cache, [list(range(pages))], [pages * PAGE - 5], [0, n])


@gpu
@pytest.mark.parametrize("G,n", KINDS, ids=lambda x: str(x))
@pytest.mark.parametrize("scales", SCALES, ids=lambda s: "_".join(f"{x:g}" for x in s))
def test_scales_far_apart(scales, G, n):
    """The pages' scales in a run of each wavefront (every fourth page is one wavefront's, or
    every page), for tokens of all weights."""
    g = gen(61, scales, G)
    H, D = 1, 64
    # the pattern, for each wavefront and for all of them
    order = [s for s in scales for _ in range(4)] + list(scales)
    P = len(order)
    cache = random_cache(g, P, H, D, FP8 if G == 5 else torch.int8)
    cache.v_scale.copy_(torch.tensor(order)[:, None])
    top = 448 if G == 5 else 127
    assert max(order) * top < 3.3e38
    q = randn(g, n, H * G, D, std=3.0)
    check(q, cache, [list(range(P))], [P * PAGE - 5], [0, n])


@gpu
@pytest.mark.parametrize("G,n", KINDS, ids=lambda x: str(x))
@pytest.mark.parametrize("scales", [(1e2, 1e-37), (1e-37, 1e2), (1e20, 1e-20), (1e-39, 1e33)],
                         ids=lambda s: "_".join(f"{x:g}" for x in s))
def test_scales_far_apart_across_joined_runs(scales, G, n):
    """Runs of one scale each, and a run in which it changes, joined."""
    g = gen(62, scales, G)
    H, D, P = 2, 32, 200
    cache = random_cache(g, P, H, D)
    cache.v_scale.copy_(torch.tensor([scales[p >= 101] for p in range(P)])[:, None])
    q = randn(g, 2 * n, H * G, D, std=2.0)
    table = [list(range(P)), list(range(150, P)) + list(range(150))]
    check(q, cache, table, [P * PAGE - 9, 45 * PAGE], [0, n, 2 * n])


@gpu
@pytest.mark.parametrize("G,n", KINDS, ids=lambda x: str(x))
def test_what_small_scales_have_left(G, n):
    """What is left of an output where the page of the largest scale is not seen through a window, has
    next to no weight, or has bytes of 0."""
    g = gen(63, G)
    H, D, P = 1, 64, 9
    cache = random_cache(g, P, H, D)
    q = randn(g, n, G, D)
    table = [list(range(P))]
    cache.v_scale.copy_(torch.tensor([1e10, 1e3, 1.0, 1.0, 1e-30, 1e-12, 1.0, 1e-20, 1e-35])[:, None])
    check(q, cache, table, [P * PAGE], [0, n], window=70)
    check(q, cache, table, [P * PAGE], [0, n], window=180)
    # scores that leave the first pages 2^-100 of the others' weight, and less
    cache.k_scale.copy_(torch.tensor([0.02] * 5 + [1e-6] * 4)[:, None])
    k = cache.k.view(torch.int8)
    k[:5] = 100
    check(-(q.abs() + 0.2), cache, table, [P * PAGE], [0, n])
    check(-(q.abs() + 2).clamp(max=4), cache, table, [P * PAGE], [0, n])
    for p in range(5):
        cache.v.view(torch.int8)[p, :, :, ::2] = 0
    check(q * 0.01, cache, table, [P * PAGE], [0, n])


@gpu
def test_every_pair_of_scales():
    """One token a page, every order of two magnitudes out of the whole range."""
    g = gen(64)
    values = [0.0, 1e-44, 1e-39, 1.2e-38, 1e-30, 1e-20, 1e-12, 1.0, 1e12, 1e20, 1e30, 2e36]
    pairs = list(itertools.product(values, repeat=2))
    H, D, B = 1, 16, len(pairs)
    cache = random_cache(g, 2 * B, H, D)
    cache.v_scale.copy_(torch.tensor(pairs).reshape(-1, 1))
    q = randn(g, B, 2, D, std=2.0)
    table = [[2 * b, 2 * b + 1] for b in range(B)]
    check(q, cache, table, [PAGE + 1] * B, list(range(B + 1)))
    # both by one wavefront
    table = [[2 * b] * 4 + [2 * b + 1] for b in range(B)]
    check(q, cache, table, [4 * PAGE + 1] * B, list(range(B + 1)))
