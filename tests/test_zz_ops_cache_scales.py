"""Attention over values that lie anywhere in fp32's range, against 64 bits.

The bound, with U = 2^-24, w a token's weight, s its page's value scale, b its byte's value:

  weights    fp16 holds w s to 2^-11 of itself, or to 2^-32 of M = max w s over the tokens that the
             row sees: the errors of a row's element sum to 2^-11 sum w |v| + 2^-32 M sum |b|.
  scores     as in test_zz_ops_cache: E each, relative 2 E, and n U for the sums.
  out        one rounding to bf16, half a step: 2^-8 relative, or half of bf16's least, 2^-134."""
from __future__ import annotations

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
                off = 2 * E + w @ E + 2.0 ** -11 + n
                bytes_ = torch.where(s[:, None] > 0, v / s[:, None], 0).abs().sum(0)
                err[t, h] = (w * off) @ v.abs() + 2.0 ** -32 * (w * s).max() * bytes_
                lerr[t, h] = E.max() + n + 8 * U * (1 + lse[t, h].abs())
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
