"""What no row of a call sees may hold anything: NaNs of e4m3 before a window, as behind a sequence."""
from __future__ import annotations

import math

import pytest
import torch

import split_bf16_gemm_amd as sbg
from test_zz_ops_cache import FP8, PAGE, check_attention, gen, gpu, ints, random_cache, randn


@gpu
@pytest.mark.parametrize("G,n", [(1, 1), (8, 1), (8, 3), (4, 14), (8, 20)])
@pytest.mark.parametrize("D", [64, 112, 192, 256])
@pytest.mark.parametrize("kind", [torch.int8, FP8], ids=["int8", "e4m3"])
def test_tokens_before_every_rows_window(kind, D, G, n):
    g = gen(91, D, G, n)
    P, window = 12, 200
    cache = random_cache(g, P, 1, D, kind)
    q = randn(g, n, G, D)
    ws = sbg.make_cache_attention_workspace(n, G, 1, D)
    table = ints([list(range(P))])

    def run(cache, end):
        return sbg.cache_attention(q, cache, table, ints([end]), row_starts=ints([0, n]),
                                   window=window, workspace=ws,
                                   lse_out=torch.empty(n, G, device="cuda"))

    for end in (700, 641, 640, 201 + n):
        check_attention(q, cache, table, [end], [0, n], window=window)
        want, lse = run(cache, end)
        poisoned = type(cache)(*(x.clone() for x in cache))
        k, v = poisoned.k.view(torch.int8), poisoned.v.view(torch.int8)
        first = end - n - window + 1       # the first token that the call's first row sees
        for t in [*range(first), *range(end, P * PAGE)]:
            k[t // PAGE, :, :, t % PAGE] = 0x7f
            v[t // PAGE, :, t % PAGE // 16, :, t % 16] = -1
        for p in range(P):      # pages of such tokens alone: their scales too
            if (p + 1) * PAGE <= first or p * PAGE >= end:
                poisoned.k_scale[p], poisoned.v_scale[p] = math.nan, math.inf
        got, lse2 = run(poisoned, end)
        assert torch.equal(got, want) and torch.equal(lse2, lse)
