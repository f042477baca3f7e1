"""token_logprobs against its formulas in 64 bits.

Tolerances, with u = 2^-24 and d = l - m: e^d carries the rounding of d and of
its scaling and the exponential's own, (3|d| + 2) u; a sum adds at most 16
terms a chunk of 4096, a rescaling a chunk (4 u) and under 64 more; log p adds
the roundings of two subtractions and a logarithm.
"""
from __future__ import annotations

import ctypes

import pytest
import torch

import split_bf16_gemm_amd as sbg
from split_bf16_gemm_amd import ops

U = 2.0 ** -24
BF16, F32 = torch.bfloat16, torch.float32
INF, NAN = float("inf"), float("nan")


def reference(x, tok, n):
    """fp64 logprob, entropy, rank, alternatives, and the bounds of both sums."""
    M, V = x.shape
    x = x.double()
    m = x.amax(1, keepdim=True)
    d = x - m
    e = torch.exp(d)
    S = e.sum(1, keepdim=True)
    held = torch.where(e > 0, d, 0)
    lp = d - torch.log(S)
    H = (torch.log(S) - (e * held).sum(1, keepdim=True) / S)[:, 0]
    mine = lp.gather(1, tok[:, None])[:, 0]
    rank = (x > x.gather(1, tok[:, None])).sum(1)
    val, ids = torch.sort(x, dim=1, descending=True, stable=True)
    val, ids = val[:, :n], ids[:, :n]
    if ids.shape[1] < n:
        pad = n - ids.shape[1]
        val = torch.cat([val, torch.full((M, pad), -INF, dtype=val.dtype)], 1)
        ids = torch.cat([ids, torch.full((M, pad), -1)], 1)
    ids = torch.where(val == -INF, -1, ids)
    top = val - m - torch.log(S)
    p = e / S
    mean_d = (p * held.abs()).sum(1, keepdim=True)
    mean_d2 = (p * held ** 2).sum(1, keepdim=True)
    steps = V / 4096 * 20 + 120
    s_err = U * (3 * mean_d + steps)
    lp_err = s_err + 4 * U * (torch.log(S) + 1)
    H_err = (s_err * (1 + mean_d) + U * (3 * mean_d2 + steps * mean_d)
             + 4 * U * (torch.log(S) + mean_d + 1))[:, 0]
    return mine, H, rank, top, ids, lp_err, H_err


def judge(x, tok, n, got):
    mine, H, rank, top, ids, lp_err, H_err = reference(x, tok, n)
    lp, ent, rk, tl, ti = (t.cpu() for t in got)
    assert torch.equal(rk.long(), rank) and torch.equal(ti.long(), ids)
    assert lp.dtype == ent.dtype == tl.dtype == F32

    def near(a, b, err):
        a = a.double()
        fin = b.isfinite()
        assert torch.equal(a[~fin], b[~fin])
        bound = (err + 3 * U * torch.where(fin, b, 0).abs())[fin]
        assert ((a - b)[fin].abs() <= bound).all(), ((a - b)[fin].abs() / bound).max()

    near(lp, mine, lp_err[:, 0])
    near(ent, H, H_err)
    near(tl, top, lp_err.expand_as(top))


def run(x, tok, n):
    """One call with a workspace of its own, which has to be zero again after it."""
    ws = sbg.make_token_logprobs_workspace(x.shape[0], x.shape[1], n)
    got = sbg.token_logprobs(x, tok, n, workspace=ws)
    torch.cuda.synchronize()
    assert ws is None or ws.count_nonzero() == 0
    return got


def logits(g, M, V, dtype, std=3.0):
    return (torch.randn(M, V, generator=g) * std).to(dtype)


@pytest.mark.gpu
@pytest.mark.parametrize("M,V", [(1, 1), (1, 7), (3, 300), (1, 4097), (2, 49152), (1, 131072),
                                 (5, 50001), (64, 8193), (300, 5000), (600, 9000), (1030, 1000)])
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("n", [0, 1, 20, 32])
def test_token_logprobs(M, V, dtype, n):
    g = torch.Generator().manual_seed(M * 7919 + V + n)
    x = logits(g, M, V, dtype)
    tok = torch.randint(0, V, (M,), generator=g)
    if V > 40:
        x[:, torch.randperm(V, generator=g)[:V // 7]] = -INF
    ttype = torch.int32 if n == 1 else torch.int64
    got = run(x.cuda(), tok.to(ttype).cuda(), n)
    torch.cuda.synchronize()
    judge(x, tok, n, got)


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", [BF16, F32])
@pytest.mark.parametrize("start", [0, 1, 2, 5])
@pytest.mark.parametrize("M", [2, 1100])
def test_strided_rows_of_any_alignment(dtype, start, M):
    g = torch.Generator().manual_seed(start)
    V, ld = 4111, 4123
    wide = torch.full((M, ld), INF, dtype=dtype)     # what lies beside a row would show
    wide[:, start:start + V] = logits(g, M, V, dtype)
    x = wide[:, start:start + V]
    tok = torch.randint(0, V, (M,), generator=g)
    got = run(wide.cuda()[:, start:start + V], tok.cuda(), 6)
    torch.cuda.synchronize()
    judge(x, tok, 6, got)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 3, 1200])
@pytest.mark.parametrize("n", [5, 32])
@pytest.mark.parametrize("kind", ["equal", "rising", "falling", "few_left", "one_left", "zeros",
                                  "two_values", "far", "lowest"])
def test_rows_that_fill_the_candidates(M, n, kind):
    V = 9001
    g = torch.Generator().manual_seed(n)
    if kind == "equal":
        x = torch.full((M, V), 2.5)
    elif kind == "rising":
        x = torch.arange(V).float().repeat(M, 1) / 64
    elif kind == "falling":
        x = -torch.arange(V).float().repeat(M, 1) / 64
    elif kind in ("few_left", "one_left"):
        x = torch.full((M, V), -INF)
        for i in range(M):
            keep = torch.randperm(V, generator=g)[:1 if kind == "one_left" else 17]
            x[i, keep] = torch.randn(len(keep), generator=g)
    elif kind == "zeros":
        x = torch.zeros(M, V)
        x[:, ::2] = -0.0
    elif kind == "two_values":
        x = torch.randint(0, 2, (M, V), generator=g).float()
    elif kind == "far":
        x = logits(g, M, V, F32) + 30000
    else:
        x = torch.full((M, V), torch.finfo(F32).min)
        x[:, 1234] = -1.0
    tok = torch.randint(0, V, (M,), generator=g)
    for dtype in (BF16, F32):
        y = x.to(dtype)
        if kind == "lowest" and dtype == BF16:
            y = y.clamp(min=torch.finfo(BF16).min)
        got = run(y.cuda(), tok.cuda(), n)
        torch.cuda.synchronize()
        judge(y, tok, n, got)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [6, 1200])
def test_rows_without_a_distribution(M):
    V, n = 20000, 4
    g = torch.Generator().manual_seed(1)
    x = logits(g, M, V, F32)
    x[1] = -INF
    x[2, 19999] = NAN
    x[3, 0] = INF
    x[4, 77] = -NAN
    tok = torch.randint(0, V, (M,), generator=g)
    tok[5] = V
    tok[0] = -1
    lp, ent, rank, tl, ti = (t.cpu() for t in run(x.cuda(), tok.cuda(), n))
    assert lp[1] == -INF and ent[1] == 0 and rank[1] == 0
    assert (tl[1] == -INF).all() and (ti[1] == -1).all()
    for r in (2, 3, 4):
        assert lp[r].isnan() and ent[r].isnan() and tl[r].isnan().all() and (ti[r] == -1).all()
        assert rank[r] == (x[r] > x[r, tok[r]]).sum()
    for r in (0, 5):
        assert lp[r].isnan() and rank[r] == -1 and ent[r].isfinite() and tl[r].isfinite().all()
        assert torch.equal(ti[r].long(), torch.sort(x[r], descending=True, stable=True).indices[:n])


def masked_rows(g, M, V, kind, v):
    x = torch.randn(M, V, generator=g) * 3
    if kind == "islands":            # ordinary logits at the end of the row only
        x[:, :V - 17] = v
    elif kind == "front":            # whole pieces masked, the rest ordinary
        x[:, :V * 3 // 4] = v
    elif kind == "back":
        x[:, V // 4:] = v
    elif kind == "scattered":
        x.masked_fill_(torch.rand(M, V, generator=g) < 0.9, v)
    elif kind == "wholly":
        x[:] = v
    elif kind == "top":              # a few equal ones of the magnitude are the most likely
        x[:, torch.randperm(V, generator=g)[:9]] = -v
    elif kind == "top_alone":        # and far below them the rest
        x[:] = v
        x[:, V // 3] = -v
    else:                            # masks of several sizes, one on top of another
        pick = torch.rand(M, V, generator=g)
        x.masked_fill_(pick < 0.9, v)
        x.masked_fill_(pick < 0.6, v * 4)
        x.masked_fill_(pick < 0.3, -INF)
        x[:, :V // 2] = v * 2
    return x


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 3, 1200])
@pytest.mark.parametrize("kind", ["islands", "front", "back", "scattered", "wholly", "top",
                                  "top_alone", "several"])
@pytest.mark.parametrize("v", [-1e4, -1e6, -1e9, -1e10, -1e11, -1e12, -1e20, -1e30, -8e37])
def test_finite_masks_of_any_size(M, kind, v):
    V = 9001 if M > 100 else 20011
    g = torch.Generator().manual_seed(M)
    x = masked_rows(g, M, V, kind, v)
    tok = torch.randint(0, V, (M,), generator=g)
    tok[0] = V - 1
    for dtype in (BF16, F32):
        y = x.to(dtype)
        judge(y, tok, 5, run(y.cuda(), tok.cuda(), 5))


@pytest.mark.gpu
@pytest.mark.parametrize("M", [2, 1200])
@pytest.mark.parametrize("centre", [2.0 ** e * s for e in (18, 19, 20, 21, 22) for s in (-1, 1)])
@pytest.mark.parametrize("kind", ["around", "rising", "ordinary_above"])
def test_maxima_on_both_sides_of_a_power_of_two(M, centre, kind):
    """Logits a few units around +-2^18 .. 2^22 (fp32 holds them to 1/64 .. 1/2), so that the
    lanes' maxima lie on either side of any bound there and join."""
    V = 9001
    g = torch.Generator().manual_seed(int(abs(centre)) + M)
    x = torch.randn(M, V, generator=g) * 3 + centre
    if kind == "rising":
        x = torch.linspace(-40, 40, V).repeat(M, 1) + centre
    elif kind == "ordinary_above" and centre < 0:
        x[:, torch.randperm(V, generator=g)[:3]] = 1.5
    tok = torch.randint(0, V, (M,), generator=g)
    judge(x, tok, 5, run(x.cuda(), tok.cuda(), 5))


@pytest.mark.gpu
def test_more_rows_than_one_launch_holds():
    """2^24 rows of a workgroup each: every row has the values of its period's row.  (Copies and
    comparisons by slices, as for the norm.)"""
    periods, period, V = 2 ** 13, 2 ** 11 + 3, 7
    g = torch.Generator().manual_seed(13)
    base, tok = logits(g, period, V, BF16).cuda(), torch.randint(0, V, (period,), generator=g).cuda()
    x = base.expand(periods, period, V).reshape(-1, V)
    toks = tok.expand(periods, period).reshape(-1)
    assert len(x) > 2 ** 24

    def same(many, few):
        many = many.view(periods, *few.shape)
        return all((many[i:i + 1024] == few).all() for i in range(0, periods, 1024))

    assert same(x, base) and same(toks, tok)
    for a, b in zip(sbg.token_logprobs(x, toks, 2), sbg.token_logprobs(base, tok, 2)):
        assert same(a, b)


@pytest.mark.gpu
def test_same_bits_each_time_and_in_a_graph():
    g = torch.Generator().manual_seed(2)
    x, tok = logits(g, 3, 50001, BF16).cuda(), torch.randint(0, 50001, (3,), generator=g).cuda()
    ws, ws2 = (sbg.make_token_logprobs_workspace(3, 50001, 20) for _ in range(2))
    outs = sbg.token_logprobs(x, tok, 20, workspace=ws)
    outs = tuple(torch.zeros_like(t) for t in outs)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sbg.token_logprobs(x, tok, 20, workspace=ws, outs=outs)
    side = torch.cuda.Stream()
    for i in range(3):
        x.copy_(logits(g, 3, 50001, BF16))
        want = sbg.token_logprobs(x, tok, 20, workspace=ws2)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        again = sbg.token_logprobs(x, tok, 20, workspace=ws2, stream=side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(again, want))
    assert sbg.load().workspace_status(ws, 8192) == (0, 0)


# -- refusals ------------------------------------------------------------------------------------
BASE = dict(logits=0x10000000, tokens=0x20000000, logprob=0x21000000, entropy=0x22000000,
            rank=0x23000000, top_logprob=0x24000000, top_id=0x25000000, workspace=0x26000000,
            workspace_bytes=1 << 20, ld=5000, M=2, V=5000, top_n=5, logits_type=0, tokens_bytes=8)


@pytest.mark.parametrize("kw,code", [
    (dict(logits=None), -1), (dict(tokens=None), -1), (dict(logprob=None), -1),
    (dict(entropy=None), -1), (dict(rank=None), -1), (dict(top_id=None), -1),
    (dict(top_logprob=None), -1), (dict(M=-1), -1), (dict(V=0), -1), (dict(ld=4999), -1),
    (dict(top_n=-1), -1), (dict(logits_type=2), -1), (dict(tokens_bytes=2), -1),
    (dict(entropy=0x21000004), -1), (dict(logprob=0x10000000), -1), (dict(top_id=0x26000000), -1),
    (dict(top_n=33), -2), (dict(V=(1 << 30) + 1, ld=1 << 31), -2), (dict(logits=0x10000001), -2),
    (dict(logits=0x10000002, logits_type=1), -2), (dict(tokens=0x20000004), -2),
    (dict(rank=0x23000002), -2), (dict(workspace=0x26000080), -2),
    (dict(workspace=None), -3), (dict(workspace_bytes=64), -3), (dict(M=0, logits=None), 0)])
def test_refuses(kw, code):
    a = ops.TokenLogprobsArgs(**{**BASE, **kw})
    assert ops.library().lib.lowm_token_logprobs(ctypes.byref(a), None) == code


def test_workspace_bytes():
    f = ops.library().lib.lowm_token_logprobs_workspace_bytes
    assert f(2048, 49152, 5) == 0                    # enough rows: no row is cut
    assert f(1, 49152, 5) == f(500, 5000, 32) == 512 * 256 + 1024 * 34 * 8
    assert f(1, 4096, 5) == 0 and f(1, 4097, 0) > 0 and f(512, 99999, 1) == 0
    assert f(0, 5, 5) == f(1, 0, 5) == f(1, 5, 33) == f(1, 5, -1) == 0


@pytest.mark.gpu
def test_one_workspace_for_all_sizes_and_none_without_it():
    g = torch.Generator().manual_seed(12)
    ws = sbg.make_token_logprobs_workspace(1, 131072, 32)
    for M, V, n in ((1, 131072, 32), (400, 9000, 3), (64, 8193, 32), (511, 5000, 0), (7, 99999, 20),
                    (1, 4097, 1)):
        x, tok = logits(g, M, V, BF16), torch.randint(0, V, (M,), generator=g)
        got = sbg.token_logprobs(x.cuda(), tok.cuda(), n, workspace=ws)
        torch.cuda.synchronize()
        judge(x, tok, n, got)
        assert ws.count_nonzero() == 0
    with pytest.raises(ValueError):
        sbg.token_logprobs(x.cuda(), tok.cuda(), 1)


def test_python_checks():
    x = torch.zeros(2, 8, dtype=BF16)
    for bad in (lambda: sbg.token_logprobs(x, torch.zeros(2, dtype=torch.int64)),
                lambda: sbg.token_logprobs(x.half(), torch.zeros(2, dtype=torch.int64))):
        with pytest.raises((ValueError, TypeError)):
            bad()
