"""The paged 8-bit cache: rotary positions, append and read, attention, forked and compacted
pages, against their formulas in 64 bits and in plain Python.

Tolerances, with u = 2^-24 (half a step of fp32), 2^-9 half a step of bf16 at the top of its
binade and 2^-8 at its bottom, 2^-12 and 2^-11 the same for fp16:

  rotary     the angle's remainder is rounded to fp32 as a number of half turns up to 1: at most
             u * pi radians off, then sine and cosine by 4 u each at most, and three roundings of
             the products and their sum: 10 u (|x| + |y|) scale, then the type's own half step.
  append     s is one quotient (u s); q = x / s is rounded to the nearest level from an fp32
             quotient: half a step and u q.  Where s grows, an earlier level is off by half a step
             more each time.
  attention  scores: fp16 products are exact, their fp32 sum of D terms in any order is within
             (D + 3) u sum |q k|, 3 more for the scale's three roundings; call that E (natural
             units) plus 4 u |x - max| from the exponent.  Weights: relative 2 E + 8 u, and fp16's
             2^-11 in the second product, or 2^-25 of the page's largest weight below its normal
             numbers.  So |out - ref| <= sum w |v| (2 E + 2^-11 + n u) + 2^-24 max |v| with n u
             for sums over the pages, tiles and places, and bf16's half step at the end.
"""
from __future__ import annotations

import itertools
import math
import random
import zlib

import pytest
import torch

import split_bf16_gemm_amd as sbg
from split_bf16_gemm_amd import cache as cache_ops
from split_bf16_gemm_amd.cache import PAGE

U = 2.0 ** -24
BF16, F32, I32, F64 = torch.bfloat16, torch.float32, torch.int32, torch.float64
FP8 = torch.float8_e4m3fn
HALF = {BF16: 2.0 ** -8, F32: U}
COUNTERS = 2 * 2 * 512 * 4     # bytes of cache_attention's workspace that are zero between calls
gpu = pytest.mark.gpu


def ints(x, dev="cuda"):
    return torch.tensor(x, dtype=I32, device=dev)


def gen(*seed):
    return torch.Generator().manual_seed(zlib.crc32(repr(seed).encode()))


def randn(g, *shape, dtype=BF16, std=1.0, dev="cuda"):
    return (torch.randn(*shape, generator=g) * std).to(dtype).to(dev)


def logical(cache):
    """(k, v) fp64 [P, 64, H, D] on the CPU, as the bytes and scales say."""
    k = cache.k.cpu().float().double() * cache.k_scale.cpu().double()[..., None, None, None]
    v = cache.v.cpu().float().double() * cache.v_scale.cpu().double()[..., None, None, None]
    P, H = k.shape[:2]
    return (k.permute(0, 3, 1, 2, 4).reshape(P, PAGE, H, -1),
            v.permute(0, 2, 4, 1, 3).reshape(P, PAGE, H, -1))


def by_token(cache):
    """The bytes of keys and values [P, 64, H, D] on the CPU."""
    k, v = (x.view(torch.int8).cpu() for x in cache[:2])
    P, H = k.shape[:2]
    return (k.permute(0, 3, 1, 2, 4).reshape(P, PAGE, H, -1),
            v.permute(0, 2, 4, 1, 3).reshape(P, PAGE, H, -1))


def random_cache(g, P, H, D, kind=torch.int8):
    """Every byte drawn (NaNs of e4m3 left out), every scale positive."""
    c = sbg.make_kv_cache(P, H, D, dtype=kind)
    for x in (c.k, c.v):
        b = torch.randint(-128, 128, x.shape, generator=g, dtype=torch.int8)
        if kind == FP8:
            b[(b == 127) | (b == -1)] = 5
        x.view(torch.int8).copy_(b)
    unit = 0.01 if kind == torch.int8 else 0.005
    for x in (c.k_scale, c.v_scale):
        x.copy_(unit * torch.exp(0.5 * torch.randn(x.shape, generator=g)))
    return c


# ---------------------------------------------------------------------------------------------
# rotary
# ---------------------------------------------------------------------------------------------
def rotary_reference(x, pos, freqs, layout, first, scale, inverse):
    x, R = x.double().cpu(), 2 * len(freqs)
    a = torch.outer(pos.double().cpu(), freqs.cpu()) * (-1 if inverse else 1)
    c, s = (scale * torch.cos(a))[:, None], (scale * torch.sin(a))[:, None]
    y = x.clone()
    one = slice(first, first + R // 2) if layout == "half" else slice(first, first + R, 2)
    two = slice(first + R // 2, first + R) if layout == "half" else slice(first + 1, first + R, 2)
    y[..., one] = x[..., one] * c - x[..., two] * s
    y[..., two] = x[..., one] * s + x[..., two] * c
    err = torch.zeros_like(x)
    err[..., one] = err[..., two] = 10 * U * scale * (x[..., one].abs() + x[..., two].abs())
    return y, err


def check_rotary(got, want, err):
    bound = err + (want.abs() + err) * HALF[got.dtype]
    assert bool(((got.double().cpu() - want).abs() <= bound).all())


@gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
@pytest.mark.parametrize("case", [
    # T, Hq, Hk, D, R, first, dtype, far
    (1, 32, 8, 128, 128, 0, BF16, 100), (5, 3, 1, 64, 32, 0, BF16, 1 << 20),
    (3, 2, 2, 80, 20, 7, F32, 5000), (70, 1, 1, 2, 2, 0, BF16, 10), (9, 7, 3, 33, 18, 15, F32, 100),
    (2, 40, 0, 256, 64, 192, BF16, 1 << 30), (513, 4, 2, 96, 96, 0, F32, 1 << 17),
    (2, 5, 1, 1024, 1024, 0, BF16, 300)], ids=lambda c: f"t{c[0]}_d{c[3]}_r{c[4]}")
def test_rotary(case, layout):
    T, Hq, Hk, D, R, first, dtype, far = case
    g = gen(T, D, R)
    freqs = sbg.rotary_frequencies(R)
    pos = torch.randint(0, far, (T,), generator=g).cuda()
    wide = randn(g, T, (Hq + 2 * Hk) * D + 3, dtype=dtype)
    q = wide[:, :Hq * D].view(T, Hq, D)
    k = wide[:, Hq * D:(Hq + Hk) * D].view(T, Hk, D) if Hk else None
    before = wide.clone()
    for scale, inverse, ps in ((1.0, False, pos), (1.25, True, pos.int())):
        qo, ko = sbg.rotary(q, k, ps, freqs, layout=layout, first=first, scale=scale,
                            inverse=inverse)
        check_rotary(qo, *rotary_reference(q, pos, freqs, layout, first, scale, inverse))
        if Hk:
            check_rotary(ko, *rotary_reference(k, pos, freqs, layout, first, scale, inverse))
        assert torch.equal(wide, before)
    # in place: the same bits, and the buffer's other columns as they were
    qo, ko = sbg.rotary(q, k, pos, freqs, layout=layout, first=first)
    sbg.rotary(q, k, pos, freqs, layout=layout, first=first, q_out=q, k_out=k)
    assert torch.equal(q, qo) and (k is None or torch.equal(k, ko))
    assert torch.equal(wide[:, (Hq + Hk) * D:], before[:, (Hq + Hk) * D:])


@gpu
@pytest.mark.parametrize("layout", ["half", "interleaved"])
def test_rotary_inverse_is_the_gradient(layout):
    """<g, J dx> = <J^T g, dx> with J^T the inverse turn, and J by differences: the map is
    linear, so a difference of any length is exact but for rounding."""
    g = gen(7, layout)
    T, H, D = 6, 3, 64
    freqs = sbg.rotary_frequencies(32)
    pos = torch.randint(0, 10000, (T,), generator=g).cuda()
    kw = dict(layout=layout, first=8, scale=1.5)
    x, dx, up = (randn(g, T, H, D, dtype=F32) for _ in range(3))
    far = sbg.rotary(x + dx, None, pos, freqs, **kw)[0].double() - \
        sbg.rotary(x, None, pos, freqs, **kw)[0].double()
    back = sbg.rotary(up, None, pos, freqs, inverse=True, **kw)[0].double()
    lhs, rhs = (far * up.double()).sum(), (back * dx.double()).sum()
    # each term off by 30 u of its operands' size at most
    slack = 30 * U * 3 * ((x.abs() + dx.abs()).double() * up.abs().double()).sum() * 2
    assert (lhs - rhs).abs() <= slack


def test_rotary_frequencies():
    f = sbg.rotary_frequencies(8, device="cpu")
    assert torch.allclose(f, torch.tensor([1, 0.1, 0.01, 0.001], dtype=F64), rtol=1e-14)
    assert torch.equal(sbg.rotary_frequencies(8, scaling="linear", factor=4, device="cpu"), f / 4)
    b = sbg.rotary_frequencies(8, scaling="base", factor=4, device="cpu")
    assert b[0] == 1 and math.isclose(b[-1], f[-1] / 4, rel_tol=1e-12)
    p = sbg.rotary_frequencies(128, scaling="by_parts", factor=8, original_length=4096,
                               device="cpu")
    f = sbg.rotary_frequencies(128, device="cpu")
    turns = 4096 * f / (2 * math.pi)
    assert torch.equal(p[turns > 32], f[turns > 32])
    assert torch.allclose(p[turns < 1], f[turns < 1] / 8, rtol=1e-14)
    mid = (turns > 1) & (turns < 32)
    assert ((p[mid] < f[mid]) & (p[mid] > f[mid] / 8)).all()
    for bad in (dict(rotary_dim=7), dict(rotary_dim=0), dict(rotary_dim=8, factor=0.5),
                dict(rotary_dim=8, scaling="x"), dict(rotary_dim=2, scaling="base", factor=2),
                dict(rotary_dim=8, scaling="by_parts", low=3, high=2), dict(rotary_dim=8, base=0)):
        with pytest.raises(ValueError):
            sbg.rotary_frequencies(**bad, device="cpu")


# ---------------------------------------------------------------------------------------------
# append and read
# ---------------------------------------------------------------------------------------------
def step_of(kind):
    """Half a level's distance, relative to (the value, the page's largest value)."""
    return (0.0, 0.5 / 127) if kind == torch.int8 else (2.0 ** -4, 2.0 ** -10 / 448)


class Model:
    """A cache's contents as they were written, with the bound that each element's value in
    the cache has to keep, followed call by call in 64 bits."""

    def __init__(self, cache):
        self.kind = FP8 if cache.k.dtype == FP8 else torch.int8
        self.val = list(logical(cache))
        self.err = [torch.zeros_like(x) for x in self.val]
        self.scale = [cache.k_scale.double().cpu(), cache.v_scale.double().cpu()]
        self.top = 448 if self.kind == FP8 else 127
        # what lies behind a sequence keeps its bytes, whatever they stand for at the new scale
        self.bytes = by_token(cache)
        self.behind = torch.zeros(len(cache.k), PAGE, dtype=torch.bool)

    def append(self, k, v, table, lens, starts):
        for which, x in enumerate((k, v)):
            x = x.double().cpu()
            for b, end in enumerate(lens):
                n = starts[b + 1] - starts[b]
                rows = x[starts[b]:starts[b + 1]]
                for p in sorted({(end - n + j) // PAGE for j in range(n) if end - n + j >= 0}):
                    page = table[b][p]
                    lo, hi = max(end - n, p * PAGE, 0), min(end, (p + 1) * PAGE)
                    new = rows[lo - (end - n):hi - (end - n)]
                    a, z = lo - p * PAGE, hi - p * PAGE
                    self.behind[page, :z], self.behind[page, z:] = False, True
                    s = new.abs().amax((0, 2)) / self.top
                    rel, flat = step_of(self.kind)
                    if a:
                        grown = s > self.scale[which][page]
                        s = torch.maximum(s, self.scale[which][page])
                        old = self.val[which][page, :a]
                        more = (rel * old.abs() + (flat * self.top) * s[None, :, None]) * 1.001
                        self.err[which][page, :a] += grown[None, :, None] * more
                    self.scale[which][page] = s
                    self.val[which][page, a:z] = new
                    self.err[which][page, a:z] = \
                        (rel * new.abs() + flat * self.top * s[None, :, None]) * 1.0001

    def check(self, cache):
        for got, want, err in zip(logical(cache), self.val, self.err):
            near = (got - want).abs() <= err + 4 * U * want.abs()
            assert bool((near | self.behind[..., None, None]).all())
        for got, want in zip(by_token(cache), self.bytes):
            assert torch.equal(got[self.behind], want[self.behind])
        for got, want in zip((cache.k_scale, cache.v_scale), self.scale):
            assert bool(((got.double().cpu() - want).abs() <= 2 * U * want).all())


APPENDS = [
    # H, D, kind, dtype, [new tokens of each sequence in each call]
    (2, 16, torch.int8, BF16, [[3, 1, 70], [1, 1, 1], [1, 130, 2], [64, 1, 63]]),
    (1, 64, FP8, F32, [[1, 64, 65], [1, 1, 1], [63, 64, 127], [1, 0, 1]]),
    (3, 80, torch.int8, F32, [[129, 1], [0, 1], [7, 200]]),
    (2, 128, torch.int8, BF16, [[1, 1, 1, 1, 1]] * 5),
    (1, 128, FP8, BF16, [[200], [1], [1]]),
    (2, 144, FP8, BF16, [[10, 100], [60, 1], [1, 1]]),
    (1, 256, torch.int8, BF16, [[64, 63], [1, 1], [1, 2]]),
]


@gpu
@pytest.mark.parametrize("case", APPENDS, ids=lambda c: f"h{c[0]}_d{c[1]}_{len(c[4])}")
def test_append_and_read(case):
    H, D, kind, dtype, calls = case
    g = gen(H, D, len(calls))
    B = len(calls[0])
    most = max(sum(c[b] for c in calls) for b in range(B))
    W = -(-most // PAGE) + 1
    P = B * W + 2
    cache = random_cache(g, P, H, D, kind)
    ids = torch.randperm(P, generator=g)[:B * W].view(B, W).tolist()
    table, model, lens = ints(ids), Model(cache), [0] * B
    for step, new in enumerate(calls):
        T = sum(new)
        starts = [0, *itertools.accumulate(new)]
        lens = [x + n for x, n in zip(lens, new)]
        # later tokens are larger more often than not, so that scales grow
        wide = randn(g, T, 2 * H * D + 5, dtype=dtype, std=1.0 + step)
        k, v = wide[:, :H * D].view(T, H, D), wide[:, H * D:2 * H * D].view(T, H, D)
        uniform = len(set(new)) == 1
        rs = None if uniform else ints(starts)
        sbg.cache_append(k, v, cache, table, ints(lens), row_starts=rs)
        model.append(k, v, ids, lens, starts)
        model.check(cache)
        rk, rv = sbg.cache_read(cache, table, ints(lens), row_starts=rs, rows=T)
        lk, lv = logical(cache)
        for got, full in ((rk, lk), (rv, lv)):
            for b in range(B):
                for j in range(new[b]):
                    pos = lens[b] - new[b] + j
                    want = full[ids[b][pos // PAGE], pos % PAGE].float().to(BF16)
                    assert torch.equal(got[starts[b] + j].cpu(), want)


@gpu
@pytest.mark.parametrize("kind", [torch.int8, FP8])
def test_append_keeps_bytes_while_the_scale_stands(kind):
    """A smaller token changes neither the scale nor another byte; the same call twice changes
    nothing at all."""
    g = gen(11)
    H, D = 2, 48
    cache = random_cache(g, 3, H, D, kind)
    table, k = ints([[1]]), randn(g, 9, H, D)
    sbg.cache_append(k, k, cache, table, ints([9]))
    before = [x.view(torch.int8).clone() for x in cache]
    small = k[:1] * 0.5
    sbg.cache_append(small, small, cache, table, ints([10]))
    for x, y in zip(cache[2:], before[2:]):
        assert torch.equal(x.view(torch.int8), y)
    kb, vb = cache.k.view(torch.int8).clone(), cache.v.view(torch.int8).clone()
    kb[1, :, :, 9], vb[1, :, 0, :, 9] = before[0][1, :, :, 9], before[1][1, :, 0, :, 9]
    assert torch.equal(kb, before[0]) and torch.equal(vb, before[1])
    now = [x.view(torch.int8).clone() for x in cache]
    sbg.cache_append(small, small, cache, table, ints([10]))
    assert all(torch.equal(x.view(torch.int8), y) for x, y in zip(cache, now))


@gpu
@pytest.mark.parametrize("kind", [torch.int8, FP8])
def test_append_zeros_and_nan(kind):
    H, D = 2, 32
    cache = random_cache(gen(3), 2, H, D, kind)
    table = ints([[1]])
    zero = torch.zeros(5, H, D, dtype=BF16, device="cuda")
    sbg.cache_append(zero, zero, cache, table, ints([5]))
    assert (cache.k_scale[1] == 0).all() and (cache.v_scale[1] == 0).all()
    k, v = sbg.cache_read(cache, table, ints([5]), rows=5)
    assert (k == 0).all() and (v == 0).all()
    one = torch.ones(1, H, D, dtype=BF16, device="cuda")
    sbg.cache_append(one, one, cache, table, ints([6]))
    k, v = sbg.cache_read(cache, table, ints([6]), rows=6)
    assert (k[:5] == 0).all() and (k[5] == 1).all() and (v[5] == 1).all()
    # an infinity, or a NaN, in one head takes that head's page, until it begins again
    bad = one.clone()
    bad[0, 1, 7] = math.inf
    sbg.cache_append(bad, one, cache, table, ints([7]))
    sbg.cache_append(one, bad * float("nan"), cache, table, ints([8]))
    k, v = sbg.cache_read(cache, table, ints([8]), rows=8)
    assert torch.isnan(k[:, 1]).all() and (k[7, 0] == 1).all()
    assert torch.isnan(v).all()
    sbg.cache_append(one, one, cache, table, ints([1]))
    k, v = sbg.cache_read(cache, table, ints([1]), rows=1)
    assert (k == 1).all() and (v == 1).all()


@gpu
def test_append_leaves_out_what_cannot_be():
    """Positions below 0 or past the table, pages that are none, rows of no sequence: nothing
    else is written, and read leaves their rows as they were."""
    g = gen(5)
    H, D, P = 2, 32, 6
    cache = random_cache(g, P, H, D)
    k = randn(g, 140, H, D)
    before = [x.clone() for x in cache]
    # sequence 0: three of its five rows before its beginning; 1: no page -7, nor page 6;
    # 2: past its table of two pages; 3: none; then rows of no sequence
    table = ints([[2, 0], [-7, P], [4, 5], [1, 3]])
    starts, lens = ints([0, 5, 70, 100, 100]), ints([2, 66, 135, 17])
    sbg.cache_append(k, k, cache, table, lens, row_starts=starts)
    for p in (0, 1, 3, 4):
        assert all(torch.equal(x[p], y[p]) for x, y in zip(cache, before))
    assert not torch.equal(cache.k[2], before[0][2]) and not torch.equal(cache.k[5], before[0][5])
    ko = torch.full((140, H, D), 9.0, dtype=BF16, device="cuda")
    vo = ko.clone()
    sbg.cache_read(cache, table, lens, row_starts=starts, k_out=ko, v_out=vo)
    lk, lv = logical(cache)
    for out, full in ((ko, lk), (vo, lv)):
        want = torch.full((140, H, D), 9.0, dtype=BF16)
        for j in (3, 4):
            want[j] = full[2, j - 3].float().to(BF16)
        for j in range(30):
            if 105 + j < 128:
                want[70 + j] = full[5, 105 + j - 64].float().to(BF16)
        assert torch.equal(out.cpu(), want)
    # garbage in the row bounds is held to the rows that are there
    sbg.cache_append(k, k, cache, table, lens, row_starts=ints([-5, 1 << 30, 3, -9, 7]))
    sbg.cache_append(k[:0], k[:0], cache, table, lens)


# ---------------------------------------------------------------------------------------------
# attention
# ---------------------------------------------------------------------------------------------
def attention_reference(q, cache, table, lens, starts, scale, window):
    """(out, lse, bound of out's error, bound of lse's), 64 bits, rows of no sequence NaN."""
    lk, lv = logical(cache)
    T, Hq, D = q.shape
    P, _, H, _ = lk.shape
    out = torch.full((T, Hq, D), math.nan, dtype=F64)
    lse = torch.full((T, Hq), math.nan, dtype=F64)
    err, lerr = torch.zeros_like(out), torch.zeros_like(lse)
    q = q.double().cpu()
    table = table.tolist()
    for b, end in enumerate(lens):
        n = starts[b + 1] - starts[b]
        pages = table[b]
        ok = torch.tensor([0 <= p < P for p in pages]).repeat_interleave(PAGE)
        ids = torch.tensor([p if 0 <= p < P else 0 for p in pages])
        K, V = lk[ids].reshape(-1, H, D), lv[ids].reshape(-1, H, D)
        for j in range(n):
            t, pos = starts[b] + j, end - n + j
            at = torch.arange(len(K))
            sees = ok & (at <= pos)
            if window:
                sees &= at > pos - window
            keys, vals = K[sees], V[sees]
            out[t], lse[t] = 0, -math.inf
            if not len(keys):
                continue
            for h in range(Hq):
                kk, vv = keys[:, h // (Hq // H)], vals[:, h // (Hq // H)]
                x = scale * (kk @ q[t, h])
                lse[t, h] = torch.logsumexp(x, 0)
                w = torch.exp(x - lse[t, h])
                out[t, h] = w @ vv
                E = abs(scale) * (D + 3) * U * (kk.abs() @ q[t, h].abs())
                E = E + 4 * U * (x.max() - x) + 4 * U * x.abs()
                n_sum = (64 + len(pages) * 4 + 16) * U
                off = 2 * E + (w @ E) + 2.0 ** -11 + n_sum
                err[t, h] = (w * off) @ vv.abs() + 2.0 ** -24 * vv.abs().amax()
                lerr[t, h] = E.max() + n_sum + 8 * U * (1 + lse[t, h].abs())
    return out, lse, err, lerr


def check_attention(q, cache, table, lens, starts, *, window=0, scale=None, rs="given", ws=None):
    T, Hq, D = q.shape
    scale = D ** -0.5 if scale is None else scale
    if ws is None:
        ws = sbg.make_cache_attention_workspace(T, Hq, cache.k.shape[1], D)
        ws[COUNTERS:].fill_(0xff)     # nothing there is read before it is written
    out = torch.full((T, Hq, D), 7.0, dtype=BF16, device="cuda")
    lse = torch.full((T, Hq), 7.0, device="cuda")
    sbg.cache_attention(q, cache, table, ints(lens), window=window, scale=scale, workspace=ws,
                        row_starts=None if rs is None else ints(starts), out=out, lse_out=lse)
    assert T == 0 or not ws[:COUNTERS].any()     # left as it was found
    ref, rl, err, lerr = attention_reference(q, cache, table, lens, starts, scale, window)
    got, gl = out.double().cpu(), lse.double().cpu()
    none = torch.isnan(rl)
    assert (got[none] == 7).all() and (gl[none] == 7).all()
    ref, rl, err, lerr, got, gl = (x[~none] for x in (ref, rl, err, lerr, got, gl))
    empty = torch.isneginf(rl)
    assert (got[empty] == 0).all() and torch.isneginf(gl[empty]).all()
    assert not torch.isnan(got).any()
    bound = err + (ref.abs() + err) * HALF[BF16]
    assert bool(((got - ref).abs() <= bound).all()), ((got - ref).abs() / bound).max().item()
    assert bool(((gl - rl).abs()[~empty] <= lerr[~empty]).all())
    return out, lse


def tables(g, P, lens, extra=1):
    counts = [-(-n // PAGE) for n in lens]
    ids = torch.randperm(P, generator=g).tolist()
    assert sum(counts) <= P
    rows, W = [], max(counts) + extra
    for n in counts:
        rows.append(ids[:n] + [-1] * (W - n))
        ids = ids[n:]
    return ints(rows)


ATTENTIONS = [
    # Hq, H, D, kind, lens, new rows, window
    (1, 1, 16, torch.int8, [1], [1], 0),
    (8, 2, 64, torch.int8, [64, 65, 63, 1], [1, 1, 1, 1], 0),
    (8, 8, 128, FP8, [200, 1, 128], [1, 1, 1], 0),
    (32, 2, 128, torch.int8, [1000], [1], 0),
    (20, 1, 80, torch.int8, [130, 5], [1, 1], 0),
    (6, 2, 96, FP8, [70, 300, 64], [5, 1, 64], 0),
    (12, 4, 112, torch.int8, [500, 129], [3, 40], 100),
    (4, 2, 192, torch.int8, [333, 90], [2, 1], 0),
    (16, 2, 208, FP8, [129, 300], [1, 7], 0),
    (8, 1, 256, torch.int8, [700, 1], [9, 1], 65),
    (4, 1, 256, FP8, [257], [1], 1),
    (16, 8, 64, FP8, [3000, 10], [1, 1], 0),
    (8, 4, 32, torch.int8, [300] * 70, [1] * 70, 0),
    (2, 1, 48, torch.int8, [257, 100, 3], [100, 100, 1], 0),
    (4, 4, 128, torch.int8, [640], [1], 64),
    (9, 3, 160, torch.int8, [190], [30], 0),
    (24, 8, 176, FP8, [65, 200], [1, 1], 0),
    (3, 1, 240, torch.int8, [100, 320], [4, 33], 33),
    (16, 2, 128, torch.int8, [2000, 100], [20, 30], 0),
    (8, 2, 64, FP8, [1500], [40], 0),
    (8, 2, 192, FP8, [900, 70], [33, 20], 0),
    (16, 2, 256, torch.int8, [1200], [25], 200),
    (8, 1, 128, torch.int8, [3000, 64], [6, 8], 0),
    (8, 1, 192, torch.int8, [600], [8], 70),
    (4, 1, 256, FP8, [500], [6], 0),
    (10, 2, 128, FP8, [20000], [26], 0),
]


@gpu
@pytest.mark.parametrize("case", ATTENTIONS,
                         ids=lambda c: f"h{c[0]}_{c[1]}_d{c[2]}_b{len(c[4])}_l{max(c[4])}")
def test_attention(case):
    Hq, H, D, kind, lens, new, window = case
    g = gen(Hq, D, len(lens))
    P = sum(-(-n // PAGE) for n in lens) + 3
    cache = random_cache(g, P, H, D, kind)
    table = tables(g, P, lens)
    T = sum(new)
    starts = [0, *itertools.accumulate(new)]
    wide = randn(g, T, (Hq + 2) * D, std=1.5)
    q = wide[:, D:(Hq + 1) * D].view(T, Hq, D)
    out, lse = check_attention(q, cache, table, lens, starts, window=window)
    if len(set(new)) == 1:
        again, lse2 = check_attention(q, cache, table, lens, starts, window=window, rs=None)
        assert torch.equal(again, out) and torch.equal(lse, lse2)
    # heads first in memory
    q2 = q.transpose(0, 1).contiguous().transpose(0, 1)
    ws = sbg.make_cache_attention_workspace(T, Hq, H, D)
    wide_table = torch.full((len(lens), table.shape[1] + 5), 1 << 30, dtype=I32, device="cuda")
    wide_table[:, :table.shape[1]] = table
    third, none = sbg.cache_attention(q2, cache, wide_table[:, :table.shape[1]], ints(lens),
                                      row_starts=ints(starts), window=window, workspace=ws)
    assert torch.equal(third, out) and none is None
    # larger products are smaller scores
    check_attention(q, cache, table, lens, starts, window=window, scale=-0.05, ws=ws)


@gpu
def test_attention_rows_that_see_nothing():
    """No tokens, rows before the beginning, pages that are none, an odd table, rows of no
    sequence (left as they were)."""
    g = gen(21)
    H, D, P = 2, 64, 12
    cache = random_cache(g, P, H, D, FP8)
    table = ints([[3, 1, 2], [4, 5, 6], [-1, -1, -1], [7, -1, 8], [9, 10, 11], [P, 0, 1 << 30]])
    lens = [0, 2, 100, 192, 1000, 100]
    starts = [0, 1, 6, 8, 9, 10, 11]
    q = randn(g, 14, 4, D)
    check_attention(q, cache, table, lens, starts)
    check_attention(q, cache, table, lens, starts, window=70)
    # a sequence longer than its table sees what the table has; windows may leave nothing
    check_attention(q, cache, table, lens, starts, window=3)
    check_attention(q[:0], cache, table[:0], [], [0], rs=None, ws=torch.empty(0, device="cuda"))


@gpu
@pytest.mark.parametrize("kind", [torch.int8, FP8])
def test_attention_what_is_masked_does_not_reach_a_row(kind):
    """Bytes behind a sequence's end may be anything, NaNs of e4m3 among them, and so may other
    pages' scales; a page with scale NaN takes the rows that see it, and no other."""
    g = gen(22)
    H, D, P = 1, 128, 8
    lens, starts = [150, 64], [0, 100, 101]
    cache = random_cache(g, P, H, D, kind)
    table = ints([[1, 2, 3], [4, 5, -1]])
    q = randn(g, 101, 2, D)
    ws = sbg.make_cache_attention_workspace(101, 2, H, D)
    run = lambda: sbg.cache_attention(q, cache, table, ints(lens), row_starts=ints(starts),  # noqa
                                      workspace=ws, lse_out=torch.empty(101, 2, device="cuda"))
    want, lse = run()
    check_attention(q, cache, table, lens, starts)
    cache.k.view(torch.int8)[3, :, :, 150 - 128:] = 0x7f
    cache.v.view(torch.int8)[3].view(H, 4, D, 16).permute(0, 1, 3, 2).reshape(H, 64, D)
    v = cache.v.view(torch.int8)
    for t in range(150 - 128, 64):
        v[3, :, t // 16, :, t % 16] = -1
    for p in (0, 5, 6, 7):
        cache.k_scale[p], cache.v_scale[p] = math.nan, math.inf
        cache.k.view(torch.int8)[p] = 0x7f
        v[p] = 0x7f
    got, lse2 = run()
    assert torch.equal(got, want) and torch.equal(lse, lse2)
    # page 2 of sequence 0: tokens 64 to 127; its rows stand at 50 to 149
    cache.v_scale[2] = math.nan
    got, _ = run()
    assert torch.isnan(got[14:100]).all()
    assert torch.equal(got[:14], want[:14]) and torch.equal(got[100], want[100])
    cache.v_scale[2] = 1.0
    cache.k_scale[2] = math.nan
    got, lse2 = run()
    assert torch.isnan(got[14:100]).all() and torch.isnan(lse2[14:100]).all()
    assert torch.equal(got[:14], want[:14])


@gpu
def test_attention_magnitudes():
    """Queries of any size, rows of zeros, scales of zero, one weight that is all, and rows of q
    with an infinity or a NaN."""
    g = gen(23)
    H, D, P = 1, 64, 5
    cache = random_cache(g, P, H, D)
    table, lens, starts = ints([[0, 1, 2]]), [170], [0, 6]
    q = randn(g, 6, 4, D)
    for r, f in enumerate((1e-30, 1e-38, 0.0, 30.0, 1e4, 1.0)):
        q[r] *= f
    check_attention(q, cache, table, lens, starts)
    check_attention(q[5:6] * 1e30, cache, table, lens, [0, 1], scale=1e-31)
    cache.k_scale[1] = 0
    cache.v_scale[2] = 0
    check_attention(q, cache, table, lens, starts)
    cache.v_scale[0] = 1e-30
    check_attention(q, cache, table, lens, starts)
    q[1, 2, 5], q[3, 0, 63] = math.inf, math.nan
    ws = sbg.make_cache_attention_workspace(6, 4, H, D)
    out, _ = sbg.cache_attention(q, cache, table, ints(lens), workspace=ws)
    bad = torch.zeros(6, 4, dtype=torch.bool, device="cuda")
    bad[1, 2] = bad[3, 0] = True
    assert torch.isnan(out[bad]).all() and torch.isfinite(out[~bad].float()).all()


@gpu
@pytest.mark.parametrize("case", [
    # Hq, H, D, kind, lens, new rows, window
    (8, 1, 64, torch.int8, [900], [700], 100),
    (8, 1, 128, FP8, [513, 70], [513, 70], 0),
    (4, 1, 192, torch.int8, [700], [650], 70),
    (2, 2, 64, torch.int8, [600, 3000], [90, 30], 65),
    (2, 2, 96, FP8, [400, 3000], [1, 40], 500),
    (32, 8, 16, torch.int8, [1100], [1000], 0),
    (32, 8, 16, FP8, [1100, 64], [1000, 3], 700),
], ids=lambda c: f"h{c[0]}_{c[1]}_d{c[2]}_n{c[5][0]}_w{c[6]}")
def test_attention_of_whole_prompts(case):
    """Rows of many tiles, which see more and more pages, or through a window ever others."""
    Hq, H, D, kind, lens, new, window = case
    g = gen(41, Hq, D, window)
    P = sum(-(-n // PAGE) for n in lens) + 2
    cache = random_cache(g, P, H, D, kind)
    starts = [0, *itertools.accumulate(new)]
    q = randn(g, sum(new) + 2, Hq, D, std=1.5)
    check_attention(q, cache, tables(g, P, lens), lens, starts, window=window)


@gpu
@pytest.mark.parametrize("Hq,H,window", [(8, 1, 100), (8, 1, 0), (2, 2, 70), (32, 8, 130)])
def test_attention_of_prompts_past_their_table(Hq, H, window):
    """Tables of fewer pages than the sequences have: later rows see what there is, or, through a
    window, nothing."""
    g = gen(42, Hq, window)
    D, P, lens, new = 32, 40, [900, 500, 64], [700, 300, 64]
    cache = random_cache(g, P, H, D, FP8)
    table = tables(g, P, lens)[:, :5].contiguous()
    starts = [0, *itertools.accumulate(new)]
    q = randn(g, sum(new), Hq, D, std=1.5)
    check_attention(q, cache, table, lens, starts, window=window)


@gpu
@pytest.mark.parametrize("G", [1, 3, 16, 40])
def test_attention_long_and_shared(G):
    """Sequences cut over many workgroups beside short ones; the rows of several tiles."""
    g = gen(24, G)
    H, D, P = 2, 64, 700
    lens, new = [20001, 3, 7000, 64, 0, 10000], [1, 1, 2, 1, 1, 3]
    cache = random_cache(g, P, H, D)
    table = tables(g, P, lens)
    starts = [0, *itertools.accumulate(new)]
    q = randn(g, sum(new), H * G, D, std=2.0)
    ws = sbg.make_cache_attention_workspace(sum(new), H * G, H, D)
    out, lse = check_attention(q, cache, table, lens, starts, ws=ws)
    check_attention(q, cache, table, lens, starts, window=5000, ws=ws)
    # whoever joins the parts, the bits are the same
    for _ in range(5):
        again, lse2 = sbg.cache_attention(q, cache, table, ints(lens), row_starts=ints(starts),
                                          workspace=ws, lse_out=torch.empty_like(lse))
        assert torch.equal(again, out) and torch.equal(lse2, lse)


@gpu
def test_attention_past_32_bits():
    """A cache whose bytes pass 2^31 in keys and in values: pages at both ends."""
    H, D = 8, 128
    P = (1 << 31) // (H * D * PAGE) + 40
    cache = sbg.make_kv_cache(P, H, D)
    g = gen(25)
    few = random_cache(g, 8, H, D)
    ids = [P - 1, 3, P - 40, P - 2, 0, P - 17, 5, P - 30]
    for x, y in zip(cache, few):
        x[torch.tensor(ids, device="cuda")] = y
    lens, starts = [300, 170], [0, 1, 2]
    q = randn(g, 2, 16, D)
    big, small = ints([ids[:5], ids[5:] + [-1] * 2]), ints([[0, 1, 2, 3, 4], [5, 6, 7, -1, -1]])
    ws = sbg.make_cache_attention_workspace(2, 16, H, D)
    want, _ = check_attention(q, few, small, lens, starts, ws=ws)
    got, _ = sbg.cache_attention(q, cache, big, ints(lens), workspace=ws)
    assert torch.equal(got, want)
    k = randn(g, 2, H, D)
    sbg.cache_append(k, k, cache, big, ints([301, 171]))
    sbg.cache_append(k, k, few, small, ints([301, 171]))
    for x, y in zip(cache, few):
        assert torch.equal(x[torch.tensor(ids, device="cuda")].view(torch.int8), y.view(torch.int8))


@gpu
def test_attention_many_sequences():
    """More sequences than a wavefront has lanes, most of one page, several of none."""
    g = gen(26)
    H, D, B = 1, 32, 200
    rng = random.Random(1)
    lens = [rng.choice([0, 1, 5, 64, 65, 300]) for _ in range(B)]
    new = [rng.choice([0, 1, 1, 2]) for _ in range(B)]
    P = sum(-(-n // PAGE) for n in lens)
    cache = random_cache(g, P, H, D)
    starts = [0, *itertools.accumulate(new)]
    q = randn(g, sum(new) + 3, 4, D)
    check_attention(q, cache, tables(g, P, lens), lens, starts)


@gpu
@pytest.mark.parametrize("G", [1, 8, 40])
def test_attention_row_starts_that_fall(G):
    """Rows counted twice: nothing is written, and nothing else is touched."""
    g = gen(27)
    cache = random_cache(g, 4, 2, 32)
    table, lens = ints([[0, 1], [2, 3], [1, 0], [3, 2]]), ints([100, 128, 70, 128])
    q = randn(g, 12, 2 * G, 32)
    ws = sbg.make_cache_attention_workspace(12, 2 * G, 2, 32)
    out, lse = torch.full_like(q, 5.0), torch.full((12, 2 * G), 5.0, device="cuda")
    for starts in ([0, 12, 0, 12, 12], [3, 12, -5, 1 << 30, 12]):
        sbg.cache_attention(q, cache, table, lens, row_starts=ints(starts), workspace=ws, out=out,
                            lse_out=lse)
        assert (out == 5).all() and (lse == 5).all() and not ws[:COUNTERS].any()


@gpu
def test_two_captured_calls_share_a_workspace():
    """Graphs of two shapes over one workspace, replayed in turn with eager calls between."""
    g = gen(28)
    cache = random_cache(g, 40, 2, 64)
    shapes = [(1, [900]), (20, [1500, 70]), (3, [64, 64, 200])]
    runs = []
    ws = sbg.make_cache_attention_workspace(40, 16, 2, 64)
    for n, lens in shapes:
        T = n * len(lens)
        table, q = tables(g, 40, lens), randn(g, T, 16, 64)
        out, lse, L = torch.empty_like(q), torch.empty(T, 16, device="cuda"), ints(lens)

        def call(q=q, table=table, L=L, out=out, lse=lse):
            sbg.cache_attention(q, cache, table, L, workspace=ws, out=out, lse_out=lse)

        call()
        want = (out.clone(), lse.clone())
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            call()
        runs.append((graph, call, out, lse, want))
    for i in range(12):
        graph, call, out, lse, want = runs[i % 3]
        out.fill_(3.0)
        graph.replay() if i % 4 else call()
        torch.cuda.synchronize()
        assert torch.equal(out, want[0]) and torch.equal(lse, want[1])


# ---------------------------------------------------------------------------------------------
# pages
# ---------------------------------------------------------------------------------------------
def fork_reference(table, lens, parents, reserve, held, P):
    """(table', lens', refs, missing, copies) in plain Python."""
    R, W = len(table), len(table[0])
    held = held or [0] * P
    rows, out_lens, on = [], [], []
    for r in range(R):
        p = r if parents is None else parents[r]
        go = 0 <= p < R
        n = min(max(lens[p], 0), W * PAGE) if go else 0
        on.append(go)
        out_lens.append(n)
        pages = [x if 0 <= x < P else -1 for x in table[p][:-(-n // PAGE)]] if go else []
        rows.append(pages)
    refs = [max(h, 0) for h in held]
    for pages in rows:
        for x in pages:
            if x >= 0:
                refs[x] += 1
    last = [rows[r][-1] if out_lens[r] % PAGE else -1 for r in range(R)]
    free = iter([p for p in range(P) if refs[p] == 0])
    missing, copies, count = 0, [], list(refs)
    for r in range(R):
        if last[r] >= 0:
            mates = [x for x in range(R) if last[x] == last[r]]
            if not (mates[0] == r and count[last[r]] == len(mates)):
                new = next(free, -1)
                refs[last[r]] -= 1
                rows[r][-1] = new
                if new < 0:
                    missing += 1
                else:
                    refs[new] += 1
                    copies.append((last[r], new))
        if on[r]:
            want = -(-(out_lens[r] + reserve) // PAGE)
            missing += max(0, want - W)
            for _ in range(min(want, W) - len(rows[r])):
                new = next(free, -1)
                rows[r].append(new)
                if new < 0:
                    missing += 1
                else:
                    refs[new] += 1
    return [x + [-1] * (W - len(x)) for x in rows], out_lens, refs, missing, copies


def page_case(seed, R, W, P, L, H, D, share=0.3):
    """A cache with drawn bytes, a table with shared beginnings, lengths, parents, held pages."""
    rng, g = random.Random(seed), gen(seed)
    cache = sbg.make_kv_cache(P, H, D, layers=L)
    for x in cache[:2]:
        x.copy_(torch.randint(-128, 128, x.shape, generator=g, dtype=torch.int8))
    for x in cache[2:]:
        x.copy_(torch.randn(x.shape, generator=g))
    ids = rng.sample(range(P), P)
    table, lens = [], []
    for r in range(R):
        n = rng.randint(0, W * PAGE)
        row = []
        if table and rng.random() < share:
            other = rng.randrange(r)
            whole = min(lens[other], n) // PAGE
            row = table[other][:rng.randint(0, whole)]
        while len(row) < -(-n // PAGE):
            if len(ids) < P // 3:
                n = len(row) * PAGE
                break
            row.append(ids.pop())
        table.append(row + [-1] * (W - len(row)))
        lens.append(n)
    parents = [rng.choice([-1, r, rng.randrange(R), 0]) for r in range(R)]
    held = [0] * P
    for p in ids[:3]:
        held[p] = 2
    return cache, table, lens, parents, held


def same_bytes(cache, before, copies):
    want = [x.clone() for x in before]
    for src, dst in copies:
        for x, y in zip(want, before):
            x[:, dst] = y[:, src]
    for x, y in zip(cache, want):
        assert torch.equal(x, y)


FORKS = [(1, 3, 2, 10, 1, 1, 16), (2, 8, 5, 40, 2, 2, 64), (3, 64, 9, 400, 3, 1, 48),
         (4, 5, 3, 6, 1, 3, 80), (5, 1, 1, 1, 1, 1, 16), (6, 130, 2, 300, 1, 1, 16),
         (7, 1500, 3, 9000, 1, 1, 16), (8, 33, 70, 5000, 1, 2, 16)]


@gpu
@pytest.mark.parametrize("case", FORKS, ids=lambda c: f"r{c[1]}_w{c[2]}_p{c[3]}")
@pytest.mark.parametrize("reserve", [0, 1, 130])
def test_fork_pages(case, reserve):
    seed, R, W, P, L, H, D = case
    cache, table, lens, parents, held = page_case(*case)
    ws = sbg.make_pages_workspace(R, W, P)
    for par, hold in ((parents, held), (None, None), ([-1] * R, held), ([R - 1] * R, None)):
        before = [x.clone() for x in cache]
        ws.fill_(0x5a)
        got = sbg.fork_pages(cache, ints(table), ints(lens), None if par is None else ints(par),
                             reserve=reserve, held=None if hold is None else ints(hold),
                             workspace=ws)
        t, n, refs, missing, copies = fork_reference(table, lens, par, reserve, hold, P)
        assert got[0].tolist() == t and got[1].tolist() == n and got[2].tolist() == refs
        assert got[3].item() == missing
        same_bytes(cache, before, copies)


@gpu
def test_fork_pages_of_a_single_layer_and_odd_tables():
    """One layer's cache; page numbers that are none, parents that are none, negative lengths and
    such past the table."""
    g = gen(31)
    P, W = 9, 3
    cache = random_cache(g, P, 2, 32, FP8)
    table = [[0, P, 1], [2, -5, 3], [4, 5, 6], [1 << 30, 7, -1]]
    lens, parents = [70, 180, 1000, -3], [1, 2, 2, 99]
    before = [x.clone() for x in cache]
    got = sbg.fork_pages(cache, ints(table), ints(lens), ints(parents), reserve=1,
                         workspace=sbg.make_pages_workspace(4, W, P))
    t, n, refs, missing, copies = fork_reference(table, lens, parents, 1, None, P)
    assert [x.tolist() for x in got] == [t, n, refs, [missing]]
    for src, dst in copies:
        for x, y in zip(cache, before):
            assert torch.equal(x[dst].view(torch.int8), y[src].view(torch.int8))


def compact_reference(table, held, P):
    held = held or [0] * P
    refs = [max(h, 0) for h in held]
    for row in table:
        for x in row:
            if 0 <= x < P:
                refs[x] += 1
    free = [p for p in range(P) if refs[p] == 0]
    high = [p for p in reversed(range(P)) if refs[p] > 0 and held[p] <= 0]
    moves = {s: d for d, s in zip(free, high) if d < s}
    for s, d in moves.items():
        refs[d], refs[s] = refs[s], 0
    out = [[moves.get(x, x) if 0 <= x < P else -1 for x in row] for row in table]
    return out, refs, [len(moves), max([p + 1 for p in range(P) if refs[p]], default=0)], moves


@gpu
@pytest.mark.parametrize("case", FORKS, ids=lambda c: f"r{c[1]}_w{c[2]}_p{c[3]}")
def test_compact_pages(case):
    seed, R, W, P, L, H, D = case
    cache, table, lens, parents, held = page_case(*case)
    ws = sbg.make_pages_workspace(R, W, P)
    for hold in (held, None, [1] * P):
        before = [x.clone() for x in cache]
        ws.fill_(0x5a)
        got = sbg.compact_pages(cache, ints(table), held=None if hold is None else ints(hold),
                                workspace=ws)
        t, refs, counts, moves = compact_reference(table, hold, P)
        assert got[0].tolist() == t and got[1].tolist() == refs and got[2].tolist() == counts
        same_bytes(cache, before, list(moves.items()))


# ---------------------------------------------------------------------------------------------
# together, on streams, in graphs
# ---------------------------------------------------------------------------------------------
class Step:
    """The attention part of a decode step for a few sequences, as a server calls it."""

    def __init__(self, kind=torch.int8, B=5, Hq=8, H=2, D=64, layers=2):
        g = gen(41, str(kind))
        self.B, self.layers = B, layers
        self.W, self.P = 8, 60
        self.cache = sbg.make_kv_cache(self.P, H, D, layers=layers, dtype=kind)
        self.qkv = randn(g, layers, B, (Hq + 2 * H) * D)
        self.split = [(x[:, :Hq * D].view(B, Hq, D), x[:, Hq * D:(Hq + H) * D].view(B, H, D),
                       x[:, (Hq + H) * D:].view(B, H, D)) for x in self.qkv]
        self.freqs = sbg.rotary_frequencies(D)
        self.table = torch.full((B, self.W), -1, dtype=I32, device="cuda")
        self.lens = torch.zeros(B, dtype=I32, device="cuda")
        self.parents = ints(list(range(B)))
        self.spare = (torch.empty_like(self.table), torch.empty_like(self.lens),
                      torch.empty(self.P, dtype=I32, device="cuda"), ints([0]))
        self.ws = sbg.make_cache_attention_workspace(B, Hq, H, D)
        self.pages_ws = sbg.make_pages_workspace(B, self.W, self.P)
        self.out = torch.empty(layers, B, Hq, D, dtype=BF16, device="cuda")
        self.qr, self.kr = (torch.empty(B, n, D, dtype=BF16, device="cuda") for n in (Hq, H))

    def __call__(self, stream=None):
        kw = {} if stream is None else {"stream": stream}
        sbg.fork_pages(self.cache, self.table, self.lens, self.parents, reserve=1,
                       workspace=self.pages_ws, outs=self.spare, **kw)
        with torch.cuda.stream(stream or torch.cuda.current_stream()):
            self.table.copy_(self.spare[0])
            torch.add(self.spare[1], 1, out=self.lens)
            pos = self.lens - 1
        for i, (q, k, v) in enumerate(self.split):
            layer = self.cache.layer(i)
            sbg.rotary(q, k, pos, self.freqs, q_out=self.qr, k_out=self.kr, **kw)
            sbg.cache_append(self.kr, v, layer, self.table, self.lens, **kw)
            sbg.cache_attention(self.qr, layer, self.table, self.lens, workspace=self.ws,
                                out=self.out[i], **kw)

    def state(self):
        return [x.view(torch.int8).clone() if x.element_size() == 1 else x.clone()
                for x in (*self.cache, self.table, self.lens, self.out)]


def drive(step, run, steps=70, seed=3):
    """Steps with changing inputs and parents; the state after each."""
    g = gen(seed)
    states = []
    for i in range(steps):
        step.qkv.copy_(randn(g, *step.qkv.shape))
        step.parents.copy_(torch.randint(0, step.B, (step.B,), generator=g).int()
                           if i % 9 == 8 else torch.arange(step.B).int())
        run()
        states.append(step.state())
    return states


@gpu
@pytest.mark.parametrize("kind", [torch.int8, FP8])
def test_a_step_eager_on_a_stream_and_captured(kind):
    """The operators together: the last step against 64 bits, and the same bits on another
    stream and replayed from a graph, while lengths, tables and parents change."""
    eager = Step(kind)
    want = drive(eager, eager)
    assert eager.spare[3].item() == 0 and eager.lens.tolist() == [70] * eager.B
    last = eager.cache.layer(eager.layers - 1)
    check_attention(eager.qr, last, eager.table, [70] * eager.B, list(range(eager.B + 1)), rs=None)

    side = Step(kind)
    s = torch.cuda.Stream()

    def on_side():
        s.wait_stream(torch.cuda.current_stream())
        side(s)
        torch.cuda.current_stream().wait_stream(s)

    for a, b in zip(drive(side, on_side), want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))

    graphed = Step(kind)
    graphed()          # first use outside a capture
    fresh = Step(kind)
    for x, y in zip((*graphed.cache, graphed.table, graphed.lens),
                    (*fresh.cache, fresh.table, fresh.lens)):
        x.copy_(y)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        graphed()

    def replay():
        graph.replay()
        torch.cuda.synchronize()

    for a, b in zip(drive(graphed, replay), want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


@gpu
def test_forked_sequences_go_their_own_ways():
    """Two rows from one parent: each appends to its own copy, the parent's pages stay."""
    g = gen(42)
    H, D, P = 1, 32, 12
    cache = random_cache(g, P, H, D)
    table, lens = ints([[5, 6], [-1, -1]]), ints([100, 0])
    lk = logical(cache)[0]
    t, n, refs, missing = sbg.fork_pages(cache, table, lens, ints([0, 0]), reserve=1,
                                         workspace=sbg.make_pages_workspace(2, 2, P))
    assert t.tolist() == [[5, 6], [5, 0]] and n.tolist() == [100, 100] and missing.item() == 0
    k = randn(g, 2, H, D, std=0.1)
    sbg.cache_append(k, k, cache, t, n + 1)
    a, b = logical(cache)[0][6], logical(cache)[0][0]
    assert torch.equal(a[:36], lk[6][:36]) and torch.equal(b[:36], lk[6][:36])
    assert not torch.equal(a[36], b[36])


# ---------------------------------------------------------------------------------------------
# refusals (no GPU needed: the C ABI refuses before it touches one)
# ---------------------------------------------------------------------------------------------
def test_tensors_off_the_gpu_are_refused():
    c = sbg.make_kv_cache(2, 1, 16, device="cpu")
    x = torch.zeros(1, 1, 16, dtype=BF16)
    t, n = ints([[0]], "cpu"), ints([1], "cpu")
    for f in (lambda: sbg.rotary(x, x, n, torch.ones(8, dtype=F64)),
              lambda: sbg.cache_append(x, x, c, t, n),
              lambda: sbg.cache_read(c, t, n),
              lambda: sbg.cache_attention(x, c, t, n, workspace=None),
              lambda: sbg.fork_pages(c, t, n, workspace=None),
              lambda: sbg.compact_pages(c, t, workspace=None)):
        with pytest.raises(ValueError, match="GPU"):
            f()
    with pytest.raises(ValueError):
        sbg.make_kv_cache(2, 1, 24, device="cpu")
    with pytest.raises(ValueError):
        sbg.make_kv_cache(2, 1, 272, device="cpu")
    with pytest.raises(TypeError):
        sbg.make_kv_cache(2, 1, 16, dtype=BF16, device="cpu")
    with pytest.raises(ValueError):
        sbg.rotary(x, x, n, torch.ones(8, dtype=F64), layout="quarter")
    assert c.layer is not None and sbg.make_kv_cache(2, 1, 16, layers=3, device="cpu").layer(
        1).k.shape == (2, 1, 1, 64, 16)


@gpu
def test_tensors_that_do_not_fit_are_refused():
    H, D = 2, 32
    c = sbg.make_kv_cache(4, H, D)
    many = sbg.make_kv_cache(4, H, D, layers=2)
    k = torch.zeros(3, H, D, dtype=BF16, device="cuda")
    q = torch.zeros(3, 4, D, dtype=BF16, device="cuda")
    t, n = ints([[0], [1], [2]]), ints([1, 1, 1])
    ws = sbg.make_cache_attention_workspace(3, 4, H, D)
    pws = sbg.make_pages_workspace(3, 1, 4)
    freqs = sbg.rotary_frequencies(D)
    pos = ints([0, 1, 2])
    V, T, E = ValueError, TypeError, sbg.LowmError
    bad = [
        (V, lambda: sbg.cache_append(k, k[:2], c, t, n)),
        (V, lambda: sbg.cache_append(k, k[..., :16], c, t, n)),
        (T, lambda: sbg.cache_append(k, k.float(), c, t, n)),
        (T, lambda: sbg.cache_append(k.half(), k.half(), c, t, n)),
        (T, lambda: sbg.cache_append(k, k, c, t.long(), n)),
        (V, lambda: sbg.cache_append(k, k, c, t, n[:2])),
        (V, lambda: sbg.cache_append(k[:2], k[:2], c, t, n)),
        (V, lambda: sbg.cache_append(k, k, c, t, n, row_starts=ints([0, 1, 2]))),
        (V, lambda: sbg.cache_append(k, k, many, t, n)),
        (V, lambda: sbg.cache_append(k, k, c._replace(v=c.k), t, n)),
        (T, lambda: sbg.cache_append(k, k, c._replace(v=c.v.view(FP8)), t, n)),
        (V, lambda: sbg.cache_append(k.transpose(1, 2), k, c, t, n)),
        (E, lambda: sbg.cache_append(k[:1].expand(3, H, D), k, c, t, n)),
        (V, lambda: sbg.cache_attention(q, c, t, n, workspace=None)),
        (V, lambda: sbg.cache_attention(q[..., :16], c, t, n, workspace=ws)),
        (T, lambda: sbg.cache_attention(q.float(), c, t, n, workspace=ws)),
        (E, lambda: sbg.cache_attention(q, c, t, n, workspace=ws[:1000])),
        (E, lambda: sbg.cache_attention(q, c, t, n, workspace=ws[16:])),
        (E, lambda: sbg.cache_attention(q[:, :3].contiguous(), c, t, n, workspace=ws)),
        (E, lambda: sbg.cache_attention(q, c, t, n, workspace=ws, window=-1)),
        (E, lambda: sbg.cache_attention(q, c, t, n, workspace=ws, out=q)),
        (V, lambda: sbg.cache_attention(q, c, t, n, workspace=ws, lse_out=pos.float())),
        (E, lambda: sbg.rotary(q, q, pos, freqs, q_out=k.new_empty(3, 4, D), k_out=q,
                               first=1)),
        (V, lambda: sbg.rotary(q, k[:2], pos, freqs)),
        (T, lambda: sbg.rotary(q, k, pos, freqs.float())),
        (T, lambda: sbg.rotary(q, k, pos.float(), freqs)),
        (V, lambda: sbg.rotary(q, k, pos[:2], freqs)),
        (E, lambda: sbg.rotary(q, q, pos, freqs, q_out=q.clone()[:, :, :], k_out=q[:, :, :],
                               first=2)),
        (E, lambda: sbg.rotary(q, None, pos, sbg.rotary_frequencies(D + 2))),
        (T, lambda: sbg.fork_pages(c, t, n.long(), workspace=pws)),
        (V, lambda: sbg.fork_pages(c, t, n, ints([0]), workspace=pws)),
        (V, lambda: sbg.fork_pages(c, t, n, held=ints([0]), workspace=pws)),
        (V, lambda: sbg.fork_pages(c, t, n, workspace=None)),
        (E, lambda: sbg.fork_pages(c, t, n, reserve=-1, workspace=pws)),
        (E, lambda: sbg.fork_pages(c, t, n, workspace=pws[:96])),
        (E, lambda: sbg.fork_pages(c, t, n, workspace=pws,
                                   outs=(t, ints([0] * 3), ints([0] * 4), ints([0])))),
        (E, lambda: sbg.compact_pages(c, t, workspace=pws[:4])),
        (V, lambda: sbg.compact_pages(c, t[0], workspace=pws)),
        (E, lambda: sbg.compact_pages(c, t, workspace=pws, outs=(t, ints([0] * 4), ints([0] * 2)))),
    ]
    for i, (kind, f) in enumerate(bad):
        with pytest.raises(kind):
            f()
            pytest.fail(f"call {i} was not refused")


def test_c_abi_refuses():
    """The checks of the C ABI itself, with addresses that are never followed."""
    import ctypes as ct

    lib = cache_ops.library().lib
    INVALID, UNSUPPORTED, WORKSPACE = -1, -2, -3
    at = lambda i: (1 << 40) + (i << 32)  # noqa: E731

    def cache(**kw):
        return cache_ops.KvCacheArg(**{**dict(k=at(0), v=at(1), k_scale=at(2), v_scale=at(3), P=4, H=2, D=64,
                               type=2, layers=1), **kw})

    def seq(**kw):
        return cache_ops.SequencesArg(**{**dict(table=at(4), lens=at(5), row_starts=None, table_ld=3, B=2, W=3,
                                   T=2), **kw})

    def append(c=None, s=None, **kw):
        a = cache_ops.CacheAppendArgs(cache=c or cache(), seq=s or seq(),
                   **{**dict(k=at(6), v=at(7), k_row=128, k_head=64, v_row=128, v_head=64, type=0),
                      **kw})
        return lib.lowm_cache_append(ct.byref(a), None)

    assert append(s=seq(T=0)) == 0
    for want, got in [
        (INVALID, append(c=cache(P=0))), (INVALID, append(c=cache(type=0))),
        (INVALID, append(c=cache(layers=2))), (INVALID, append(c=cache(k=None))),
        (UNSUPPORTED, append(c=cache(D=72))), (UNSUPPORTED, append(c=cache(D=272))),
        (UNSUPPORTED, append(c=cache(H=1025))), (UNSUPPORTED, append(c=cache(k=at(0) + 8))),
        (UNSUPPORTED, append(c=cache(k_scale=at(2) + 2))),
        (INVALID, append(c=cache(v=at(0) + 16))), (INVALID, append(c=cache(k_scale=at(5)))),
        (INVALID, append(s=seq(T=-1))), (INVALID, append(s=seq(T=3))),
        (INVALID, append(s=seq(table_ld=2))), (INVALID, append(s=seq(lens=None))),
        (UNSUPPORTED, append(s=seq(B=65537, T=65537))), (UNSUPPORTED, append(s=seq(W=65537))),
        (INVALID, append(k=None)), (INVALID, append(type=3)), (UNSUPPORTED, append(k=at(6) + 1)),
        (INVALID, append(k_row=64)), (INVALID, append(k_head=63)), (INVALID, append(v_row=-1)),
        (INVALID, append(k=at(0))), (INVALID, lib.lowm_cache_append(None, None)),
        (INVALID, lib.lowm_cache_read(None, None)),
    ]:
        assert got == want

    size = lib.lowm_cache_attention_workspace_bytes

    def attend(c=None, s=None, **kw):
        a = cache_ops.CacheAttentionArgs(cache=c or cache(), seq=s or seq(),
                      **{**dict(q=at(6), out=at(7), lse=at(8), workspace=at(9),
                                workspace_bytes=size(2, 8, 2, 64), q_row=512, q_head=64, Hq=8, window=0,
                                scale=1.0), **kw})
        return lib.lowm_cache_attention(ct.byref(a), None)

    assert size(2, 8, 2, 64) > 0 and size(0, 8, 2, 64) == size(2, 8, 3, 64) == 0
    assert size(2, 8, 2, 72) == size(2, 8, 2, 272) == size(2, 2048, 2, 64) == size(1 << 24, 256, 2, 64) == 0
    for want, got in [
        (INVALID, attend(Hq=7)), (INVALID, attend(Hq=0)), (INVALID, attend(window=-1)),
        (INVALID, attend(q=None)), (INVALID, attend(out=None)), (UNSUPPORTED, attend(q=at(6) + 2)),
        (UNSUPPORTED, attend(out=at(7) + 8)), (UNSUPPORTED, attend(lse=at(8) + 1)),
        (UNSUPPORTED, attend(q_head=68)), (INVALID, attend(q_row=64)),
        (WORKSPACE, attend(workspace=None)), (WORKSPACE, attend(workspace_bytes=size(2, 8, 2, 64) - 1)),
        (UNSUPPORTED, attend(workspace=at(9) + 128)), (INVALID, attend(out=at(6))),
        (INVALID, attend(lse=at(7))), (INVALID, attend(workspace=at(0))),
        (INVALID, attend(out=at(4))), (UNSUPPORTED, attend(Hq=2048, q_row=2048 * 64)),
        (INVALID, attend(c=cache(layers=3))), (INVALID, lib.lowm_cache_attention(None, None)),
        (UNSUPPORTED, attend(s=seq(T=1 << 20, B=1, W=65536, table_ld=65536),
                             workspace_bytes=size(1 << 20, 8, 2, 64), workspace=at(12))),
    ]:
        assert got == want

    def rotary(**kw):
        a = cache_ops.RotaryArgs(**{**dict(q=at(0), k=at(1), q_out=at(2), k_out=at(3), positions=at(4),
                             freqs=at(5), q_row=256, q_head=64, k_row=64, k_head=64,
                             q_out_row=256, q_out_head=64, k_out_row=64, k_out_head=64, T=2, Hq=4,
                             Hk=1, D=64, R=64, first=0, type=0, positions_bytes=8, flags=0,
                             scale=1.0), **kw})
        return lib.lowm_rotary(ct.byref(a), None)

    assert rotary(T=0) == 0
    for want, got in [
        (INVALID, rotary(T=-1)), (INVALID, rotary(R=63)), (INVALID, rotary(R=0)),
        (INVALID, rotary(first=2)), (INVALID, rotary(first=-1)), (INVALID, rotary(R=66)),
        (INVALID, rotary(Hk=0)), (INVALID, rotary(type=2)), (INVALID, rotary(flags=4)),
        (INVALID, rotary(positions_bytes=2)), (INVALID, rotary(q=None)),
        (INVALID, rotary(k_out=None)), (INVALID, rotary(freqs=None)),
        (UNSUPPORTED, rotary(D=1025)), (UNSUPPORTED, rotary(Hq=1025)),
        (UNSUPPORTED, rotary(q=at(0) + 1)), (UNSUPPORTED, rotary(freqs=at(5) + 4)),
        (UNSUPPORTED, rotary(positions=at(4) + 4)), (INVALID, rotary(q_out_row=64)),
        (INVALID, rotary(q_out=at(0) + 64)), (INVALID, rotary(k_out=at(0))),
        (INVALID, rotary(k_out=at(2))), (INVALID, rotary(q_out=at(4))),
        (INVALID, lib.lowm_rotary(None, None)),
    ]:
        assert got == want

    room = lib.lowm_pages_workspace_bytes

    def fork(c=None, **kw):
        a = cache_ops.ForkPagesArgs(cache=c or cache(layers=3),
                 **{**dict(table=at(4), lens=at(5), parents=None, held=None, table_out=at(6),
                           lens_out=at(7), refs_out=at(8), missing_out=at(9), workspace=at(10),
                           workspace_bytes=room(4, 3, 4), R=4, W=3, reserve=1), **kw})
        return lib.lowm_fork_pages(ct.byref(a), None)

    assert room(0, 1, 1) == room(1, 0, 1) == room(1, 1, 0) == room(4097, 1, 1) == 0
    for want, got in [
        (INVALID, fork(R=0)), (INVALID, fork(W=0)), (INVALID, fork(reserve=-1)),
        (INVALID, fork(table=None)), (INVALID, fork(lens_out=None)), (INVALID, fork(refs_out=None)),
        (UNSUPPORTED, fork(R=4097)), (UNSUPPORTED, fork(W=65537)),
        (UNSUPPORTED, fork(c=cache(P=(1 << 24) + 1))), (UNSUPPORTED, fork(held=at(11) + 2)),
        (UNSUPPORTED, fork(reserve=65536 * 64 + 1)), (WORKSPACE, fork(workspace=None)),
        (WORKSPACE, fork(workspace_bytes=room(4, 3, 4) - 1)), (UNSUPPORTED, fork(workspace=at(10) + 4)),
        (INVALID, fork(table_out=at(4))), (INVALID, fork(lens_out=at(5))),
        (INVALID, fork(refs_out=at(6))), (INVALID, fork(missing_out=at(0))),
        (INVALID, fork(table=at(1))), (INVALID, fork(held=at(8))),
        (INVALID, lib.lowm_fork_pages(None, None)), (INVALID, lib.lowm_compact_pages(None, None)),
    ]:
        assert got == want
