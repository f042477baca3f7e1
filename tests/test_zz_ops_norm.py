"""residual_norm and quantize_rows against their formulas in 64 bits.

Tolerances, with u = 2^-24: a sum of squares in the kernel adds at most 16
terms in a lane, 6 levels in a wavefront and 16 wavefronts, 38 roundings, so a
root mean square is off by at most 19 u, and the divide, square root and the
three or four products add less than 13 u more: 32 u in all for each norm.
Every output is then rounded once, by half a step of its type.
"""
from __future__ import annotations

import ctypes

import pytest
import torch

import split_bf16_gemm_amd as sbg
from split_bf16_gemm_amd import ops

U = 2.0 ** -24
NORM = 32 * U
HALF = {torch.bfloat16: 2.0 ** -8, torch.float32: U}
BF16, F32 = torch.bfloat16, torch.float32


def unit(v, center, eps):
    """(normalised, 1/rms, bound of its absolute error in fp32)."""
    mean_err = 0.0
    if center:
        mean = v.mean(-1, keepdim=True)
        mean_err = 40 * U * v.abs().mean(-1, keepdim=True) + U * v.abs()
        v = v - mean
    k = 1 / torch.sqrt((v * v).mean(-1, keepdim=True) + eps)
    n = v * k
    # an error e in the elements moves the root mean square by at most e
    return n, k, NORM * n.abs() + k * mean_err * (1 + n.abs())


def reference(y, r, post, w_post, w_pre, gate, b, a, eps, center):
    y, r = y.double(), r.double()
    p, perr = y, torch.zeros_like(y)
    if post:
        p, _, perr = unit(y, center, eps)
    g = torch.ones_like(y)
    if w_post is not None:
        g = g * w_post.double()
    if gate is not None:
        g = g * gate.double()
    branch = b * g * p
    r2 = a * r + branch
    r2_err = 6 * U * (a * r).abs() + 6 * U * branch.abs() + (b * g).abs() * perr
    x, k, xerr = unit(r2, center, eps)
    worst = r2_err.amax(-1, keepdim=True)
    xerr = xerr + k * (r2_err + worst * (1 + x.abs()))
    if w_pre is not None:
        x, xerr = x * w_pre.double(), (xerr + 2 * U * x.abs()) * w_pre.double().abs()
    return r2, r2_err, x, xerr


def rand(g, *shape, dtype=BF16, std=1.0, dev="cpu"):
    return (torch.randn(*shape, generator=g, dtype=F32) * std).to(dtype).to(dev)


def check_type(got, want, err):
    bound = err + (want.abs() + err) * HALF[got.dtype]
    diff = (got.double().cpu() - want).abs()
    assert (diff <= bound).all(), (diff / bound).max()


def check_i8(q, s, x, err):
    s = s.double().cpu()[:, None]
    top = x.abs().amax(-1, keepdim=True)
    worst = err.amax(-1, keepdim=True)
    assert ((s - top / 127).abs() <= worst / 127 + 2 * U * top).all()
    q = q.double().cpu()
    assert q.abs().max() <= 127
    assert ((q * s - x).abs() <= 0.5 * s * (1 + 300 * U) + err + worst).all()


CASES = [
    # M, D, y, residual, weights, gate kind, gate type, center, post, int8, in place
    (1, 4096, BF16, BF16, BF16, None, BF16, False, True, False, False),
    (3, 1, BF16, F32, BF16, None, BF16, False, True, False, False),
    (5, 7, BF16, BF16, F32, "channel", BF16, False, True, True, False),
    (4, 64, F32, F32, F32, "token", F32, True, True, False, True),
    (9, 512, BF16, BF16, BF16, "element", BF16, False, True, True, True),
    (9, 520, BF16, F32, BF16, "element", F32, True, False, False, False),
    (2, 2047, F32, BF16, BF16, "channel", BF16, True, True, True, False),
    (70, 2048, BF16, BF16, None, "token", BF16, False, True, False, False),
    (6, 4096, F32, F32, BF16, "channel", F32, False, False, True, True),
    (3, 4104, BF16, BF16, BF16, None, BF16, False, True, True, False),
    (2, 8191, BF16, F32, F32, "element", BF16, True, True, False, False),
    (2, 8192, BF16, BF16, BF16, "channel", BF16, False, True, False, False),
    (3, 16384, BF16, F32, BF16, "element", BF16, True, True, True, False),
    (2, 16383, BF16, BF16, BF16, "token", F32, False, True, False, True),
    (6, 9, F32, BF16, F32, "element", BF16, True, True, True, False),
    (7, 8, BF16, F32, BF16, "channel", BF16, False, True, True, True),
    (5, 511, BF16, BF16, BF16, "element", F32, True, True, True, False),
    (3, 4095, F32, F32, F32, "element", F32, False, True, False, True),
    (3, 4097, BF16, BF16, BF16, "channel", BF16, True, True, True, False),
    (2, 8193, BF16, F32, BF16, "element", BF16, False, True, True, True),
]


@pytest.mark.gpu
@pytest.mark.parametrize("case", CASES, ids=lambda c: f"m{c[0]}_d{c[1]}")
@pytest.mark.parametrize("pad", [0, 8, 3], ids=["dense", "pad8", "pad3"])
def test_residual_norm(case, pad):
    M, D, yt, rt, wt, gk, gt, center, post, i8, inplace = case
    g = torch.Generator().manual_seed(M * 100003 + D + pad)
    dev = "cuda"

    def rows(dtype, std):
        wide = rand(g, M, D + pad, dtype=dtype, std=std, dev=dev)
        return wide[:, :D]

    y, r = rows(yt, 1.5), rows(rt, 3.0)
    w0 = None if wt is None else rand(g, D, dtype=wt, dev=dev)
    w1 = None if wt is None else rand(g, D, dtype=wt, dev=dev)
    gate = {None: None, "channel": (D,), "token": (M, 1), "element": (M, D)}[gk]
    gate = None if gate is None else rand(g, *gate, dtype=gt, std=0.5, dev=dev)
    a, b, eps = 0.875, 1.25, 1e-5
    r2, r2_err, x, xerr = reference(*(t if t is None else t.cpu() for t in (y, r)), post,
                                    *(t.cpu() if t is not None and use else None
                                      for t, use in ((w0, post), (w1, True), (gate, True))),
                                    b, a, eps, center)
    wide_r, wide_x = (torch.full((M, D + pad), 77, dtype=t, device=dev)
                      for t in (rt, torch.int8 if i8 else BF16))
    r_out = r if inplace else wide_r[:, :D]
    got_r, got_x, s = sbg.residual_norm(
        y, r, post_norm=post, post_weight=w0, pre_weight=w1, gate=gate, residual_scale=a,
        branch_scale=b, eps=eps, center=center, quantize=i8, residual_out=r_out,
        out=wide_x[:, :D])
    torch.cuda.synchronize()
    assert got_r.data_ptr() == r_out.data_ptr() and (s is not None) == i8
    check_type(got_r, r2, r2_err)
    if i8:
        check_i8(got_x, s, x, xerr)
    else:
        check_type(got_x, x, xerr)
    # nothing past the rows is written
    assert (wide_x[:, D:] == 77).all() and (inplace or (wide_r[:, D:] == 77).all())


@pytest.mark.gpu
def test_residual_norm_without_the_second_norm():
    g = torch.Generator().manual_seed(3)
    y, r = rand(g, 4, 96, dev="cuda"), rand(g, 4, 96, dev="cuda")
    out, x, s = sbg.residual_norm(y, r, pre_norm=False, post_norm=False)
    assert x is None and s is None
    assert torch.equal(out, (y.float() + r.float()).to(BF16))


@pytest.mark.gpu
def test_rows_do_not_depend_on_their_batch():
    """A row alone, in a batch, and run twice: the same bits."""
    g = torch.Generator().manual_seed(4)
    y, r = rand(g, 37, 2048, dev="cuda"), rand(g, 37, 2048, dev="cuda")
    many = sbg.residual_norm(y, r, quantize=True)
    again = sbg.residual_norm(y, r, quantize=True)
    for i in (0, 17, 36):
        one = sbg.residual_norm(y[i:i + 1], r[i:i + 1], quantize=True)
        for o, m, n in zip(one, many, again):
            assert torch.equal(o[0], m[i]) and torch.equal(m[i], n[i])


@pytest.mark.gpu
@pytest.mark.parametrize("i8", [False, True])
def test_rows_of_zeros_infinities_and_nans(i8):
    y = torch.zeros(4, 300, dtype=BF16, device="cuda")
    r = torch.ones(4, 300, dtype=BF16, device="cuda")
    r[0] = 0
    r[2, 5] = float("inf")
    r[3, 299] = float("nan")
    out, x, s = sbg.residual_norm(y, r, eps=1e-6, quantize=i8)
    torch.cuda.synchronize()
    assert torch.equal(out[:2], r[:2]) and out[2, 5] == float("inf") and out[3, 299].isnan()
    if i8:
        assert s[0] == 0 and (x[0] == 0).all()
        assert (x[1] == 127).all()
        assert s[2:].isnan().all() and (x[2:] == 0).all()
    else:
        assert (x[0] == 0).all()
        assert (x[1].float() == 1).all()
        assert x[2, 5].isnan() and (x[2, :5] == 0).all() and x[3].isnan().all()


@pytest.mark.gpu
@pytest.mark.parametrize("M,K", [(1, 1), (3, 17), (64, 4096), (5, 8200), (2, 32768), (7, 30001),
                                 (4, 8), (4, 7), (5, 9), (3, 513), (2, 16391)])
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_quantize_rows_is_the_formula_exactly(M, K, dtype):
    """fp32 divides are correctly rounded on both sides: the same bits."""
    g = torch.Generator().manual_seed(M + K)
    x = rand(g, M, K, dtype=dtype, std=2.0, dev="cuda")
    q, s = sbg.quantize_rows(x)
    want_s = x.cpu().float().abs().amax(-1) / 127
    want_q = torch.round(x.cpu().float() / want_s[:, None]).to(torch.int8)
    assert torch.equal(s.cpu(), want_s) and torch.equal(q.cpu(), want_q)
    assert q.abs().max() == 127


@pytest.mark.gpu
def test_quantize_rows_strided_tiny_and_non_finite_rows():
    wide = torch.zeros(6, 40, device="cuda")
    x = wide[:, 3:36]
    x[0] = 1e-43          # the scale falls among the subnormals
    x[1, 4], x[2, 0], x[3, 32] = float("inf"), float("nan"), -float("inf")
    x[4, 32] = -5
    q, s = sbg.quantize_rows(x)
    assert s[1:4].isnan().all() and (q[1:4] == 0).all()
    assert s[5] == 0 and (q[5] == 0).all()
    assert q[4, 32] == -127 and (q[4, :32] == 0).all()
    assert (q[0] <= 127).all() and (q[0] >= 0).all()


@pytest.mark.gpu
def test_on_another_stream_and_in_a_graph():
    g = torch.Generator().manual_seed(8)
    y, r = rand(g, 5, 1000, dev="cuda"), rand(g, 5, 1000, dev="cuda")
    want = sbg.residual_norm(y, r, quantize=True)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    got = sbg.residual_norm(y, r, quantize=True, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    bufs = [torch.zeros_like(t) for t in want]
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        sbg.residual_norm(y, r, quantize=True, residual_out=bufs[0], out=bufs[1],
                          scale_out=bufs[2])
    for i in range(3):
        y.copy_(rand(g, 5, 1000, dev="cuda"))
        want = sbg.residual_norm(y, r, quantize=True)
        for b in bufs:
            b.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(bufs, want))


@pytest.mark.gpu
@pytest.mark.parametrize("D", [64, 100])
def test_operands_that_are_columns_of_one_tensor(D):
    """Column ranges of one tensor share no element though their spans of memory meet."""
    g = torch.Generator().manual_seed(D)
    y, r = rand(g, 6, D, dev="cuda"), rand(g, 6, D, dev="cuda")
    want_r, want_x, _ = sbg.residual_norm(y, r)
    for order in ((0, 1, 2, 3), (3, 2, 1, 0), (1, 3, 0, 2)):
        wide = torch.full((6, 4 * D), 5.0, dtype=BF16, device="cuda")
        at = [wide[:, i * D:(i + 1) * D] for i in order]
        at[0].copy_(y)
        at[1].copy_(r)
        sbg.residual_norm(at[0], at[1], residual_out=at[2], out=at[3])
        assert torch.equal(at[2], want_r) and torch.equal(at[3], want_x)
        assert torch.equal(at[0], y) and torch.equal(at[1], r)
    wide = torch.zeros(6, 4 * D, dtype=BF16, device="cuda")
    a, b, c = wide[:, :D], wide[:, D:2 * D], wide[:, 2 * D:3 * D]
    for o in (wide[:, 3 * D - 1:4 * D - 1], wide[:, D - 1:2 * D - 1], wide[:, 1:D + 1]):
        with pytest.raises(sbg.LowmError):         # one shared column is an overlap
            sbg.residual_norm(a, b, residual_out=c, out=o)


@pytest.mark.gpu
def test_more_rows_than_one_launch_holds():
    """2^26 rows of 64 lanes each: every row has the values of its period's row.  (Copies and
    comparisons by slices: torch's gather of as many rows leaves most of them zero.)"""
    periods, period, D = 2 ** 15, 2 ** 11 + 3, 8
    g = torch.Generator().manual_seed(12)
    base = [rand(g, period, D, dev="cuda") for _ in range(2)]
    y, r = (b.expand(periods, period, D).reshape(-1, D) for b in base)
    assert len(y) > 2 ** 26

    def same(many, few):
        many = many.view(periods, *few.shape)
        return all((many[i:i + 1024] == few).all() for i in range(0, periods, 1024))

    assert same(y, base[0]) and same(r, base[1])
    for got, few in ((sbg.quantize_rows(y), sbg.quantize_rows(base[0])),
                     (sbg.residual_norm(y, r)[:2], sbg.residual_norm(*base)[:2])):
        assert all(same(*p) for p in zip(got, few))


@pytest.mark.gpu
def test_no_rows_at_all():
    y = torch.zeros(0, 64, dtype=BF16, device="cuda")
    r, x, s = sbg.residual_norm(y, y, quantize=True)
    assert r.shape == x.shape == (0, 64) and s.shape == (0,)
    assert sbg.quantize_rows(y)[0].shape == (0, 64)
    lp = sbg.token_logprobs(y, torch.zeros(0, dtype=torch.int64, device="cuda"), 3)
    assert lp[0].shape == (0,) and lp[3].shape == (0, 3)


@pytest.mark.gpu
def test_tensors_that_do_not_fit_are_refused():
    y, w = torch.zeros(4, 64, dtype=BF16, device="cuda"), torch.ones(64, device="cuda")
    for kw, error in ((dict(post_weight=w[:32]), ValueError), (dict(post_weight=w.double()), TypeError),
                      (dict(post_weight=w, pre_weight=w.to(BF16)), TypeError),
                      (dict(gate=w[:5]), ValueError), (dict(gate=y.t()[:4]), ValueError),
                      (dict(out=y.float()), TypeError), (dict(out=y[:2]), ValueError),
                      (dict(residual_out=y.float()), TypeError), (dict(post_weight=7), TypeError),
                      (dict(quantize=True, pre_norm=False), ValueError),
                      (dict(residual_out=y), sbg.LowmError)):     # an output over an input
        with pytest.raises(error):
            sbg.residual_norm(y, y.clone(), **kw)
    for a in ((y.t(), y.t()), (y.expand(2, 4, 64)[0], y[0]), (y.half(), y)):
        with pytest.raises((ValueError, TypeError)):
            sbg.residual_norm(*a)


# -- refusals: no kernel is launched, no pointer is read -----------------------------------------
A0, B0, C0, D0 = 0x1000000, 0x2000000, 0x3000000, 0x4000000


def args(**kw):
    base = dict(y=A0, r=B0, r_out=C0, x=D0, ld_y=64, ld_r=64, ld_r_out=64, ld_x=64, M=4, D=64,
                residual_scale=1.0, branch_scale=1.0, eps=1e-6)
    base.update(kw)
    return ops.ResidualNormArgs(**base)


def call(**kw):
    return ops.library().lib.lowm_residual_norm(ctypes.byref(args(**kw)), None)


@pytest.mark.parametrize("kw", [
    dict(y=None), dict(r=None), dict(r_out=None), dict(x=None), dict(M=-1), dict(D=0),
    dict(ld_y=63), dict(ld_r=63), dict(ld_r_out=63), dict(ld_x=63), dict(flags=8),
    dict(y_type=2), dict(r_type=3), dict(w_type=-1), dict(gate_type=2), dict(x_type=1),
    dict(x_type=2), dict(gate=0x5000000, gate_col=2), dict(gate=0x5000000, gate_row=-1),
    dict(r_out=A0), dict(x=B0), dict(x=C0), dict(r_out=B0 + 2), dict(x_type=2, x_scale=D0),
    dict(w_post=D0 + 8), dict(gate=C0, gate_col=1)])
def test_residual_norm_refuses(kw):
    assert call(**kw) == sbg.binding.LOWM_ERR_INVALID_ARG


@pytest.mark.parametrize("kw", [
    dict(D=16385, ld_y=16385, ld_r=16385, ld_r_out=16385, ld_x=16385), dict(y=A0 + 1),
    dict(r=B0 + 2, r_type=1), dict(w_post=0x5000002, w_type=1), dict(x_type=2, x_scale=0x5000002)])
def test_residual_norm_does_not_support(kw):
    assert call(**kw) == sbg.binding.LOWM_ERR_UNSUPPORTED


@pytest.mark.parametrize("kw", [
    dict(x=A0 + 2 * 63), dict(x=A0 + 2 * (128 - 63)), dict(x=A0 + 2 * 64, ld_x=129),
    dict(x=A0 + 2 * (128 + 63)), dict(r_out=B0 + 2), dict(r_out=B0 - 2), dict(r_out=C0, x=C0 - 126)])
def test_columns_that_overlap_are_refused(kw):
    base = dict(ld_y=128, ld_r=128, ld_r_out=128, ld_x=128)
    assert call(**{**base, **kw}) == sbg.binding.LOWM_ERR_INVALID_ARG


def test_no_rows_is_no_work():
    assert call(M=0) == 0 and call(M=0, y=None) == 0
    assert ops.library().lib.lowm_quantize_rows(None, 0, 8, 0, 8, None, None, None) == 0
    assert ops.library().lib.lowm_residual_norm(None, None) == sbg.binding.LOWM_ERR_INVALID_ARG


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), -1), (dict(q=None), -1), (dict(scale=None), -1), (dict(K=0), -1),
    (dict(ld=63), -1), (dict(t=2), -1), (dict(q=A0), -1), (dict(scale=A0), -1),
    (dict(K=32769, ld=32769), -2), (dict(x=A0 + 1), -2), (dict(scale=C0 + 2), -2)])
def test_quantize_rows_refuses(kw, code):
    a = dict(x=A0, t=0, ld=64, M=4, K=64, q=B0, scale=C0)
    a.update(kw)
    assert ops.library().lib.lowm_quantize_rows(a["x"], a["t"], a["ld"], a["M"], a["K"], a["q"],
                                                a["scale"], None) == code


def test_python_checks():
    y = torch.zeros(2, 8, dtype=BF16)
    for bad in (lambda: sbg.residual_norm(y, y), lambda: sbg.quantize_rows(y),
                lambda: sbg.quantize_rows(y.to(torch.float16)),
                lambda: sbg.quantize_rows(y.to(torch.int8))):
        with pytest.raises((ValueError, TypeError)):
            bad()
