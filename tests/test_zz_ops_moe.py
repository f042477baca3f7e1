"""moe against its formula in 64 bits.

Integers chosen so that every step is exact are compared bit for bit.  For
random values, with u = 2^-24: a product's sum of n terms is off by at most
(n + 8) u times the sum of the terms' magnitudes, h is rounded to bf16 (2^-8) and
so is the output; the bound of the second product carries both.
"""
from __future__ import annotations

import ctypes

import pytest
import torch

import split_bf16_gemm_amd as sbg
from split_bf16_gemm_amd import ops

U = 2.0 ** -24
BF16, F32, F64 = torch.bfloat16, torch.float32, torch.float64


def route(x, router, k, score, bias, renorm, scale):
    l = x.double() @ router.double().t()
    s = torch.sigmoid(l) if score == "sigmoid" else torch.softmax(l, 1)
    by = l if bias is None else s + bias.double()
    top = torch.sort(by, dim=1, descending=True, stable=True)
    ids = top.indices[:, :k]
    g = s.gather(1, ids)
    if renorm:
        g = g / g.sum(1, keepdim=True)
    return ids, g * scale, by


def reference(x, w13, w2, ids, gates):
    """(out, bound of the error before the output's rounding), fp64."""
    T, D = x.shape
    E, _, I = w2.shape
    X = x.double()
    out, err = torch.zeros(T, D, dtype=F64), torch.zeros(T, D, dtype=F64)
    for e in torch.unique(ids).tolist():
        t, slot = (ids == e).nonzero(as_tuple=True)
        W, V = w13[e].double(), w2[e].double()
        a = X[t] @ W.t()
        mag = (X[t].abs() @ W.abs().t()) * (D + 8) * U
        g, up = a[:, :I], a[:, I:]
        sg = torch.sigmoid(g)
        h = g * sg * up
        # |silu'| <= 1.1
        herr = 1.1 * mag[:, :I] * (up.abs() + mag[:, I:]) + (g * sg).abs() * mag[:, I:]
        herr = herr + 8 * U * h.abs() * (1 + g.abs()) + 2.0 ** -8 * (h.abs() + herr)
        w = gates[t, slot][:, None]
        y = h @ V.t()
        yerr = (herr + (I + 40) * U * (h.abs() + herr)) @ V.abs().t()
        out[t] += w * y
        err[t] += w.abs() * (yerr + 40 * U * y.abs())
    return out, err


def draw(g, T, D, I, E, k):
    def r(*shape, std):
        return (torch.randn(*shape, generator=g) * std).to(BF16)
    return (r(T, D, std=1.0), r(E, D, std=D ** -0.5 * 1.5), r(E, 2 * I, D, std=D ** -0.5),
            r(E, D, I, std=I ** -0.5))


def workspace_is_clean(ws, T, D, I, E, k):
    """What has to be zero between calls: all of the front part."""
    front = 256 * (5 + 65536 // 16) + 4 * (4 * 64 * 256 + 512 * 64 * 16 + 2 * 64 * 16)
    assert ws[:front].count_nonzero() == 0


SIZES = [(1, 8, 8, 1, 1), (1, 4096, 1024, 64, 4), (2, 64, 8, 3, 3), (3, 520, 136, 20, 8),
         (16, 512, 128, 8, 2), (17, 256, 72, 5, 5), (64, 128, 40, 8, 2), (64, 64, 64, 1, 1),
         (33, 2048, 768, 128, 8), (64, 1024, 264, 256, 16), (5, 4104, 200, 12, 4),
         (48, 72, 1032, 40, 7), (20, 1536, 64, 200, 16), (64, 4096, 256, 6, 3),
         (31, 8, 2048, 9, 1)]


@pytest.mark.gpu
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "t%d_d%d_i%d_e%d_k%d" % s)
@pytest.mark.parametrize("score,bias,renorm,scale", [
    ("softmax", False, True, 1.0), ("sigmoid", True, True, 2.5), ("softmax", True, False, 1.0),
    ("sigmoid", False, False, 0.5)])
def test_moe(size, score, bias, renorm, scale):
    T, D, I, E, k = size
    g = torch.Generator().manual_seed(sum(size))
    x, router, w13, w2 = draw(g, *size)
    b = torch.randn(E, generator=g) * 0.1 if bias else None
    ws = sbg.make_moe_workspace(T, D, I, E, k)
    out, ids, gates = sbg.moe(x.cuda(), router.cuda(), w13.cuda(), w2.cuda(), k, score=score,
                              bias=None if b is None else b.cuda(), renormalize=renorm,
                              routed_scale=scale, workspace=ws)
    torch.cuda.synchronize()
    out, ids, gates = out.cpu().double(), ids.cpu().long(), gates.cpu().double()
    want_ids, want_gates, by = route(x, router, k, score, b, renorm, scale)
    # an expert out of the reference's order has the reference's value but for rounding
    near = (by.gather(1, ids) - by.gather(1, want_ids)).abs()
    assert (near <= 64 * U * (1 + by.abs().amax(1, keepdim=True))).all()
    assert all(len(set(r)) == k for r in ids.tolist())
    assert (ids == want_ids).double().mean() > 0.99
    s = torch.sigmoid(x.double() @ router.double().t()) if score == "sigmoid" else \
        torch.softmax(x.double() @ router.double().t(), 1)
    want_gates = s.gather(1, ids)
    if renorm:
        want_gates = want_gates / want_gates.sum(1, keepdim=True)
    want_gates = want_gates * scale
    assert ((gates - want_gates).abs() <= 200 * U * want_gates).all()
    want, err = reference(x, w13, w2, ids, gates)
    assert ((out - want).abs() <= err + 2.0 ** -8 * (want.abs() + err)).all()
    assert (out - want).norm() <= 2.0 ** -7 * want.norm()
    workspace_is_clean(ws, *size)


def exact_operands(g, T, D, I, E):
    """Integers for which every step is exact: the gate product is 32 (silu(32) is 32 in fp32),
    the up products stay below 2^8 and the second products' sums below 2^24."""
    x = torch.randint(-1, 2, (T, D), generator=g).float()
    x[:, 0] = 1
    w13 = torch.zeros(E, 2 * I, D)
    w13[:, :I, 0] = 32
    dense = min(1.0, 200 / D)
    up = torch.randint(-1, 2, (E, I, D), generator=g).float()
    w13[:, I:] = up * (torch.rand(E, I, D, generator=g) < dense)
    w2 = torch.randint(-2, 3, (E, D, I), generator=g).float()
    router = torch.randint(-1, 2, (E, D), generator=g).float()
    return x, router, w13, w2


@pytest.mark.gpu
@pytest.mark.parametrize("size", SIZES, ids=lambda s: "t%d_d%d_i%d_e%d_k%d" % s)
def test_integers_are_exact(size):
    T, D, I, E, _ = size
    g = torch.Generator().manual_seed(1 + sum(size))
    x, router, w13, w2 = exact_operands(g, T, D, I, E)
    ws = sbg.make_moe_workspace(T, D, I, E, 1)
    args = [t.to(BF16).cuda() for t in (x, router, w13, w2)]
    out, ids, gates = sbg.moe(*args, 1, workspace=ws)
    torch.cuda.synchronize()
    # whole logits, with many ties: the lowest expert among the equal ones
    logits = x.double() @ router.double().t()
    want = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :1]
    assert torch.equal(ids.cpu().long(), want) and (gates == 1).all()
    for t in range(T):
        e = int(want[t])
        a = w13[e].double() @ x[t].double()
        assert (a[:I] == 32).all() and a[I:].abs().max() < 256
        y = w2[e].double() @ (32 * a[I:])
        assert y.abs().max() < 2 ** 24
        assert torch.equal(out[t].cpu(), y.to(F32).to(BF16)), t
    workspace_is_clean(ws, T, D, I, E, 1)


@pytest.mark.gpu
@pytest.mark.parametrize("T,E", [(1, 7), (6, 7), (40, 7), (50, 3), (64, 2)])
@pytest.mark.parametrize("D,I", [(72, 16), (520, 200), (648, 24), (1240, 328), (1312, 408),
                                 (1960, 88), (2104, 120), (264, 1048), (512, 64)])
@pytest.mark.parametrize("offset", [0, 8, 56])
def test_rows_anywhere_in_a_line_of_memory(T, E, D, I, offset):
    """Weights that start `offset` elements into their storage, among NaN, which also fills
    every expert that no token chose: exact integers, so a byte too many or too few shows."""
    g = torch.Generator().manual_seed(T + D + I + offset)
    x, router, w13, w2 = exact_operands(g, T, D, I, E)
    logits = x.double() @ router.double().t()
    want = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, 0]
    idle = [e for e in range(E) if not (want == e).any()]

    def placed(w):
        w = w.to(BF16)
        w[idle] = float("nan")
        room = torch.full((w.numel() + offset + 512,), float("nan"), dtype=BF16, device="cuda")
        view = room[offset:offset + w.numel()].view(w.shape)
        view.copy_(w)
        return view

    out, ids, _ = sbg.moe(x.to(BF16).cuda(), router.to(BF16).cuda(), placed(w13), placed(w2), 1,
                          workspace=sbg.make_moe_workspace(T, D, I, E, 1))
    assert torch.equal(ids[:, 0].cpu().long(), want)
    for t in range(T):
        e = int(want[t])
        h = 32 * (w13[e, I:].double() @ x[t].double())
        y = (w2[e].double() @ h.to(BF16).double()).to(torch.float32).to(BF16)
        assert torch.equal(out[t].cpu(), y)


@pytest.mark.gpu
@pytest.mark.parametrize("T,D,I,E,k", [(64, 264, 120, 4, 3), (64, 256, 128, 6, 2), (61, 512, 64, 2, 2),
                                       (33, 136, 200, 3, 2), (64, 128, 64, 16, 8), (40, 64, 264, 1, 1)])
def test_many_rows_to_an_expert(T, D, I, E, k):
    """Every token's first choices the same experts, so that some get all rows, others none."""
    g = torch.Generator().manual_seed(T + D + I)
    x, router, w13, w2 = draw(g, T, D, I, E, k)
    bias = torch.arange(E, 0, -1).float() * 4
    out, ids, gates = sbg.moe(x.cuda(), router.cuda(), w13.cuda(), w2.cuda(), k, score="sigmoid",
                              bias=bias.cuda(), workspace=sbg.make_moe_workspace(T, D, I, E, k))
    assert (ids.cpu() == torch.arange(k, dtype=torch.int32)).all()
    want, err = reference(x, w13, w2, ids.cpu().long(), gates.cpu().double())
    diff = (out.cpu().double() - want).abs()
    assert (diff <= err + 2.0 ** -8 * (want.abs() + err)).all()


@pytest.mark.gpu
def test_every_token_count_and_one_workspace_for_all():
    D, I, E, k = 256, 64, 7, 3
    g = torch.Generator().manual_seed(5)
    x, router, w13, w2 = draw(g, 64, D, I, E, k)
    ws = sbg.make_moe_workspace(64, D, I, E, k)
    dev = [t.cuda() for t in (x, router, w13, w2)]
    whole, ids, gates = sbg.moe(*dev, k, workspace=ws)
    for T in list(range(1, 64)):
        out, i, gt = sbg.moe(dev[0][:T], *dev[1:], k, workspace=ws)
        assert torch.equal(i, ids[:T])
        want, err = reference(x[:T], w13, w2, i.cpu().long(), gt.cpu().double())
        diff = (out.cpu().double() - want).abs()
        assert (diff <= err + 2.0 ** -8 * (want.abs() + err)).all(), T
    workspace_is_clean(ws, 64, D, I, E, k)


@pytest.mark.gpu
def test_a_workspace_serves_other_sizes():
    big = (64, 1024, 512, 32, 4)
    ws = sbg.make_moe_workspace(*big)
    for size in (big, (1, 520, 136, 20, 8), (17, 2048, 64, 5, 5), (3, 64, 512, 32, 4), big):
        g = torch.Generator().manual_seed(sum(size))
        x, router, w13, w2 = draw(g, *size)
        dev = [t.cuda() for t in (x, router, w13, w2)]
        a = sbg.moe(*dev, size[4], workspace=ws)
        b = sbg.moe(*dev, size[4], workspace=sbg.make_moe_workspace(*size))
        assert all(torch.equal(p, q) for p, q in zip(a, b))
        workspace_is_clean(ws, *size)


@pytest.mark.gpu
def test_same_bits_each_time_in_a_graph_and_on_another_stream():
    size = (13, 1032, 136, 24, 4)
    g = torch.Generator().manual_seed(9)
    x, router, w13, w2 = (t.cuda() for t in draw(g, *size))
    ws, ws2 = sbg.make_moe_workspace(*size), sbg.make_moe_workspace(*size)
    outs = [torch.zeros_like(t) for t in sbg.moe(x, router, w13, w2, 4, workspace=ws)]
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        sbg.moe(x, router, w13, w2, 4, workspace=ws, out=outs[0], ids_out=outs[1],
                gates_out=outs[2])
    for i in range(4):
        x.copy_(torch.randn(13, 1032, generator=g))
        want = sbg.moe(x, router, w13, w2, 4, workspace=ws2)
        torch.cuda.synchronize()
        graph.replay()
        other = sbg.moe(x, router, w13, w2, 4, workspace=ws2, stream=side)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(outs, want))
        assert all(torch.equal(a, b) for a, b in zip(other, want))
    assert sbg.load().workspace_status(ws, 1032 + 80) == (0, 0)


@pytest.mark.gpu
def test_a_token_of_nan_stays_its_own():
    size = (18, 256, 64, 6, 2)
    g = torch.Generator().manual_seed(10)
    x, router, w13, w2 = draw(g, *size)
    dev = [t.cuda() for t in (router, w13, w2)]
    ws = sbg.make_moe_workspace(*size)
    want = sbg.moe(x.cuda(), *dev, 2, workspace=ws)
    y = x.clone()
    y[3, 7] = float("nan")
    got = sbg.moe(y.cuda(), *dev, 2, workspace=ws)
    ok = torch.arange(18) != 3
    assert torch.equal(got[0].cpu()[ok], want[0].cpu()[ok])
    assert got[0][3].isnan().all() and (got[1][3] < 6).all() and (got[1][3] >= 0).all()
    workspace_is_clean(ws, *size)


@pytest.mark.gpu
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("biased", [False, True])
@pytest.mark.parametrize("lift", [0, 2, 16])
def test_gates_of_scores_below_the_smallest_number(score, biased, lift):
    """Chosen experts whose scores are 0 in fp32 (logits of -120 to -500, or that far below the
    largest) still share the gate by the ratios of their scores.  The logits are exact."""
    T, D, I, E, k = 5, 64, 32, 12, 4
    g = torch.Generator().manual_seed(21)
    x, router, w13, w2 = draw(g, T, D, I, E, k)
    x[:, 0] = torch.tensor([1, 2, 4, 1, 2])
    router[:] = 0
    router[:, 0] = -(120 + torch.arange(E) / 2)
    bias = None
    if biased:
        bias = torch.arange(E).float() * 4         # the choice goes by the bias
    if lift:
        router[0, 0] = lift / 4                     # one expert far above the others
    want_ids, want, _ = route(x, router, k, score, bias, True, 1.0)
    assert want.isfinite().all()
    out, ids, gates = sbg.moe(x.cuda(), router.cuda(), w13.cuda(), w2.cuda(), k, score=score,
                              bias=None if bias is None else bias.cuda(),
                              workspace=sbg.make_moe_workspace(T, D, I, E, k))
    assert torch.equal(ids.cpu().long(), want_ids)
    gates = gates.cpu().double()
    # gates below the smallest normal fp32 may be 0
    assert ((gates - want).abs() <= 200 * U * want + 2.0 ** -126).all()
    want_out, err = reference(x, w13, w2, want_ids, gates)
    diff = (out.cpu().double() - want_out).abs()
    assert (diff <= err + 2.0 ** -8 * (want_out.abs() + err)).all()


@pytest.mark.gpu
@pytest.mark.parametrize("given", [False, True])
def test_no_tokens_at_all(given):
    size = (0, 64, 32, 6, 2)
    _, router, w13, w2 = (t.cuda() for t in draw(torch.Generator().manual_seed(1), 1, *size[1:]))
    x = torch.zeros(0, 64, dtype=BF16, device="cuda")
    ws = sbg.make_moe_workspace(4, *size[1:]) if given else sbg.make_moe_workspace(*size)
    out, ids, gates = sbg.moe(x, router, w13, w2, 2, workspace=ws)
    assert out.shape == (0, 64) and ids.shape == gates.shape == (0, 2)
    with pytest.raises(ValueError):                # one token needs a workspace
        sbg.moe(torch.zeros(1, 64, dtype=BF16, device="cuda"), router, w13, w2, 2, workspace=None)


@pytest.mark.gpu
def test_nothing_beside_the_outputs_is_written():
    size = (5, 72, 40, 6, 2)
    g = torch.Generator().manual_seed(11)
    dev = [t.cuda() for t in draw(g, *size)]
    out = torch.full((9, 72), 3.0, dtype=BF16, device="cuda")
    ids = torch.full((9, 2), 99, dtype=torch.int32, device="cuda")
    gates = torch.full((9, 2), 9.0, device="cuda")
    sbg.moe(*dev, 2, workspace=sbg.make_moe_workspace(*size), out=out[2:7], ids_out=ids[2:7],
            gates_out=gates[2:7])
    for t, v in ((out, 3), (ids, 99), (gates, 9)):
        assert (t[:2] == v).all() and (t[7:] == v).all() and (t[2:7] != v).any()


# -- refusals ------------------------------------------------------------------------------------
BASE = dict(x=0x10000000, router=0x20000000, w13=0x30000000, w2=0x40000000, out=0x50000000,
            ids=0x51000000, gates=0x52000000, bias=0x53000000, workspace=0x60000000,
            workspace_bytes=1 << 24, T=4, D=64, I=32, E=8, top_k=2, routed_scale=1.0)


def test_fewer_tokens_need_no_more_workspace():
    size = ops.library().lib.lowm_moe_workspace_bytes
    for D, I in ((64, 8), (4096, 1024)):
        for E in (1, 2, 7, 8, 20, 64, 66, 128, 256):
            for k in range(1, min(E, 16) + 1):
                need = [size(T, D, I, E, k) for T in range(1, 65)]
                assert need == sorted(need) and need[0] > 0


@pytest.mark.parametrize("kw,code", [
    (dict(x=None), -1), (dict(router=None), -1), (dict(w13=None), -1), (dict(w2=None), -1),
    (dict(out=None), -1), (dict(T=-1), -1), (dict(D=0), -1), (dict(I=0), -1), (dict(E=0), -1),
    (dict(top_k=0), -1), (dict(top_k=9), -1), (dict(flags=4), -1), (dict(out=0x10000040), -1),
    (dict(out=0x30000100), -1), (dict(ids=0x50000010), -1), (dict(gates=0x60000000), -1),
    (dict(workspace=0x40000000), -1), (dict(T=65), -2), (dict(D=68), -2), (dict(I=36), -2),
    (dict(E=257, top_k=2), -2), (dict(E=200, top_k=17), -2), (dict(D=65544), -2),
    (dict(x=0x10000008), -2), (dict(w2=0x40000002), -2), (dict(ids=0x51000002), -2),
    (dict(workspace=0x60000080), -2), (dict(workspace=None), -3), (dict(workspace_bytes=4096), -3),
    (dict(T=0, x=None), 0)])
def test_refuses(kw, code):
    a = ops.MoeArgs(**{**BASE, **kw})
    assert ops.library().lib.lowm_moe(ctypes.byref(a), None) == code


def test_workspace_bytes():
    f = ops.library().lib.lowm_moe_workspace_bytes
    assert f(4, 64, 32, 8, 2) > 0 and f(64, 4096, 1024, 128, 8) > 2 * 512 * 1024
    assert f(65, 64, 32, 8, 2) == f(4, 60, 32, 8, 2) == f(4, 64, 32, 8, 9) == f(0, 64, 32, 8, 2) == 0


def test_python_checks():
    x = torch.zeros(2, 8, dtype=BF16)
    w13, w2 = torch.zeros(3, 16, 8, dtype=BF16), torch.zeros(3, 8, 8, dtype=BF16)
    for bad in (lambda: sbg.moe(x, torch.zeros(3, 8, dtype=BF16), w13, w2, 1, workspace=None),
                lambda: sbg.moe(x, x, w13[0], w2, 1, workspace=x)):
        with pytest.raises((ValueError, TypeError)):
            bad()
