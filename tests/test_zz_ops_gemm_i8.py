"""gemm_i8 against its formula, bit for bit: the int32 sum is exact, and the
conversion, the two products and the final rounding are each rounded correctly
on both sides."""
from __future__ import annotations

import ctypes

import pytest
import torch

import split_bf16_gemm_amd as sbg
from split_bf16_gemm_amd import ops

BF16, F32, I8 = torch.bfloat16, torch.float32, torch.int8


def formula(q, sa, W, sw, dtype):
    total = (q.double() @ W.double().t()).long()        # below 2^53: exact
    assert total.abs().max() < 2 ** 31
    return (total.to(torch.int32).float() * sa[:, None] * sw).to(dtype)


def workspace_is_clean(ws):
    """What has to be zero between calls: the counters and the partial sums."""
    assert ws[:256 * 512 + 8192 * 1024].count_nonzero() == 0


def operands(g, M, N, K, lo=-128):
    q = torch.randint(lo, 128, (M, K), generator=g, dtype=I8)
    W = torch.randint(lo, 128, (N, K), generator=g, dtype=I8)
    return q, torch.rand(M, generator=g) + 0.5, W, torch.rand(N, generator=g) - 0.5


SHAPES = [(1, 1, 16), (1, 17, 48), (2, 16, 128), (3, 33, 144), (5, 100, 496), (16, 64, 512),
          (17, 65, 528), (23, 2304, 1040), (32, 31, 2048), (33, 48, 4096), (40, 257, 1616),
          (48, 15, 640), (49, 4099, 1024), (64, 96, 4112), (64, 9000, 256), (7, 13000, 256),
          (1, 768, 12304), (30, 6151, 400), (64, 6150, 384), (4, 49152, 112), (17, 16385, 144), (33, 16400, 272),
          (64, 20000, 1040), (24, 33000, 400), (50, 49152, 512), (64, 66000, 128)]


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("dtype", [BF16, F32])
def test_int8_rows(M, N, K, dtype):
    g = torch.Generator().manual_seed(M + N + K)
    q, sa, W, sw = operands(g, M, N, K)
    args = (q.cuda(), W.cuda(), sw.cuda())
    ws = sbg.make_gemm_i8_workspace(M, N, K)
    whole = sbg.gemm_i8(*args, a_scale=sa.cuda(), out_dtype=dtype)
    split = sbg.gemm_i8(*args, a_scale=sa.cuda(), out_dtype=dtype, workspace=ws)
    torch.cuda.synchronize()
    want = formula(q, sa, W, sw, dtype)
    assert torch.equal(whole.cpu(), want) and torch.equal(split.cpu(), want)
    workspace_is_clean(ws)


@pytest.mark.gpu
@pytest.mark.parametrize("M", range(1, 65))
def test_every_row_count(M):
    g = torch.Generator().manual_seed(M)
    q, sa, W, sw = operands(g, M, 50, 1168)
    ws = sbg.make_gemm_i8_workspace(M, 50, 1168)
    for w in (None, ws):
        got = sbg.gemm_i8(q.cuda(), W.cuda(), sw.cuda(), a_scale=sa.cuda(), out_dtype=F32,
                          workspace=w)
        assert torch.equal(got.cpu(), formula(q, sa, W, sw, F32))
    workspace_is_clean(ws)


@pytest.mark.gpu
def test_the_largest_sums():
    K = 131056
    q = torch.full((2, K), -128, dtype=I8)
    W = torch.full((3, K), -128, dtype=I8)
    W[1] = 127
    one = torch.ones(3)
    for ws in (None, sbg.make_gemm_i8_workspace(2, 3, K)):
        got = sbg.gemm_i8(q.cuda(), W.cuda(), one.cuda(), a_scale=one[:2].cuda(), out_dtype=F32,
                          workspace=ws)
        assert torch.equal(got.cpu(), formula(q, one[:2], W, one, F32))


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 6144, 4096), (1, 40, 16), (4, 300, 8192), (13, 70, 4112),
                                   (16, 512, 4096), (17, 128, 1536), (64, 1000, 4096),
                                   (2, 48, 32768), (64, 64, 32768), (1, 33, 32752),
                                   (3, 100, 48), (4, 16384, 512), (5, 700, 4096), (8, 6144, 4080),
                                   (8, 16400, 640), (2, 12000, 8192), (4, 90, 8176), (6, 50, 1040),
                                   (7, 2304, 144), (8, 9000, 4096), (1, 20, 4112)])
def test_bf16_rows_are_quantised_as_quantize_rows_does(M, N, K):
    g = torch.Generator().manual_seed(K + M)
    _, _, W, sw = operands(g, 1, N, K)
    x = torch.randn(M, K, generator=g).to(BF16)
    x[0, K // 2] = 9.0
    sa = x.float().abs().amax(1) / 127
    q = torch.round(x.float() / sa[:, None]).to(I8)
    ws = sbg.make_gemm_i8_workspace(M, N, K)
    for dtype in (BF16, F32):
        got = sbg.gemm_i8(x.cuda(), W.cuda(), sw.cuda(), out_dtype=dtype, workspace=ws)
        assert torch.equal(got.cpu(), formula(q, sa, W, sw, dtype))
    workspace_is_clean(ws)


@pytest.mark.gpu
@pytest.mark.parametrize("M,N,K", [(1, 40, 16), (3, 500, 112), (16, 700, 400), (64, 4100, 144),
                                   (64, 16000, 1040), (40, 24700, 528),
                                   # 2^24 bytes of W and more
                                   (1, 2056, 8208), (1, 16400, 1072), (3, 5000, 3376),
                                   (8, 9100, 1872), (6, 13000, 1296), (4, 1100, 15904),
                                   (8, 70000, 240), (16, 1400, 12016), (16, 40000, 432),
                                   (31, 9000, 1904), (32, 65600, 256), (20, 16500, 1040),
                                   (40, 24700, 688), (64, 4100, 4112), (64, 12500, 1360),
                                   (33, 16000, 2064), (64, 50000, 400), (50, 150000, 112),
                                   (9, 33000, 512), (16, 49152, 640), (1, 40000, 528),
                                   (12, 66000, 272), (2, 100000, 256)])
@pytest.mark.parametrize("offset", [0, 16, 112])
def test_rows_anywhere_in_a_line_of_memory(M, N, K, offset):
    """W starts `offset` bytes into its storage, among bytes of 127."""
    g = torch.Generator().manual_seed(M + N + K + offset)
    q, sa, W, sw = operands(g, M, N, K)
    room = torch.full((offset + N * K + 512,), 127, dtype=I8, device="cuda")
    placed = room[offset:offset + N * K].view(N, K)
    placed.copy_(W)
    ws = sbg.make_gemm_i8_workspace(M, N, K)
    want = formula(q, sa, W, sw, F32)
    for w in (None, ws):
        got = sbg.gemm_i8(q.cuda(), placed, sw.cuda(), a_scale=sa.cuda(), out_dtype=F32, workspace=w)
        assert torch.equal(got.cpu(), want)
    if M <= 8:
        x = q.to(BF16)
        x[:, 0] = -127.0                                # so that the scales are ones
        x.clamp_(min=-127.0)
        got = sbg.gemm_i8(x.cuda(), placed, sw.cuda(), out_dtype=F32, workspace=ws)
        assert torch.equal(got.cpu(), formula(x.to(I8), torch.ones(M), W, sw, F32))
    workspace_is_clean(ws)


@pytest.mark.gpu
@pytest.mark.parametrize("M", [1, 4, 8])
@pytest.mark.parametrize("N,K", [(40, 16), (4096, 112), (8192, 256), (12000, 384), (4000, 640),
                                 # rows that are not whole lines, 2^24 bytes of W
                                 (8150, 2064), (6000, 2800), (5000, 3376)])
def test_bf16_rows_shorter_than_the_ring(M, N, K):
    """Wavefronts with fewer steps than their ring has slots, or with none: the slots' loads end
    before the sums take their place."""
    g = torch.Generator().manual_seed(M + N + K)
    _, _, W, sw = operands(g, 1, N, K)
    x = torch.randint(-126, 127, (M, K), generator=g).to(BF16)
    x[:, K // 3] = 127.0                                # so that the scales are ones
    ws = sbg.make_gemm_i8_workspace(M, N, K)
    want = formula(x.to(I8), torch.ones(M), W, sw, F32)
    x, W, sw = x.cuda(), W.cuda(), sw.cuda()
    for _ in range(4):
        assert torch.equal(sbg.gemm_i8(x, W, sw, out_dtype=F32, workspace=ws).cpu(), want)


@pytest.mark.gpu
@pytest.mark.parametrize("K", [512, 4096, 32768])
def test_rows_of_zeros_and_without_a_scale(K):
    g = torch.Generator().manual_seed(6)
    _, _, W, sw = operands(g, 1, 20, K)
    x = torch.randn(4, K, generator=g).to(BF16)
    x[0] = 0
    x[1, K - 3], x[2, 0] = float("inf"), float("nan")
    got = sbg.gemm_i8(x.cuda(), W.cuda(), sw.cuda(),
                      workspace=sbg.make_gemm_i8_workspace(4, 20, K)).cpu()
    assert (got[0] == 0).all() and got[1:3].isnan().all() and got[3].isfinite().all()


@pytest.mark.gpu
def test_nothing_beside_the_output_is_written():
    g = torch.Generator().manual_seed(7)
    q, sa, W, sw = operands(g, 5, 37, 400)
    whole = torch.full((9, 37), 5.0, device="cuda")
    sbg.gemm_i8(q.cuda(), W.cuda(), sw.cuda(), a_scale=sa.cuda(), out=whole[2:7])
    assert (whole[:2] == 5).all() and (whole[7:] == 5).all()
    assert torch.equal(whole[2:7].cpu(), formula(q, sa, W, sw, F32))


@pytest.mark.gpu
def test_on_another_stream_and_in_a_graph():
    g = torch.Generator().manual_seed(8)
    _, _, W, sw = operands(g, 1, 1000, 2048)
    W, sw = W.cuda(), sw.cuda()
    x = torch.randn(6, 2048, generator=g).to(BF16).cuda()
    ws, ws2 = (sbg.make_gemm_i8_workspace(6, 1000, 2048) for _ in range(2))
    out = sbg.gemm_i8(x, W, sw, workspace=ws)
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    with torch.cuda.graph(graph):
        sbg.gemm_i8(x, W, sw, workspace=ws, out=out)
    for i in range(3):
        x.copy_(torch.randn(6, 2048, generator=g))
        want = sbg.gemm_i8(x, W, sw, workspace=ws2)
        torch.cuda.synchronize()
        other = sbg.gemm_i8(x, W, sw, workspace=ws2, stream=side)
        side.synchronize()
        out.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want) and torch.equal(other, want)
    assert sbg.load().workspace_status(ws, 8192) == (0, 0)


# -- refusals ------------------------------------------------------------------------------------
BASE = dict(A=0x10000000, W=0x20000000, a_scale=0x30000000, w_scale=0x31000000, C=0x32000000,
            workspace=0x33000000, workspace_bytes=1 << 24, M=4, N=64, K=512, a_type=2, c_type=0)


@pytest.mark.parametrize("kw,code", [
    (dict(A=None), -1), (dict(W=None), -1), (dict(a_scale=None), -1), (dict(w_scale=None), -1),
    (dict(C=None), -1), (dict(M=0), -1), (dict(N=0), -1), (dict(K=0), -1), (dict(a_type=1), -1),
    (dict(c_type=2), -1), (dict(C=0x10000400), -1), (dict(C=0x31000010), -1),
    (dict(a_type=0, C=0x33000000), -1), (dict(a_type=0, workspace=0x20000100), -1),
    (dict(workspace=0x20000100), -1),
    (dict(M=65), -2), (dict(K=520), -2), (dict(K=131072), -2), (dict(a_type=0, K=32784), -2),
    (dict(A=0x10000008), -2), (dict(W=0x20000004), -2), (dict(C=0x32000001), -2),
    (dict(C=0x32000002, c_type=1), -2), (dict(w_scale=0x31000002), -2),
    (dict(a_scale=0x30000001), -2), (dict(workspace=0x33000080), -2),
    (dict(a_type=0, workspace=None), -3), (dict(a_type=0, workspace_bytes=1 << 20), -3),
    (dict(workspace_bytes=1 << 20), -3)])
def test_refuses(kw, code):
    a = ops.GemmI8Args(**{**BASE, **kw})
    assert ops.library().lib.lowm_gemm_i8(ctypes.byref(a), None) == code


def test_workspace_bytes():
    f = ops.library().lib.lowm_gemm_i8_workspace_bytes
    assert f(4, 64, 512) == 256 * 512 + 8192 * 1024 + 2048 + 256
    assert f(65, 64, 512) == f(4, 64, 520) == f(0, 64, 512) == f(4, 64, 131072) == 0


def test_more_columns_than_one_launch_holds_are_refused():
    f = ops.library().lib.lowm_gemm_i8_workspace_bytes
    most = 2 ** 30 - 256
    assert f(1, most, 16) > 0
    for N in (most + 1, 2 ** 30, 2 ** 31 - 1):
        a = ops.GemmI8Args(**{**BASE, "N": N, "K": 16})
        assert ops.library().lib.lowm_gemm_i8(ctypes.byref(a), None) == -2
        assert f(1, N, 16) == 0


def test_python_checks():
    q = torch.zeros(2, 16, dtype=I8)
    for bad in (lambda: sbg.gemm_i8(q, q, torch.ones(2)),
                lambda: sbg.gemm_i8(q.to(BF16), q, torch.ones(2)), lambda: sbg.gemm_i8(q.half(), q, q),
                lambda: sbg.gemm_i8(q, q[:, :8], q)):
        with pytest.raises((ValueError, TypeError)):
            bad()
