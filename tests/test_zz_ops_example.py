"""The operators run together (examples/decode_block.py), each output against the
64-bit formula of the outputs before it; and the C ABI of include/lowm_ops.h."""
from __future__ import annotations

import re
import sys
from pathlib import Path

import pytest
import torch

import split_bf16_gemm_amd as sbg
from split_bf16_gemm_amd import ops

ROOT = Path(__file__).resolve().parents[1]
sys.path.insert(0, str(ROOT / "examples"))


def unit(v):
    return v / torch.sqrt((v * v).mean(-1, keepdim=True) + 1e-6)


def near(got, want, rel):
    got, want = got.double().cpu(), want.cpu()
    assert (got - want).norm() <= rel * want.norm(), ((got - want).norm() / want.norm())


@pytest.mark.gpu
@pytest.mark.parametrize("tokens,hidden,inner,experts,top_k,vocab", [
    (1, 1024, 128, 8, 2, 5000), (5, 512, 264, 20, 4, 9000), (33, 2048, 64, 6, 3, 3001)])
def test_decode_block(tokens, hidden, inner, experts, top_k, vocab):
    from decode_block import DecodeBlock
    b = DecodeBlock(tokens, hidden, inner, experts, top_k, vocab)
    graph, o = b.capture()
    for _ in range(3):
        graph.replay()
        eager = b.step()
        torch.cuda.synchronize()
        for k in o:
            assert torch.equal(o[k], eager[k]), k
    # A rounding to bf16 is off by at most 2^-8 of the value; the norms of whole
    # outputs are held to that, times the roundings on the way.
    step = 2.0 ** -8
    d = {k: v.double().cpu() for k, v in o.items()}
    n = [w.double().cpu() for w in b.norms]
    r1 = b.r.double().cpu() + b.gate.double().cpu() * unit(b.y.double().cpu()) * n[0]
    x1 = unit(r1) * n[1]
    # int8: half a step of the row's scale, in the root mean square under a third
    err = (d["q"] * d["scale"][:, None] - x1).abs()
    assert (err <= 0.501 * d["scale"][:, None]).all()
    dense = (d["q"] @ b.W.double().cpu().t()) * d["scale"][:, None] * b.w_scale.double().cpu()
    near(o["dense"], dense, step)
    r2 = r1 + unit(d["dense"]) * n[2]
    near(o["x2"], unit(r2) * n[3], step)
    mixed = torch.zeros(tokens, hidden, dtype=torch.float64)
    for t in range(tokens):
        for e, g in zip(d["ids"][t].long().tolist(), d["gates"][t].tolist()):
            a = b.w13[e].double().cpu() @ d["x2"][t]
            h = a[:inner] * torch.sigmoid(a[:inner]) * a[inner:]
            mixed[t] += g * (b.w2[e].double().cpu() @ h)
    near(o["mixed"], mixed, 2 * step)
    r3 = r2 + unit(d["mixed"]) * n[4]
    near(o["residual"], r3, 2.0 ** -20)
    near(o["x3"], unit(r3) * n[5], step)
    near(o["logits"], d["x3"] @ b.head.double().cpu().t(), step)
    lp = torch.log_softmax(d["logits"], 1)
    tok = b.tokens.cpu()
    near(o["logprob"], lp.gather(1, tok[:, None])[:, 0], 2.0 ** -18)
    near(o["entropy"], -(lp.exp() * lp).sum(1), 2.0 ** -16)
    assert torch.equal(o["top_ids"].cpu().long(),
                       torch.sort(d["logits"], dim=1, descending=True, stable=True).indices[:, :5])


def test_a_stream_of_another_gpu_is_refused():
    class Stream:
        cuda_stream, device = 0x1230, torch.device("cuda", 1)

    assert ops._stream(Stream(), torch.device("cuda", 1)) == 0x1230
    with pytest.raises(ValueError, match="cuda:1.*cuda:0"):
        ops._stream(Stream(), torch.device("cuda", 0))


@pytest.mark.gpu
@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs a second GPU")
def test_tensors_on_a_gpu_that_is_not_the_current_one():
    """The calls run where the tensors are, and leave the current device as it was."""
    assert torch.cuda.current_device() == 0
    g = torch.Generator().manual_seed(1)
    x = torch.randn(3, 4096, generator=g).to(torch.bfloat16).cuda(1)
    W = torch.randint(-127, 128, (64, 4096), generator=g, dtype=torch.int8).cuda(1)
    w_scale, tokens = torch.ones(64, device="cuda:1"), torch.zeros(3, dtype=torch.int64, device="cuda:1")

    def calls():
        return (*sbg.residual_norm(x, x)[:2], *sbg.quantize_rows(x),
                sbg.gemm_i8(x, W, w_scale, workspace=sbg.make_gemm_i8_workspace(3, 64, 4096, "cuda:1")),
                *sbg.token_logprobs(x, tokens))

    got = calls()
    assert torch.cuda.current_device() == 0 and all(t.device.index == 1 for t in got)
    with torch.cuda.device(1):
        want = calls()
    torch.cuda.synchronize(1)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def header():
    return re.sub(r"/\*.*?\*/", "", (ROOT / "include" / "lowm_ops.h").read_text(), flags=re.S)


def test_every_declared_symbol_is_exported():
    names = sorted(set(re.findall(r"\b(lowm_\w+)\s*\(", header())))
    assert len(names) >= 8
    for name in names:
        assert hasattr(ops.library().lib, name), name


@pytest.mark.parametrize("struct,cls", [
    ("lowm_residual_norm_args", ops.ResidualNormArgs), ("lowm_gemm_i8_args", ops.GemmI8Args),
    ("lowm_moe_args", ops.MoeArgs), ("lowm_token_logprobs_args", ops.TokenLogprobsArgs)])
def test_structs_are_the_headers(struct, cls):
    body = re.search(r"typedef struct %s \{(.*?)\}" % struct, header(), re.S).group(1)
    names = []
    for line in body.split(";"):
        words = line.replace("*", " ").replace(",", " ").split()
        names += [w for w in words if w not in ("const", "void", "float", "int32_t", "int64_t",
                                                "size_t")]
    assert names == [f[0] for f in cls._fields_]


def test_public_names():
    for name in ("residual_norm", "quantize_rows", "gemm_i8", "make_gemm_i8_workspace", "moe",
                 "make_moe_workspace", "token_logprobs", "make_token_logprobs_workspace"):
        assert name in sbg.__all__ and callable(getattr(sbg, name))
        assert getattr(sbg, name).__doc__
