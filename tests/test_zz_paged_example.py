"""The attention part run together (examples/paged_decode.py), against the 64-bit formula of what
it read; and the C ABI of include/lowm_cache.h."""
from __future__ import annotations

import math
import re
import sys
from pathlib import Path

import pytest
import torch

import split_bf16_gemm_amd as sbg
from split_bf16_gemm_amd import cache

ROOT = Path(__file__).resolve().parents[1]
sys.path.insert(0, str(ROOT / "examples"))


def contents(c, table, n):
    """Keys and values [n, H, D] of one sequence as the cache holds them, fp64 on the CPU."""
    out = []
    for t, scale, order in ((c.k, c.k_scale, (0, 3, 1, 2, 4)), (c.v, c.v_scale, (0, 2, 4, 1, 3))):
        pages = table[:-(-n // 64)].long()
        x = t.view(torch.int8)[pages].view(t.dtype).float().double()
        x = (x * scale[pages].double()[..., None, None, None]).permute(*order)
        out.append(x.reshape(len(pages) * 64, t.shape[1], -1)[:n].cpu())
    return out


@pytest.mark.gpu
@pytest.mark.parametrize("beams,heads,kv_heads,head_dim,dtype", [
    (1, 4, 4, 64, torch.int8), (5, 8, 2, 48, torch.float8_e4m3fn), (7, 6, 1, 128, torch.int8)])
def test_paged_decode(beams, heads, kv_heads, head_dim, dtype):
    from paged_decode import PagedDecode
    hidden, layers, steps = 256, 2, 75
    make = lambda: PagedDecode(beams, hidden, heads, kv_heads, head_dim, layers, steps + 1,  # noqa
                               8 * beams, dtype)
    eager, graphed = make(), make()
    graph = graphed.capture()
    g = torch.Generator().manual_seed(beams)
    for i in range(steps):
        x = torch.randn(beams, hidden, generator=g).to(torch.bfloat16)
        parents = torch.randint(0, beams, (beams,), generator=g) if i % 7 == 6 \
            else torch.arange(beams)
        for run in (eager, graphed):
            run.x.copy_(x)
            run.parents.copy_(parents)
        eager.step()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(eager.result, graphed.result), i
        assert torch.equal(eager.attended, graphed.attended)
        assert int(eager.forked[3]) == 0
        if i % 30 == 29:     # other page numbers, the same sequences
            used = graphed.compact()
            assert used <= int((graphed.forked[2] > 0).sum())
    assert eager.lens.tolist() == [steps] * beams
    # The attention's output is rounded to bf16 (2^-8) and its weights to fp16 (2^-11).
    for layer in range(layers):
        for b in range(beams):
            k, v = contents(eager.cache.layer(layer), eager.table[b], steps)
            q = eager.queries[layer, b].double().cpu()
            for h in range(heads):
                w = torch.softmax(k[:, h * kv_heads // heads] @ q[h] / math.sqrt(head_dim), 0)
                want = w @ v[:, h * kv_heads // heads]
                got = eager.attended[layer, b, h].double().cpu()
                slack = 2.0 ** -8 * want.abs() + 2.0 ** -10 * (w @ v[:, h * kv_heads // heads].abs())
                assert bool(((got - want).abs() <= slack).all())


@pytest.mark.gpu
@pytest.mark.skipif(torch.cuda.device_count() < 2, reason="needs a second GPU")
def test_tensors_on_a_gpu_that_is_not_the_current_one():
    """The calls run where the tensors are, and leave the current device as it was."""
    assert torch.cuda.current_device() == 0
    g = torch.Generator().manual_seed(1)
    q, k, v = (torch.randn(3, h, 64, generator=g).to(torch.bfloat16).cuda(1) for h in (4, 2, 2))
    pos = torch.arange(3, device="cuda:1")

    def calls():
        c = sbg.make_kv_cache(8, 2, 64, device="cuda:1")
        table, lens, refs, missing = sbg.fork_pages(
            c, torch.full((3, 2), -1, dtype=torch.int32, device="cuda:1"),
            torch.zeros(3, dtype=torch.int32, device="cuda:1"), reserve=1,
            workspace=sbg.make_pages_workspace(3, 2, 8, "cuda:1"))
        lens = lens + 1
        q2, k2 = sbg.rotary(q, k, pos, sbg.rotary_frequencies(64, device="cuda:1"))
        sbg.cache_append(k2, v, c, table, lens)
        out, _ = sbg.cache_attention(
            q2, c, table, lens,
            workspace=sbg.make_cache_attention_workspace(3, 4, 2, 64, "cuda:1"))
        table2, refs2, counts = sbg.compact_pages(
            c, table, workspace=sbg.make_pages_workspace(3, 2, 8, "cuda:1"))
        return (table, lens, refs, missing, q2, k2, out, *sbg.cache_read(c, table2, lens), refs2,
                counts)

    got = calls()
    assert torch.cuda.current_device() == 0 and all(t.device.index == 1 for t in got)
    with torch.cuda.device(1):
        want = calls()
    torch.cuda.synchronize(1)
    assert all(torch.equal(a, b) for a, b in zip(got, want))


def header():
    return re.sub(r"/\*.*?\*/", "", (ROOT / "include" / "lowm_cache.h").read_text(), flags=re.S)


def test_every_declared_symbol_is_exported():
    names = sorted(set(re.findall(r"\b(lowm_\w+)\s*\(", header())))
    assert len(names) >= 8
    for name in names:
        assert hasattr(cache.library().lib, name), name


@pytest.mark.parametrize("struct,cls", [
    ("lowm_kv_cache", cache.KvCacheArg), ("lowm_sequences", cache.SequencesArg),
    ("lowm_rotary_args", cache.RotaryArgs), ("lowm_cache_append_args", cache.CacheAppendArgs),
    ("lowm_cache_read_args", cache.CacheReadArgs),
    ("lowm_cache_attention_args", cache.CacheAttentionArgs),
    ("lowm_fork_pages_args", cache.ForkPagesArgs),
    ("lowm_compact_pages_args", cache.CompactPagesArgs)])
def test_structs_are_the_headers(struct, cls):
    body = re.search(r"typedef struct %s \{(.*?)\}" % struct, header(), re.S).group(1)
    names = []
    for line in body.split(";"):
        words = line.replace("*", " ").replace(",", " ").split()
        names += [w for w in words if w not in ("const", "void", "float", "double", "int32_t",
                                                "int64_t", "size_t", "lowm_kv_cache",
                                                "lowm_sequences")]
    assert names == [f[0] for f in cls._fields_]


def test_public_names():
    for name in ("KVCache", "make_kv_cache", "rotary_frequencies", "rotary", "cache_append",
                 "cache_read", "cache_attention", "make_cache_attention_workspace", "fork_pages",
                 "compact_pages", "make_pages_workspace"):
        assert name in sbg.__all__ and callable(getattr(sbg, name))
        assert getattr(sbg, name).__doc__
