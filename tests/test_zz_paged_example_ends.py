"""The paged example (examples/paged_decode.py) with sequences that end and begin anew, and with too
few pages."""
from __future__ import annotations

import math
import sys

import pytest
import torch

import test_zz_paged_example as example
from test_zz_paged_example import contents

sys.path.insert(0, str(example.ROOT / "examples"))


@pytest.mark.gpu
@pytest.mark.parametrize("beams,heads,kv_heads,head_dim,dtype", [
    (5, 8, 2, 48, torch.float8_e4m3fn), (7, 6, 1, 128, torch.int8)])
def test_sequences_that_end_and_begin_anew(beams, heads, kv_heads, head_dim, dtype):
    """Replayed and eager; a host's count of the lengths; no page lacking; the last step's attention
    against 64 bits (out rounded to bf16, 2^-8, and weights to fp16, 2^-11)."""
    from paged_decode import PagedDecode
    hidden, layers, steps = 256, 2, 140
    make = lambda: PagedDecode(beams, hidden, heads, kv_heads, head_dim, layers, steps + 1,  # noqa
                               8 * beams, dtype)
    eager, graphed = make(), make()
    graph = graphed.capture()
    g = torch.Generator().manual_seed(beams)
    parents, lens, ended, anew = torch.arange(beams), [0] * beams, 0, 0
    for i in range(steps):
        x = torch.randn(beams, hidden, generator=g).to(torch.bfloat16)
        parents = torch.arange(beams).where(parents >= 0, -1)
        if i % 7 == 6:
            parents = torch.randint(-1, beams, (beams,), generator=g)
        anew += sum(lens[p] == 0 and p >= 0 for p in parents.tolist()) if i else 0
        lens = [lens[p] + 1 if p >= 0 else 0 for p in parents.tolist()]
        ended += lens.count(0)
        for run in (eager, graphed):
            run.x.copy_(x)
            run.parents.copy_(parents)
        eager.step()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(eager.result, graphed.result), i
        assert torch.equal(eager.attended, graphed.attended)
        assert eager.lens.tolist() == graphed.lens.tolist() == lens
        for b in range(beams):
            if lens[b] == 0:
                assert not eager.attended[:, b].any()
                assert torch.equal(eager.result[b].cpu(), x[b])
                assert (eager.table[b] == -1).all()
        if i % 30 == 29:
            graphed.compact()
    assert int(eager.missing) == int(graphed.missing) == 0
    assert ended > 10 and anew > 0 and max(lens) > 0
    for layer in range(layers):
        for b in range(beams):
            if lens[b] == 0:
                continue
            k, v = contents(eager.cache.layer(layer), eager.table[b], lens[b])
            q = eager.queries[layer, b].double().cpu()
            for h in range(heads):
                kv = h * kv_heads // heads
                w = torch.softmax(k[:, kv] @ q[h] / math.sqrt(head_dim), 0)
                want = w @ v[:, kv]
                slack = 2.0 ** -8 * want.abs() + 2.0 ** -10 * (w @ v[:, kv].abs())
                got = eager.attended[layer, b, h].double().cpu()
                assert bool(((got - want).abs() <= slack).all())


@pytest.mark.gpu
def test_pages_that_lacked_at_any_step_are_counted():
    """One page for two beams: the second's is missing at each of the steps.  When the first has
    ended, the second begins anew with its page, and nothing is missing in that last step."""
    from paged_decode import PagedDecode
    run = PagedDecode(2, 64, 2, 1, 16, 1, 64, 1)
    for _ in range(5):
        run.step()
    run.parents.copy_(torch.tensor([-1, -1]))
    run.step()
    run.parents.copy_(torch.tensor([-1, 1]))
    run.step()
    assert int(run.forked[3]) == 0 and int(run.missing) == 5 and run.lens.tolist() == [0, 1]
