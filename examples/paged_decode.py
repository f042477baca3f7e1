"""A decode step's attention layers over a paged 8-bit cache, as they are used together.

    python examples/paged_decode.py [--beams 6] [--hidden 512] [--layers 2] [--steps 80] ...

Per step, for one token of each beam:

    table, lens = fork_pages(parents, reserve=1)     beams reordered, a page where one is full
    for each layer:
        q, k, v  = gemm_batched([x, x, x], [Wq, Wk, Wv])
        q, k     = rotary(q, k, positions)
        cache_append(k, v)                           quantised into the beams' pages
        y        = cache_attention(q)
        x        = x + gemm(y, Wo)

The step is captured into a HIP graph once and replayed with other inputs, parents and lengths;
every buffer and workspace is made beforehand.  A beam whose parent is -1 ends: it has no tokens,
its pages are free and its row of the result is x as it came, until it goes on as another's or
its own.  Now and then compact_pages moves the pages in use together.  Weights are random.
"""
from __future__ import annotations

import argparse
import sys
from pathlib import Path

import torch

sys.path.insert(0, str(Path(__file__).resolve().parents[1]))
import split_bf16_gemm_amd as sbg  # noqa: E402


class PagedDecode:
    def __init__(self, beams: int, hidden: int, heads: int, kv_heads: int, head_dim: int,
                 layers: int, most: int, pages: int, dtype=torch.int8, seed: int = 0,
                 device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def randn(*shape, std=1.0):
            return (torch.randn(*shape, generator=g, device=device) * std).to(torch.bfloat16)

        self.shape = (beams, hidden, heads, kv_heads, head_dim)
        self.sizes = [heads * head_dim, kv_heads * head_dim, kv_heads * head_dim]
        self.weights = [([randn(n, hidden, std=hidden ** -0.5) for n in self.sizes],
                         randn(hidden, heads * head_dim, std=(heads * head_dim) ** -0.5))
                        for _ in range(layers)]
        self.cache = sbg.make_kv_cache(pages, kv_heads, head_dim, layers=layers, dtype=dtype,
                                       device=device)
        self.freqs = sbg.rotary_frequencies(head_dim, device=device)
        width = -(-most // 64)
        self.table = torch.full((beams, width), -1, dtype=torch.int32, device=device)
        self.lens = torch.zeros(beams, dtype=torch.int32, device=device)
        self.parents = torch.arange(beams, dtype=torch.int32, device=device)
        self.positions = torch.zeros(beams, dtype=torch.int32, device=device)
        self.forked = (torch.empty_like(self.table), torch.empty_like(self.lens),
                       torch.empty(pages, dtype=torch.int32, device=device),
                       torch.zeros(1, dtype=torch.int32, device=device))
        self.missing = torch.zeros(1, dtype=torch.int32, device=device)     # over all steps
        self.x = torch.zeros(beams, hidden, dtype=torch.bfloat16, device=device)
        self.attended = torch.zeros(layers, beams, heads, head_dim, dtype=torch.bfloat16,
                                    device=device)
        self.queries = torch.zeros_like(self.attended)
        self.result = torch.zeros_like(self.x)
        self.ws_pages = sbg.make_pages_workspace(beams, width, pages, device)
        self.ws_attention = sbg.make_cache_attention_workspace(beams, heads, kv_heads, head_dim,
                                                               device)

    def step(self):
        """One token of every beam: self.x to self.result."""
        beams, hidden, heads, kv_heads, head_dim = self.shape
        sbg.fork_pages(self.cache, self.table, self.lens, self.parents, reserve=1,
                       workspace=self.ws_pages, outs=self.forked)
        self.table.copy_(self.forked[0])
        self.missing.add_(self.forked[3])
        self.positions.copy_(self.forked[1])
        # a token for every beam that goes on
        torch.add(self.forked[1], self.parents.ge(0), out=self.lens)
        x = self.x
        for i, (wqkv, wo) in enumerate(self.weights):
            layer = self.cache.layer(i)
            q, k, v = (y.view(beams, -1, head_dim)
                       for y in sbg.gemm_batched([x, x, x], wqkv, 1, workspace=None))
            sbg.rotary(q, k, self.positions, self.freqs, q_out=self.queries[i], k_out=k)
            sbg.cache_append(k, v, layer, self.table, self.lens)
            sbg.cache_attention(self.queries[i], layer, self.table, self.lens,
                                workspace=self.ws_attention, out=self.attended[i])
            x = x + sbg.gemm(self.attended[i].view(beams, -1), wo, 1)
        self.result.copy_(x)

    def reset(self):
        self.table.fill_(-1)
        self.lens.zero_()
        self.missing.zero_()
        self.parents.copy_(torch.arange(self.shape[0]))

    def capture(self) -> torch.cuda.CUDAGraph:
        """The step as a graph; the sequences begin anew."""
        self.step()
        self.reset()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            self.step()
        return graph

    def compact(self) -> int:
        """Moves the pages in use to the lowest numbers; how many there then are."""
        table, _, counts = sbg.compact_pages(self.cache, self.table, workspace=self.ws_pages)
        self.table.copy_(table)
        return int(counts[1])


def main():
    ap = argparse.ArgumentParser()
    ap.add_argument("--beams", type=int, default=6)
    ap.add_argument("--hidden", type=int, default=512)
    ap.add_argument("--heads", type=int, default=8)
    ap.add_argument("--kv-heads", type=int, default=2)
    ap.add_argument("--head-dim", type=int, default=64)
    ap.add_argument("--layers", type=int, default=2)
    ap.add_argument("--steps", type=int, default=80)
    ap.add_argument("--e4m3", action="store_true")
    args = ap.parse_args()
    run = PagedDecode(args.beams, args.hidden, args.heads, args.kv_heads, args.head_dim,
                      args.layers, args.steps, 4 * args.beams * (-(-args.steps // 64) + 1),
                      torch.float8_e4m3fn if args.e4m3 else torch.int8)
    graph = run.capture()
    g = torch.Generator().manual_seed(1)
    parents = torch.arange(args.beams)
    for i in range(args.steps):
        run.x.copy_(torch.randn(args.beams, args.hidden, generator=g).to(torch.bfloat16))
        # each goes on, and where beams are reordered, as another, anew (as one that has ended), or
        # not at all
        parents = torch.arange(args.beams).where(parents >= 0, -1)
        if i % 10 == 9:
            parents = torch.randint(-1, args.beams, (args.beams,), generator=g)
        run.parents.copy_(parents)
        graph.replay()
        if i % 40 == 39:
            print(f"step {i + 1}: pages in use end at {run.compact()}")
    torch.cuda.synchronize()
    print(f"{args.steps} steps, lengths {run.lens.tolist()}, missing pages "
          f"{int(run.missing)}, output norm {run.result.float().norm():.3f}")


if __name__ == "__main__":
    main()
