"""One decode step's work around the attention: the operators of this package as
they are used together.

    python examples/decode_block.py [--tokens 4] [--hidden 4096] ...

For a few tokens, from the attention's output y and the residual stream r:

    r, q, s  = residual_norm(y, r, quantize)        norm, gate, residual; int8 rows
    y        = gemm_i8(q, W, ...)                   a dense projection in int8
    r, x, _  = residual_norm(y, r)
    y        = moe(x, ...)                          the experts
    r, x, _  = residual_norm(y, r)
    logits   = gemm(x, head)                        the low-M bf16 product
    logprob, entropy, rank, alternatives = token_logprobs(logits, tokens)

The step is captured into a HIP graph once and replayed, as a server would; every
buffer and workspace is made beforehand.  Weights are random.
"""
from __future__ import annotations

import argparse
import sys
from pathlib import Path

import torch

sys.path.insert(0, str(Path(__file__).resolve().parents[1]))
import split_bf16_gemm_amd as sbg  # noqa: E402


class DecodeBlock:
    def __init__(self, tokens: int, hidden: int, inner: int, experts: int, top_k: int, vocab: int,
                 top_n: int = 5, seed: int = 0, device="cuda"):
        g = torch.Generator(device=device)
        g.manual_seed(seed)

        def randn(*shape, std=1.0, dtype=torch.bfloat16):
            return (torch.randn(*shape, generator=g, device=device) * std).to(dtype)

        self.top_k, self.top_n = top_k, top_n
        std = hidden ** -0.5
        self.norms = [1 + randn(hidden, std=0.1) for _ in range(6)]
        self.gate = randn(hidden, std=0.5)
        # a dense projection, quantised once: a scale for each output column
        self.W, self.w_scale = sbg.quantize_rows(randn(hidden, hidden, std=std))
        self.router = randn(experts, hidden, std=std)
        self.w13 = randn(experts, 2 * inner, hidden, std=std)
        self.w2 = randn(experts, hidden, inner, std=inner ** -0.5)
        self.head = randn(vocab, hidden, std=std)

        self.y = randn(tokens, hidden)
        self.r = randn(tokens, hidden, dtype=torch.float32)
        self.tokens = torch.randint(0, vocab, (tokens,), generator=g, device=device)

        self.split_k = sbg.pick_split_k(tokens, vocab, hidden)
        self.ws_i8 = sbg.make_gemm_i8_workspace(tokens, hidden, hidden, device)
        self.ws_moe = sbg.make_moe_workspace(tokens, hidden, inner, experts, top_k, device)
        self.ws_head = sbg.make_workspace(tokens, vocab, hidden, self.split_k, device)
        self.ws_logprobs = sbg.make_token_logprobs_workspace(tokens, vocab, top_n, device)

    def step(self):
        """The step on the current stream; its outputs by name."""
        n = self.norms
        r1, q, s = sbg.residual_norm(self.y, self.r, post_weight=n[0], pre_weight=n[1],
                                     gate=self.gate, quantize=True)
        dense = sbg.gemm_i8(q, self.W, self.w_scale, a_scale=s, workspace=self.ws_i8)
        r2, x2, _ = sbg.residual_norm(dense, r1, post_weight=n[2], pre_weight=n[3],
                                      residual_out=r1)
        mixed, ids, gates = sbg.moe(x2, self.router, self.w13, self.w2, self.top_k,
                                    workspace=self.ws_moe)
        r3, x3, _ = sbg.residual_norm(mixed, r2, post_weight=n[4], pre_weight=n[5],
                                      residual_out=r2)
        logits = sbg.gemm(x3, self.head, self.split_k, workspace=self.ws_head)
        logprob, entropy, rank, top, top_ids = sbg.token_logprobs(
            logits, self.tokens, self.top_n, workspace=self.ws_logprobs)
        return {"q": q, "scale": s, "dense": dense, "x2": x2, "ids": ids, "gates": gates,
                "mixed": mixed, "residual": r3, "x3": x3, "logits": logits, "logprob": logprob,
                "entropy": entropy, "rank": rank, "top": top, "top_ids": top_ids}

    def capture(self):
        """(graph, outputs): the step as a HIP graph."""
        self.step()                       # load the kernels outside the capture
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            outputs = self.step()
        return graph, outputs


def main():
    p = argparse.ArgumentParser(description=__doc__.splitlines()[0])
    for name, default in (("tokens", 4), ("hidden", 4096), ("inner", 1024), ("experts", 64),
                          ("top-k", 4), ("vocab", 49152), ("steps", 50)):
        p.add_argument(f"--{name}", type=int, default=default)
    a = p.parse_args()
    block = DecodeBlock(a.tokens, a.hidden, a.inner, a.experts, a.top_k, a.vocab)
    graph, out = block.capture()
    graph.replay()
    start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
    start.record()
    for _ in range(a.steps):
        graph.replay()
    end.record()
    torch.cuda.synchronize()
    print(f"{a.tokens} tokens, hidden {a.hidden}, {a.experts} experts of {a.inner}, "
          f"vocabulary {a.vocab}: {start.elapsed_time(end) * 1e3 / a.steps:.1f} us a step")
    for t in range(min(a.tokens, 4)):
        print(f"  token {int(block.tokens[t])}: log p {out['logprob'][t]:.3f}, rank "
              f"{int(out['rank'][t])}, entropy {out['entropy'][t]:.3f}, most likely "
              f"{out['top_ids'][t].tolist()}")


if __name__ == "__main__":
    main()
