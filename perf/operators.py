"""The operators that stand next to the low-M GEMM in a decode step, as cases to measure.

Four operators: the residual norm at a block's border, the int8 product of a few rows, a
mixture-of-experts layer for a few tokens, and the log probabilities of given tokens.  Where
``own`` is false, ``run`` computes them with elementary torch operations in 32 bits; where it is
true it calls this package.
"""
import math

import torch

own = False

DEV = "cuda"
BF16, F32 = torch.bfloat16, torch.float32


def listed():
    return [
        # one token of a decode step: the border between two blocks, latency counts
        norm("norm_m1_d4096", 1, 4096),
        # a small decode batch whose next product runs in int8, an fp32 residual stream, a learned
        # gate per channel
        norm("norm_m48_d6144_i8", 48, 6144, res="f32", gate="channel", i8=True),
        # a long prompt with a gate for every token and channel
        norm("norm_m16384_d4096", 16384, 4096, gate="element", alpha=0.875),
        # one token through an attention-output-sized projection, activations quantised in the call
        i8("i8_m1_n6144_k4096", 1, 6144, 4096),
        # an odd decode batch through a long-K projection, activations already in int8
        i8("i8_m23_n2304_k12288", 23, 2304, 12288, given=True),
        # the largest: a full decode batch through a vocabulary-sized projection
        i8("i8_m64_n49152_k4096", 64, 49152, 4096),
        # one token, few wide experts
        moe("moe_t1_d4096_i1024_e64_k4", 1, 4096, 1024, 64, 4),
        # an odd batch over many small experts, sigmoid scores with a selection bias
        moe("moe_t13_d2048_i768_e128_k8", 13, 2048, 768, 128, 8, score="sigmoid"),
        # a full decode batch that touches nearly every expert
        moe("moe_t64_d4096_i1024_e128_k8", 64, 4096, 1024, 128, 8),
        # one sampled token's log probability and its alternatives
        logp("logp_m1_v49152_n5", 1, 49152, 5),
        # a decode batch over fp32 logits of an odd vocabulary, the most alternatives
        logp("logp_m61_v50001_n20_f32", 61, 50001, 20, "f32"),
        # scoring a prompt
        logp("logp_m2048_v49152_n5", 2048, 49152, 5),
    ]


def norm(name, m, d, res="bf16", gate="none", i8=False, alpha=1.0, center=False):
    return {"name": name, "op": "norm", "m": m, "d": d, "res": res, "gate": gate, "i8": i8,
            "alpha": alpha, "center": center}


def i8(name, m, n, k, given=False):
    return {"name": name, "op": "i8", "m": m, "n": n, "k": k, "given": given}


def moe(name, t, d, i, e, k, score="softmax"):
    return {"name": name, "op": "moe", "t": t, "d": d, "i": i, "e": e, "k": k, "score": score}


def logp(name, m, v, n, dtype="bf16"):
    return {"name": name, "op": "logp", "m": m, "v": v, "n": n, "dtype": dtype}


def _log(rng, lo, hi, step=1):
    x = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(x / step)) * step))


def draw(rng):
    op = rng.choice(["norm", "i8", "moe", "logp"])
    if op == "norm":
        c = norm("", _log(rng, 1, 16384), _log(rng, 256, 4096, rng.choice([1, 8, 8])),
                 rng.choice(["bf16", "f32"]), rng.choice(["none", "channel", "token", "element"]),
                 rng.random() < 0.4, rng.choice([1.0, 0.875, 0.5]), rng.random() < 0.3)
    elif op == "i8":
        c = i8("", _log(rng, 1, 64), _log(rng, 256, 16384), _log(rng, 512, 12288, 16),
               rng.random() < 0.5)
    elif op == "moe":
        e = rng.choice([8, 20, 32, 64, 128])
        c = moe("", _log(rng, 1, 64), _log(rng, 512, 4096, 8), _log(rng, 128, 1024, 8), e,
                rng.randint(1, 8), rng.choice(["softmax", "sigmoid"]))
    else:
        c = logp("", _log(rng, 1, 1024), _log(rng, 1000, 98304), rng.randint(0, 20),
                 rng.choice(["bf16", "f32"]))
        c["m"] = min(c["m"], 40_000_000 // c["v"])
    del c["name"]
    return c


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)

    def randn(*shape, dtype=BF16, std=1.0):
        return torch.randn(*shape, generator=g, device=DEV, dtype=dtype).mul_(std)

    def empty(*shape, dtype=F32):
        return torch.empty(*shape, device=DEV, dtype=dtype)

    s = dict(case)
    op = case["op"]
    if op == "norm":
        m, d = case["m"], case["d"]
        res = F32 if case["res"] == "f32" else BF16
        s["y"] = randn(m, d)
        s["r"] = randn(m, d, dtype=F32, std=3.0).to(res)
        s["w_post"] = (1 + randn(d, dtype=F32, std=0.1)).to(BF16)
        s["w_pre"] = (1 + randn(d, dtype=F32, std=0.1)).to(BF16)
        shape = {"none": None, "channel": (d,), "token": (m, 1), "element": (m, d)}[case["gate"]]
        s["g"] = None if shape is None else randn(*shape, std=0.5)
        s["r_out"] = empty(m, d, dtype=res)
        s["x_out"] = empty(m, d, dtype=torch.int8 if case["i8"] else BF16)
        s["s_out"] = empty(m) if case["i8"] else None
        s["stands_for"] = empty(m, d, dtype=BF16) if case["i8"] else None
    elif op == "i8":
        m, n, k = case["m"], case["n"], case["k"]
        x = randn(m, k)
        s["W"] = torch.randint(-127, 128, (n, k), generator=g, device=DEV, dtype=torch.int8)
        s["sw"] = torch.rand(n, generator=g, device=DEV) * 2e-4 + 2e-4
        s["a"], s["sa"] = x, None
        if case["given"]:
            s["a"] = torch.randint(-127, 128, (m, k), generator=g, device=DEV, dtype=torch.int8)
            s["sa"] = torch.rand(m, generator=g, device=DEV) * 0.01 + 0.02
        s["out"] = empty(m, n, dtype=BF16)
        s["ws"] = None if not own else _sbg().make_gemm_i8_workspace(m, n, k)
    elif op == "moe":
        t, d, i, e, k = (case[x] for x in ("t", "d", "i", "e", "k"))
        s["x"] = randn(t, d)
        s["wr"] = randn(e, d, std=0.02)
        s["w13"] = randn(e, 2 * i, d, std=0.02)
        s["w2"] = randn(e, d, i, std=0.02)
        sig = case["score"] == "sigmoid"
        s["bias"] = randn(e, dtype=F32, std=0.1) if sig else None
        s["scale"] = 2.5 if sig else 1.0
        s["out"] = empty(t, d, dtype=BF16)
        s["ids"], s["gates"] = empty(t, k, dtype=torch.int32), empty(t, k)
        s["ws"] = None if not own else _sbg().make_moe_workspace(t, d, i, e, k)
    else:
        m, v, n = case["m"], case["v"], case["n"]
        x = randn(m, v, dtype=F32, std=3.0)
        # a tenth of the vocabulary is masked away, as by a grammar or a list of banned tokens
        banned = torch.rand(v, generator=g, device=DEV) < 0.1
        banned[:32] = False
        x.masked_fill_(banned, -math.inf)
        s["x"] = x if case["dtype"] == "f32" else x.to(BF16)
        s["tok"] = torch.randint(0, 32, (m,), generator=g, device=DEV)
        s["outs"] = (empty(m), empty(m), empty(m, dtype=torch.int32),
                     empty(m, n), empty(m, n, dtype=torch.int32))
        s["ws"] = None if not own else _sbg().make_token_logprobs_workspace(m, v, n)
    return s


def run(s):
    return (RUN_OWN if own else RUN_PLAIN)[s["op"]](s)


# ---------------------------------------------------------------------------------------------
# this package's calls
# ---------------------------------------------------------------------------------------------
def _sbg():
    import split_bf16_gemm_amd
    return split_bf16_gemm_amd


def own_norm(s):
    r, x, sx = _sbg().residual_norm(
        s["y"], s["r"], post_weight=s["w_post"], pre_weight=s["w_pre"], gate=s["g"],
        residual_scale=s["alpha"], center=s["center"], quantize=s["i8"],
        residual_out=s["r_out"], out=s["x_out"], scale_out=s["s_out"])
    # an int8 row stands for its values times the row's scale
    return (r, torch.mul(x, sx[:, None], out=s["stands_for"]), sx) if s["i8"] else (r, x)


def own_i8(s):
    return _sbg().gemm_i8(s["a"], s["W"], s["sw"], a_scale=s["sa"], out=s["out"],
                          workspace=s["ws"])


def own_moe(s):
    return _sbg().moe(s["x"], s["wr"], s["w13"], s["w2"], s["k"], score=s["score"],
                      bias=s["bias"], routed_scale=s["scale"], workspace=s["ws"], out=s["out"],
                      ids_out=s["ids"], gates_out=s["gates"])


def own_logp(s):
    return _sbg().token_logprobs(s["x"], s["tok"], s["n"], workspace=s["ws"], outs=s["outs"])


# ---------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------
EPS = 1e-6


def plain_normalise(v, center):
    if center:
        v = v - v.mean(-1, keepdim=True)
    return v / torch.sqrt((v * v).mean(-1, keepdim=True) + EPS)


def plain_quantise(v):
    scale = v.abs().amax(-1, keepdim=True) / 127
    return torch.round(v / scale), scale


def plain_norm(s):
    p = plain_normalise(s["y"].float(), s["center"]) * s["w_post"].float()
    if s["g"] is not None:
        p = p * s["g"].float()
    r = s["alpha"] * s["r"].float() + p
    x = plain_normalise(r, s["center"]) * s["w_pre"].float()
    if s["i8"]:
        q, scale = plain_quantise(x)
        return r.to(s["r"].dtype), (q * scale).to(BF16), scale[:, 0]
    return r.to(s["r"].dtype), x.to(BF16)


def plain_i8(s):
    if s["given"]:
        q, scale = s["a"].float(), s["sa"][:, None]
    else:
        q, scale = plain_quantise(s["a"].float())
    return (q @ s["W"].float().t() * scale * s["sw"]).to(BF16)


def plain_moe(s):
    t, d, i, e, k = (s[x] for x in ("t", "d", "i", "e", "k"))
    # scores next to the border of the k best lie closer than 32 bits tell apart
    logits = s["x"].double() @ s["wr"].double().t()
    if s["score"] == "sigmoid":
        score = torch.sigmoid(logits)
        ids = torch.topk(score + s["bias"], k).indices
    else:
        score = torch.softmax(logits, -1)
        ids = torch.topk(logits, k).indices
    gates = score.gather(1, ids)
    gates = (gates / gates.sum(-1, keepdim=True) * s["scale"]).float()
    x = s["x"].float()
    if t * k <= e:   # few pairs: each with its own expert's weights
        h = s["w13"][ids].float() @ x[:, None, :, None]              # [t, k, 2i, 1]
        h = h[:, :, :i] * torch.sigmoid(h[:, :, :i]) * h[:, :, i:]
        y = (s["w2"][ids].float() @ h)[..., 0]                       # [t, k, d]
        out = (y * gates[..., None]).sum(1)
    else:            # every expert on every token, then each token's own ones
        h = x @ s["w13"].float().transpose(1, 2).contiguous()        # [e, t, 2i]
        h = h[..., :i] * torch.sigmoid(h[..., :i]) * h[..., i:]
        share = torch.zeros(t, e, device=x.device).scatter_(1, ids, gates)
        h = h * share.t()[..., None]
        out = (h @ s["w2"].float().transpose(1, 2).contiguous()).sum(0)
    return out.to(BF16), ids.to(torch.int32), gates


def plain_logp(s):
    x, v = s["x"].float(), s["v"]
    lz = torch.log(torch.exp(x - x.amax(-1, keepdim=True)).sum(-1, keepdim=True))
    lp = x - x.amax(-1, keepdim=True) - lz
    p = torch.exp(lp)
    entropy = -torch.where(p > 0, p * lp, 0).sum(-1)
    own_x = x.gather(1, s["tok"][:, None])
    rank = (x > own_x).sum(-1).to(torch.int32)
    # whole-number keys in the order of the values, the lower index first among equal ones
    bits = (x + 0.0).view(torch.int32)
    key = (bits ^ ((bits >> 31) & 0x7fffffff)).long() * 2 ** 32
    key = key + (v - 1 - torch.arange(v, device=x.device))
    ids = torch.topk(key, s["n"]).indices
    return (lp.gather(1, s["tok"][:, None])[:, 0], entropy, rank, lp.gather(1, ids),
            ids.to(torch.int32))


RUN_OWN = {"norm": own_norm, "i8": own_i8, "moe": own_moe, "logp": own_logp}
RUN_PLAIN = {"norm": plain_norm, "i8": plain_i8, "moe": plain_moe, "logp": plain_logp}


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without, and what it means in 64 bits
# ---------------------------------------------------------------------------------------------
def work(case):
    op = case["op"]
    if op == "norm":
        m, d = case["m"], case["d"]
        res = 4 if case["res"] == "f32" else 2
        gate = {"none": 0, "channel": 2 * d, "token": 2 * m, "element": 2 * m * d}[case["gate"]]
        return {"bytes": m * d * (2 + 2 * res + (1 if case["i8"] else 2)) + 4 * d + gate
                + (4 * m if case["i8"] else 0), "flops": 16 * m * d}
    if op == "i8":
        m, n, k = case["m"], case["n"], case["k"]
        return {"bytes": n * k + m * k * (1 if case["given"] else 2) + 2 * m * n + 4 * n
                + (4 * m if case["given"] else 0), "flops": 2 * m * n * k}
    if op == "moe":
        t, d, i, e, k = (case[x] for x in ("t", "d", "i", "e", "k"))
        # experts that t independent choices of k of e reach, on average
        active = e * (1 - (1 - min(k, e) / e) ** t)
        return {"bytes": active * 6 * d * i + 2 * e * d + 4 * t * d + 8 * t * k,
                "flops": 6 * t * k * d * i + 2 * t * e * d}
    m, v, n = case["m"], case["v"], case["n"]
    return {"bytes": m * v * (4 if case["dtype"] == "f32" else 2) + m * (20 + 8 * n),
            "flops": 6 * m * v}


def exact(case, seed):
    s = prepare(case, seed)
    return EXACT[case["op"]](s)


def exact_norm(s):
    y = s["y"].double()
    w = s["w_post"].double()

    def unit(z):
        if s["center"]:
            mean = z.sum(1) / s["d"]
            z = z - mean[:, None]
        power = torch.linalg.vector_norm(z, dim=1) ** 2 / s["d"]
        return z * torch.rsqrt(power + EPS)[:, None]

    branch = unit(y) * w
    if s["g"] is not None:
        branch *= s["g"].double()
    r = s["r"].double() * s["alpha"] + branch
    x = unit(r) * s["w_pre"].double()
    if not s["i8"]:
        return r, x
    top = torch.maximum(x.max(1).values, -x.min(1).values)
    levels = (x * (127 / top)[:, None]).round().clamp(-127, 127)
    return r, levels * (top / 127)[:, None], top / 127


def exact_i8(s):
    a = s["a"].double()
    if s["given"]:
        step = s["sa"].double()
    else:
        step = torch.linalg.vector_norm(a, ord=math.inf, dim=1) / 127
        a = (a / step[:, None]).round()
    out = torch.empty(s["m"], s["n"], dtype=torch.float64, device=a.device)
    for c in range(0, s["n"], 4096):
        out[:, c:c + 4096] = a @ s["W"][c:c + 4096].double().t()
    return out * torch.outer(step, s["sw"].double())


def exact_moe(s):
    x = s["x"].double()
    z = x @ s["wr"].double().t()
    if s["score"] == "sigmoid":
        score = 1 / (1 + torch.exp(-z))
        order = score + s["bias"].double()
    else:
        score = torch.exp(z - torch.logsumexp(z, 1, keepdim=True))
        order = z
    ids = torch.sort(order, dim=1, descending=True, stable=True).indices[:, :s["k"]]
    share = torch.gather(score, 1, ids)
    share = s["scale"] * share / share.sum(1, keepdim=True)
    out = torch.zeros_like(x)
    for e in torch.unique(ids).tolist():
        rows, slot = (ids == e).nonzero(as_tuple=True)
        gate, up = (x[rows] @ s["w13"][e].double().t()).split(s["i"], 1)
        h = gate / (1 + torch.exp(-gate)) * up
        out[rows] += share[rows, slot][:, None] * (h @ s["w2"][e].double().t())
    return out, ids.to(torch.int32), share


def exact_logp(s):
    parts = []
    for r in range(0, s["m"], 256):
        z = s["x"][r:r + 256].double()
        z = z - torch.logsumexp(z, 1, keepdim=True)
        tok = s["tok"][r:r + 256]
        mine = z[torch.arange(len(z), device=z.device), tok]
        h = torch.special.entr(torch.exp(z)).sum(1)
        ahead = (s["x"][r:r + 256] > s["x"][r:r + 256].gather(1, tok[:, None])).sum(1)
        top, ids = torch.sort(z, dim=1, descending=True, stable=True)
        parts.append((mine, h, ahead.int(), top[:, :s["n"]], ids[:, :s["n"]].int()))
    return tuple(torch.cat(p) for p in zip(*parts))


EXACT = {"norm": exact_norm, "i8": exact_i8, "moe": exact_moe, "logp": exact_logp}
