"""The attention part of a decode step and the 8-bit cache that it reads, as cases to measure.

Five operators: rotary positions for the queries and keys of a step, appending keys and values to
a paged cache held in 8 bits with a scale for each page of 64 tokens and head (and reading it
back), attention over that cache, forking the cache's sequences (with freeing and reserving their
pages), and compacting its pages.  Where ``own`` is false, ``run`` computes them with elementary
torch operations in 32 bits; where it is true it calls this package.
"""
import math
import random

import torch

own = False

DEV = "cuda"
BF16, F32, I32 = torch.bfloat16, torch.float32, torch.int32
FP8 = torch.float8_e4m3fn
PAGE = 64


def listed():
    return [
        # one token of a decode step: 32 query and 8 key heads, latency counts
        rot("rotary_t1_h32_8_d128", 1, 32, 8, 128, 128),
        # a long prompt, pairs side by side, half of each head, positions far out, cosines scaled
        rot("rotary_t8192_h64_8_d128_r64", 8192, 64, 8, 128, 64, layout="interleaved", far=1 << 20,
            scale=1.25),
        # an odd decode batch: one token a sequence, at any place in its page
        app("append_b61_n1_h8_d128", 61, 1, 2000, 8, 128, spread=1),
        # two prompts at once, after a cached beginning, e4m3
        app("append_b2_n4100_h8_d128_e4m3", 2, 4100, 700, 8, 128, spread=2, kind="e4m3"),
        # one token of a short conversation, latency counts
        att("attention_b1_l640_h32_8_d128", 1, 1, 640, 32, 8, 128),
        # an odd decode batch whose sequences are from one token to 16384 long
        att("attention_b61_ragged16384_h64_8_d128", 61, 1, 16384, 64, 8, 128, spread=3),
        # two very long contexts, e4m3
        att("attention_b2_l131001_h64_8_d128_e4m3", 2, 1, 131001, 64, 8, 128, kind="e4m3"),
        # a few sequences with several new tokens each (a piece of a prompt, drafts to verify)
        att("attention_b4_n1to61_l20000_h32_4_d192", 4, 61, 20000, 32, 4, 192, spread=4),
        # eight beams reordered, a page reserved where one is full
        fork("fork_r8_l3", 8, 40, 64, 3, 8, 128, spread=5),
        # a large pool of beams
        fork("fork_r64_l6", 64, 1400, 2048, 6, 8, 128, spread=6),
        # after a few sequences have ended
        comp("compact_r8_p96_l2", 8, 96, 12, 2, 4, 64, spread=7),
        # half of a large pool has been freed
        comp("compact_r48_p1500_l6", 48, 1500, 32, 6, 8, 128, spread=8),
    ]


def rot(name, t, hq, hk, d, r, layout="half", far=8192, scale=1.0, dtype="bf16"):
    return {"name": name, "op": "rot", "t": t, "hq": hq, "hk": hk, "d": d, "r": r,
            "layout": layout, "far": far, "scale": scale, "dtype": dtype}


def app(name, b, n, l, h, d, spread=0, kind="int8"):
    return {"name": name, "op": "app", "b": b, "n": n, "l": l, "h": h, "d": d, "spread": spread,
            "kind": kind}


def att(name, b, n, l, hq, hk, d, window=0, spread=0, kind="int8"):
    return {"name": name, "op": "att", "b": b, "n": n, "l": l, "hq": hq, "hk": hk, "d": d,
            "window": window, "spread": spread, "kind": kind}


def fork(name, r, pages, l, layers, h, d, spread):
    return {"name": name, "op": "fork", "r": r, "pages": pages, "l": l, "layers": layers, "h": h,
            "d": d, "spread": spread}


def comp(name, r, pages, w, layers, h, d, spread):
    return {"name": name, "op": "comp", "r": r, "pages": pages, "w": w, "layers": layers, "h": h,
            "d": d, "spread": spread}


def _log(rng, lo, hi, step=1):
    x = math.exp(rng.uniform(math.log(lo), math.log(hi)))
    return max(lo, min(hi, int(round(x / step)) * step))


def draw(rng):
    op = rng.choice(["rot", "app", "att", "att", "fork", "comp"])
    kind = rng.choice(["int8", "e4m3"])
    spread = rng.randrange(1, 1 << 20)
    hk = rng.choice([1, 2, 4, 8])
    d = rng.choice([64, 80, 96, 128, 128, 192, 256])
    if op == "rot":
        c = rot("", _log(rng, 1, 8192), hk * rng.choice([1, 2, 4, 8]), hk, d,
                rng.choice([d, d, d // 2]), rng.choice(["half", "interleaved"]),
                _log(rng, 64, 1 << 20), rng.choice([1.0, 1.25]), rng.choice(["bf16", "f32"]))
        c["t"] = min(c["t"], 8192 * 72 * 128 // (2 * (c["hq"] + hk) * d))
    elif op == "app":
        b = _log(rng, 1, 64)
        c = app("", b, rng.choice([1, 1, _log(rng, 1, 8192 // b)]), _log(rng, 1, 2000), hk, d,
                spread, kind)
    elif op == "att":
        b = _log(rng, 1, 64)
        n = rng.choice([1, 1, 1, _log(rng, 1, max(1, 64 // b))])
        c = att("", b, n, _log(rng, 1, min(131001, 260000 // b)), hk * rng.randint(1, 8), hk, d,
                rng.choice([0, 0, 0, 1000]), spread, kind)
    elif op == "fork":
        r = _log(rng, 1, 64)
        c = fork("", r, 24 * r + rng.randint(2, 64), _log(rng, 1, 1000), rng.randint(1, 4), hk,
                 d, spread)
    else:
        r = _log(rng, 1, 48)
        c = comp("", r, 2 * r * 8 + rng.randint(1, 200), 16, rng.randint(1, 4), hk, d, spread)
    del c["name"]
    return c


# ---------------------------------------------------------------------------------------------
# the sequences of a case
# ---------------------------------------------------------------------------------------------
def sequences(c):
    """(new tokens, tokens before them) of each sequence of an appending or attending step: equal
    ones without a spread, else lengths spread over their logarithm, and one empty sequence."""
    b, n, l = c["b"], c["n"], c["l"]
    if not c["spread"]:
        return [n] * b, [l - n if c["op"] == "att" else l] * b
    rng = random.Random(c["spread"])
    new = [n if c["op"] == "app" else rng.randint(1, n) for _ in range(b)]
    old = [_log(rng, 1, l) - 1 for _ in range(b)]
    if b > 2:
        new[0], old[0] = n, l - 1
        old[b // 2], new[b // 2] = 0, 1
    return new, old


def pages_of(tokens):
    return -(-tokens // PAGE)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    s = dict(case)
    PREPARE[case["op"]](s, g)
    return s


def randn(g, *shape, dtype=BF16, std=1.0):
    return torch.randn(*shape, generator=g, device=DEV, dtype=dtype).mul_(std)


def bell(g, shape, kind):
    """8-bit values of a bell shape."""
    if kind == "e4m3":
        return randn(g, *shape, std=100.0).clamp_(-448, 448).to(FP8)
    a = torch.randint(-64, 64, shape, generator=g, device=DEV, dtype=torch.int8)
    return a.add_(torch.randint(-63, 64, shape, generator=g, device=DEV, dtype=torch.int8))


def make_pages(s, g, pages, h, d, kind, layers=()):
    """A cache: keys [page][head][D / 16][64][16], values [page][head][4][D][16 tokens] and the
    scales of both."""
    lead = (*layers, pages, h)
    s["ck"] = bell(g, (*lead, d // 16, PAGE, 16), kind)
    s["cv"] = bell(g, (*lead, PAGE // 16, d, 16), kind)
    unit = 0.01 if kind == "e4m3" else 0.02
    s["ks"] = torch.exp(randn(g, *lead, dtype=F32, std=0.2)).mul_(unit)
    s["vs"] = torch.exp(randn(g, *lead, dtype=F32, std=0.2)).mul_(unit)
    if own:
        s["cache"] = _sbg().KVCache(s["ck"], s["cv"], s["ks"], s["vs"])


def make_table(g, counts, width, pages, first=0):
    """Page numbers in no order, -1 past a sequence's last."""
    ids = (torch.randperm(pages - first, generator=g, device=DEV) + first).tolist()
    table = torch.full((len(counts), width), -1, dtype=I32)
    for r, n in enumerate(counts):
        table[r, :n] = torch.tensor(ids[:n], dtype=I32)
        ids = ids[n:]
    return table.to(DEV)


def ints(values):
    return torch.tensor(values, dtype=I32, device=DEV)


def prepare_rot(s, g):
    t, d, r = s["t"], s["d"], s["r"]
    dtype = F32 if s["dtype"] == "f32" else BF16
    # columns of one buffer, as a product over all heads writes them
    qkv = randn(g, t, (s["hq"] + 2 * s["hk"]) * d, dtype=dtype)
    s["q"] = qkv[:, :s["hq"] * d].view(t, s["hq"], d)
    s["k"] = qkv[:, s["hq"] * d:(s["hq"] + s["hk"]) * d].view(t, s["hk"], d)
    s["pos"] = torch.randint(0, s["far"], (t,), generator=g, device=DEV)
    s["freqs"] = 10000.0 ** -(torch.arange(0, r, 2, dtype=torch.float64, device=DEV) / r)
    s["q_out"] = torch.empty(t, s["hq"], d, dtype=dtype, device=DEV)
    s["k_out"] = torch.empty(t, s["hk"], d, dtype=dtype, device=DEV)


def prepare_app(s, g):
    new, old = sequences(s)
    b, h, d = s["b"], s["h"], s["d"]
    lens = [x + y for x, y in zip(new, old)]
    counts = [pages_of(x) for x in lens]
    pages = sum(counts) + 5
    make_pages(s, g, pages, h, d, s["kind"])
    s["table"] = make_table(g, counts, max(counts) + 1, pages, first=1)
    s["lens"] = ints(lens)
    t = sum(new)
    s["starts"] = ints([sum(new[:i]) for i in range(b + 1)])
    kv = randn(g, t, 2 * h * d)
    kv *= torch.exp(randn(g, t, 1, std=0.5))
    s["k"] = kv[:, :h * d].view(t, h, d)
    s["v"] = kv[:, h * d:].view(t, h, d)
    # what comes back: the pages that got tokens
    seen = [x - (y // PAGE) * PAGE for x, y in zip(lens, old)]
    s["seen"] = ints([sum(seen[:i]) for i in range(b + 1)])
    s["k_seen"] = torch.empty(sum(seen), h, d, dtype=BF16, device=DEV)
    s["v_seen"] = torch.empty(sum(seen), h, d, dtype=BF16, device=DEV)
    s["most"] = max(pages_of(x) - y // PAGE for x, y in zip(lens, old))
    s["rows"], s["seen_rows"] = t, sum(seen)


def prepare_att(s, g):
    new, old = sequences(s)
    b, hk, d = s["b"], s["hk"], s["d"]
    lens = [x + y for x, y in zip(new, old)]
    counts = [pages_of(x) for x in lens]
    pages = sum(counts) + 3
    make_pages(s, g, pages, hk, d, s["kind"])
    s["table"] = make_table(g, counts, max(counts), pages)
    s["lens"] = ints(lens)
    t = sum(new)
    s["starts"] = ints([sum(new[:i]) for i in range(b + 1)])
    s["q"] = randn(g, t, s["hq"], d, std=2.0)
    s["out"] = torch.empty(t, s["hq"], d, dtype=BF16, device=DEV)
    s["lse"] = torch.empty(t, s["hq"], dtype=F32, device=DEV)
    s["rows"], s["longest"], s["widest"] = t, max(lens), max(new)
    s["ws"] = _sbg().make_cache_attention_workspace(t, s["hq"], hk, d) if own else None


def fork_shape(c):
    """Tokens of each row and its parent: a tenth of the rows end, a few of the others go on."""
    rng = random.Random(c["spread"])
    r = c["r"]
    lens = [_log(rng, 1, c["l"]) for _ in range(r)]
    kept = rng.sample(range(r), max(1, r // 3))
    parents = [-1 if rng.random() < 0.1 else rng.choice(kept) for _ in range(r)]
    return lens, parents


def prepare_fork(s, g):
    lens, parents = fork_shape(s)
    counts = [pages_of(x) for x in lens]
    width = pages_of(s["l"]) + 2
    # what the rows' pages need, should the pool be smaller: a larger pool
    pages = max(s["pages"], 2 * sum(counts) + 2 * s["r"])
    make_pages(s, g, pages, s["h"], s["d"], "int8", (s["layers"],))
    s["table"] = make_table(g, counts, width, pages)
    s["lens"], s["parents"] = ints(lens), ints(parents)
    s["outs"] = (torch.empty_like(s["table"]), torch.empty_like(s["lens"]),
                 torch.empty(pages, dtype=I32, device=DEV), torch.empty(1, dtype=I32, device=DEV))
    s["ws"] = _sbg().make_pages_workspace(s["r"], width, pages) if own else None


def comp_shape(c):
    rng = random.Random(c["spread"])
    most = min(c["w"], max(1, c["pages"] // c["r"]))
    return [rng.randint(0, most) for _ in range(c["r"])]


def prepare_comp(s, g):
    counts = comp_shape(s)
    make_pages(s, g, s["pages"], s["h"], s["d"], "int8", (s["layers"],))
    s["table"] = make_table(g, counts, s["w"], s["pages"])
    # the pages that two sequences share, from their beginning
    if s["r"] > 1:
        s["table"][1, :1] = s["table"][0, :1]
    s["outs"] = (torch.empty_like(s["table"]), torch.empty(s["pages"], dtype=I32, device=DEV),
                 torch.empty(2, dtype=I32, device=DEV))
    s["ws"] = _sbg().make_pages_workspace(s["r"], s["w"], s["pages"]) if own else None


PREPARE = {"rot": prepare_rot, "app": prepare_app, "att": prepare_att, "fork": prepare_fork,
           "comp": prepare_comp}


def run(s):
    return (RUN_OWN if own else RUN_PLAIN)[s["op"]](s)


# ---------------------------------------------------------------------------------------------
# this package's calls
# ---------------------------------------------------------------------------------------------
def _sbg():
    import split_bf16_gemm_amd
    return split_bf16_gemm_amd


def own_rot(s):
    return _sbg().rotary(s["q"], s["k"], s["pos"], s["freqs"], layout=s["layout"],
                         scale=s["scale"], q_out=s["q_out"], k_out=s["k_out"])


def own_app(s):
    _sbg().cache_append(s["k"], s["v"], s["cache"], s["table"], s["lens"],
                        row_starts=s["starts"])
    # an 8-bit cache stands for its values times their page's scale
    k, v = _sbg().cache_read(s["cache"], s["table"], s["lens"], row_starts=s["seen"],
                             k_out=s["k_seen"], v_out=s["v_seen"])
    return k, v, s["ks"], s["vs"]


def own_att(s):
    return _sbg().cache_attention(s["q"], s["cache"], s["table"], s["lens"],
                                  row_starts=s["starts"], window=s["window"], workspace=s["ws"],
                                  out=s["out"], lse_out=s["lse"])


def own_fork(s):
    outs = _sbg().fork_pages(s["cache"], s["table"], s["lens"], s["parents"], reserve=1,
                             outs=s["outs"], workspace=s["ws"])
    return (*outs, s["ck"], s["cv"], s["ks"], s["vs"])


def own_comp(s):
    outs = _sbg().compact_pages(s["cache"], s["table"], outs=s["outs"], workspace=s["ws"])
    return (*outs, s["ck"], s["cv"], s["ks"], s["vs"])


# ---------------------------------------------------------------------------------------------
# plain forms
# ---------------------------------------------------------------------------------------------
def plain_rot(s):
    turn = s["pos"].double()[:, None] * s["freqs"]
    cos = (torch.cos(turn) * s["scale"]).float()[:, None]
    sin = (torch.sin(turn) * s["scale"]).float()[:, None]

    def rotate(x):
        r = s["r"]
        y = x.float()
        if s["layout"] == "half":
            a, b = y[..., :r // 2], y[..., r // 2:r]
            turned = torch.cat((a * cos - b * sin, a * sin + b * cos), -1)
        else:
            a, b = y[..., :r:2], y[..., 1:r:2]
            turned = torch.stack((a * cos - b * sin, a * sin + b * cos), -1).flatten(-2)
        return torch.cat((turned, y[..., r:]), -1).to(x.dtype)

    return rotate(s["q"]), rotate(s["k"])


def bytes_of(x):
    return x.view(torch.int8)


def values(x, kind):
    """8-bit values, as bytes, in 32 bits."""
    return x.view(FP8).float() if kind == "e4m3" else x.float()


def to_8_bits(x, kind):
    return x.to(FP8).view(torch.int8) if kind == "e4m3" else torch.round(x).to(torch.int8)


def rows_of_k(x):
    """[..., head, D / 16, 64, 16] to [..., 64, head, D]."""
    return x.movedim(-2, -4).flatten(-2)


def rows_of_v(x):
    """[..., head, 4, D, 16 tokens] to [..., 64, head, D]."""
    return x.movedim((-3, -1), (-4, -3)).flatten(-4, -3)


def k_of_rows(x):
    return x.unflatten(-1, (x.shape[-1] // 16, 16)).movedim(-4, -2)


def v_of_rows(x):
    return x.unflatten(-3, (PAGE // 16, 16)).movedim((-4, -3), (-3, -1))


def plain_app(s):
    b, h, d, kind, most = s["b"], s["h"], s["d"], s["kind"], s["most"]
    top = 448.0 if kind == "e4m3" else 127.0
    lens, starts = s["lens"].long(), s["starts"].long()
    new = starts[1:] - starts[:-1]
    old = lens - new
    # the pages that get tokens; page 0 is nobody's and stands for those past a sequence's last
    at = old[:, None] // PAGE + torch.arange(most, device=DEV)
    some = at * PAGE < lens[:, None]
    page = s["table"].long().gather(1, at.clamp(max=s["table"].shape[1] - 1))
    page = torch.where(some, page, 0)
    where = at[..., None] * PAGE + torch.arange(PAGE, device=DEV)          # [b, most, 64]
    fresh = (where >= old[:, None, None]) & (where < lens[:, None, None])
    kept = (where < old[:, None, None])[..., None, None]
    row = (starts[:-1, None, None] + where - old[:, None, None]).clamp(0, s["rows"] - 1)
    begun = (some & (at * PAGE < old[:, None]))[..., None]
    for x, cache, scales, rows_of, of_rows in (
            (s["k"], s["ck"], s["ks"], rows_of_k, k_of_rows),
            (s["v"], s["cv"], s["vs"], rows_of_v, v_of_rows)):
        x = torch.where(fresh[..., None, None], x.float()[row], 0)         # [b, most, 64, h, d]
        before = scales[page]
        scale = x.abs().amax((2, 4)) / top
        scale = torch.where(begun, torch.maximum(scale, before), scale)
        held = bytes_of(cache)[page]
        q = rows_of(held)
        ratio = torch.where(begun, before / scale, 1)[:, :, None, :, None]
        again = to_8_bits(values(q.contiguous(), kind) * ratio, kind)
        fine = torch.where(scale > 0, scale, 1)[:, :, None, :, None]
        put = to_8_bits(x / fine, kind)
        q = torch.where(fresh[..., None, None], put, torch.where(kept, again, q))
        done = torch.where(some[..., None, None, None, None], of_rows(q), held)
        bytes_of(cache)[page] = done
        scales[page] = torch.where(some[..., None], scale, before)
    # what the cache then holds there
    seen = s["seen"].long()
    t = torch.arange(s["seen_rows"], device=DEV)
    seq = torch.searchsorted(seen, t, right=True) - 1
    pos = lens[seq] - (seen[seq + 1] - t)
    page = s["table"].long()[seq, pos // PAGE]
    off = pos % PAGE
    hd = torch.arange(d, device=DEV)[None, None, :]
    hh = torch.arange(h, device=DEV)[None, :, None]
    page, off = page[:, None, None], off[:, None, None]
    k = bytes_of(s["ck"])[page, hh, hd // 16, off, hd % 16]
    v = bytes_of(s["cv"])[page, hh, off // 16, hd, off % 16]
    k = values(k, kind) * s["ks"][page[..., 0], hh[..., 0]][..., None]
    v = values(v, kind) * s["vs"][page[..., 0], hh[..., 0]][..., None]
    return k.to(BF16), v.to(BF16), s["ks"], s["vs"]


def plain_att(s):
    hq, hk, d, kind = s["hq"], s["hk"], s["d"], s["kind"]
    b, group, n = s["b"], hq // hk, s["widest"]
    lens, starts = s["lens"].long(), s["starts"].long()
    new = starts[1:] - starts[:-1]
    page = s["table"].long().clamp(min=0)
    k = values(bytes_of(s["ck"])[page], kind) * s["ks"][page][..., None, None, None]
    k = rows_of_k(k).flatten(1, 2).movedim(2, 1)                           # [b, hk, tokens, d]
    v = values(bytes_of(s["cv"])[page], kind) * s["vs"][page][..., None, None, None]
    v = rows_of_v(v).flatten(1, 2).movedim(2, 1)
    j = torch.arange(n, device=DEV)
    row = (starts[:-1, None] + j).clamp(max=s["rows"] - 1)
    q = s["q"].float()[row].view(b, n, hk, group, d).permute(0, 2, 1, 3, 4)
    x = q.reshape(b, hk, n * group, d) @ k.transpose(2, 3) / math.sqrt(d)
    token = torch.arange(x.shape[-1], device=DEV)
    at = (lens - new)[:, None] + j                                         # [b, n]
    seen = token <= at[..., None]
    if s["window"]:
        seen &= token > at[..., None] - s["window"]
    x = x.view(b, hk, n, group, -1).masked_fill(~seen[:, None, :, None], -math.inf)
    top = x.amax(-1, keepdim=True)
    p = torch.exp(x - top)
    total = p.sum(-1, keepdim=True)
    out = (p.view(b, hk, n * group, -1) @ v).view(b, hk, n, group, d) / total
    lse = (top + torch.log(total))[..., 0]
    t = torch.arange(s["rows"], device=DEV)
    seq = torch.searchsorted(starts, t, right=True) - 1
    nth = t - starts[seq]
    out = out.permute(0, 2, 1, 3, 4).reshape(b, n, hq, d)[seq, nth]
    return out.to(BF16), lse.permute(0, 2, 1, 3).reshape(b, n, hq)[seq, nth]


def copy_plain(s, src, dst):
    for x in (s["ck"], s["cv"], s["ks"], s["vs"]):
        x[:, dst] = x[:, src]


def plain_fork(s):
    table, lens, parents = s["table"].long(), s["lens"].long(), s["parents"].long()
    r, width = table.shape
    pages = s["ck"].shape[1]
    alive = parents >= 0
    parent = parents.clamp(min=0)
    length = torch.where(alive, lens[parent], 0)
    count = (length + PAGE - 1) // PAGE
    w = torch.arange(width, device=DEV)
    out = torch.where(w < count[:, None], table[parent], -1)
    refs = torch.zeros(pages + 1, dtype=torch.long, device=DEV)
    refs.index_add_(0, out.flatten() + 1, torch.ones_like(out).flatten())
    refs = refs[1:].clone()
    # rows that end inside a page: all but the first of those that share it get their own copy
    part = length % PAGE != 0
    last = torch.where(part, out.gather(1, (count - 1).clamp(min=0)[:, None])[:, 0], -1)
    same = (last[:, None] == last[None, :]) & part[None, :]
    first = ~(same & (torch.arange(r, device=DEV)[None, :] < torch.arange(r, device=DEV)[:, None])
              ).any(1)
    own_page = first & (refs[last.clamp(min=0)] == same.sum(1))
    copy = part & ~own_page
    # one more token wants a new page where the last one is full
    more = alive & (length % PAGE == 0)
    fits = count < width
    wants = torch.stack((copy, more & fits), 1)
    rank = torch.cumsum(wants.flatten(), 0).view(r, 2) - 1
    free = torch.sort((refs != 0).int(), stable=True).indices
    n_free = (refs == 0).sum()
    got = wants & (rank < n_free)
    page = torch.where(got, free[rank.clamp(0, pages - 1)], -1)
    missing = (wants & ~got).sum() + (more & ~fits).sum()
    is_last = w == (count - 1)[:, None]
    out = torch.where(is_last & copy[:, None], page[:, :1], out)
    out = torch.where((w == count[:, None]) & (more & fits)[:, None], page[:, 1:], out)
    refs.index_add_(0, last.clamp(min=0), -copy.long())
    refs.index_add_(0, page.clamp(min=0).flatten(), got.long().flatten())
    rows = got[:, 0].nonzero()[:, 0]
    copy_plain(s, last[rows], page[rows, 0])
    return (out.int(), length.int(), refs.int(), missing.int()[None], s["ck"], s["cv"], s["ks"],
            s["vs"])


def plain_comp(s):
    table, pages = s["table"].long(), s["pages"]
    refs = torch.zeros(pages + 1, dtype=torch.long, device=DEV)
    refs.index_add_(0, table.flatten() + 1, torch.ones_like(table).flatten())
    refs = refs[1:].clone()
    # the highest page in use moves to the lowest free one, and so on while that is lower
    free = (refs == 0).nonzero()[:, 0]
    used = (refs != 0).nonzero()[:, 0].flip(0)
    n = min(len(free), len(used))
    go = free[:n] < used[:n]
    src, dst = used[:n][go], free[:n][go]
    to = torch.arange(pages, device=DEV)
    to[src] = dst
    refs[dst] = refs[src]
    refs[src] = 0
    out = torch.where(table >= 0, to[table.clamp(min=0)], -1)
    copy_plain(s, src, dst)
    counts = ints([len(src), 0])
    counts[1] = torch.where(refs != 0, torch.arange(1, pages + 1, device=DEV), 0).amax()
    return out.int(), refs.int(), counts, s["ck"], s["cv"], s["ks"], s["vs"]


RUN_OWN = {"rot": own_rot, "app": own_app, "att": own_att, "fork": own_fork, "comp": own_comp}
RUN_PLAIN = {"rot": plain_rot, "app": plain_app, "att": plain_att, "fork": plain_fork,
             "comp": plain_comp}


# ---------------------------------------------------------------------------------------------
# what a pass cannot do without, and what it means in 64 bits
# ---------------------------------------------------------------------------------------------
def visible(c):
    """How many tokens each row of an attending step sees, by sequence."""
    new, old = sequences(c)
    far = c["window"] or 1 << 30
    return [[min(y + j + 1, far) for j in range(x)] for x, y in zip(new, old)]


def copied_by_fork(c):
    lens, parents = fork_shape(c)
    part = [p for p in parents if p >= 0 and lens[p] % PAGE]
    return len(part) - len(set(part))


def moved_by_comp(c):
    """Half of those above the number in use, which the pages' random order gives on average."""
    used = sum(comp_shape(c))
    return used * (c["pages"] - used) / c["pages"]


def work(case):
    c = case
    op = c["op"]
    if op == "rot":
        size = 4 if c["dtype"] == "f32" else 2
        n = c["t"] * (c["hq"] + c["hk"]) * c["d"]
        return {"bytes": 2 * size * n + 8 * c["t"] + 4 * c["r"], "flops": 3 * n}
    if op == "app":
        new, old = sequences(c)
        seen = sum(x + y - y // PAGE * PAGE for x, y in zip(new, old))
        n = sum(new) * 2 * c["h"] * c["d"]
        # rows read, written as bytes, and read back as values
        return {"bytes": 3 * n + 3 * seen * 2 * c["h"] * c["d"] + 16 * c["h"] * c["b"],
                "flops": 6 * n}
    if op == "att":
        seen = visible(c)
        far = c["window"] or 1 << 30
        read = sum(min(v[-1] + len(v) - 1, far + len(v)) if c["window"] else v[-1] for v in seen)
        t = sum(len(v) for v in seen)
        return {"bytes": read * c["hk"] * (2 * c["d"] + 0.125)
                + t * c["hq"] * (4 * c["d"] + 4),
                "flops": 4 * c["hq"] * c["d"] * sum(sum(v) for v in seen)}
    page = c["layers"] * c["h"] * (2 * PAGE * c["d"] + 8)
    if op == "fork":
        entries = c["r"] * (pages_of(c["l"]) + 2)
        return {"bytes": 2 * page * copied_by_fork(c) + 8 * entries + 4 * c["pages"],
                "flops": entries}
    return {"bytes": 2 * page * moved_by_comp(c) + 8 * c["r"] * c["w"] + 4 * c["pages"],
            "flops": c["r"] * c["w"]}


def exact(case, seed):
    return EXACT[case["op"]](prepare(case, seed))


def exact_rot(s):
    phase = torch.outer(s["pos"].double(), s["freqs"])
    unit = torch.polar(torch.full_like(phase, s["scale"]), phase)[:, None]

    def turn(x):
        y, r = x.double(), s["r"]
        z = torch.empty_like(y)
        z[..., r:] = y[..., r:]
        if s["layout"] == "half":
            first, second = slice(0, r // 2), slice(r // 2, r)
        else:
            first, second = slice(0, r, 2), slice(1, r, 2)
        w = torch.complex(y[..., first], y[..., second]) * unit
        z[..., first], z[..., second] = w.real, w.imag
        return z

    return turn(s["q"]), turn(s["k"])


def exact_app(s):
    e4m3, h, d = s["kind"] == "e4m3", s["h"], s["d"]
    most = 448 if e4m3 else 127
    starts, lens, seen = (s[x].tolist() for x in ("starts", "lens", "seen"))
    table = s["table"].tolist()
    ks, vs = s["ks"].double(), s["vs"].double()
    shown = [torch.empty(s["seen_rows"], h, d, dtype=torch.float64, device=DEV) for _ in "kv"]

    def levels(x):
        return x.clamp(-448, 448).float().to(FP8).double() if e4m3 else x.round()

    for i, end in enumerate(lens):
        old = end - (starts[i + 1] - starts[i])
        out = seen[i]
        for p in range(old // PAGE, pages_of(end)):
            lo, hi = p * PAGE, min(end, p * PAGE + PAGE)
            page, a = table[i][p], max(lo, old)
            for which, (x, cache, scale) in enumerate(((s["k"], s["ck"], ks),
                                                       (s["v"], s["cv"], vs))):
                x = x[starts[i] + a - old:starts[i] + hi - old].double()
                rows = torch.empty(hi - lo, h, d, dtype=torch.float64, device=DEV)
                stored = cache[page].float().double()
                was = scale[page].clone()
                now = torch.linalg.vector_norm(x, ord=math.inf, dim=(0, 2)) / most
                if a > lo:
                    now = torch.maximum(now, was)
                    for k in range(a - lo):
                        old_row = stored[:, :, k].reshape(h, d) if which == 0 else \
                            stored[:, k // 16, :, k % 16]
                        rows[k] = levels(old_row * (was / now)[:, None])
                rows[a - lo:] = levels(x / now[:, None])
                scale[page] = now
                shown[which][out:out + hi - lo] = rows * now[:, None]
            out += hi - lo
    return *shown, ks, vs


def exact_att(s):
    hk, d = s["hk"], s["d"]
    group = s["hq"] // hk
    out = torch.zeros(s["rows"], s["hq"], d, dtype=torch.float64, device=DEV)
    lse = torch.full((s["rows"], s["hq"]), -math.inf, dtype=torch.float64, device=DEV)
    starts, lens = s["starts"].tolist(), s["lens"].tolist()
    for i, end in enumerate(lens):
        ids = s["table"][i, :pages_of(end)].long()
        for h in range(hk):
            k = s["ck"].view(torch.int8)[ids, h].view(s["ck"].dtype).float().double()
            v = s["cv"].view(torch.int8)[ids, h].view(s["cv"].dtype).float().double()
            k = (k * s["ks"].double()[ids, h][:, None, None, None]).permute(0, 2, 1, 3)
            v = (v * s["vs"].double()[ids, h][:, None, None, None]).permute(0, 1, 3, 2)
            k, v = k.reshape(-1, d)[:end], v.reshape(-1, d)[:end]
            heads = slice(h * group, (h + 1) * group)
            for t in range(starts[i], starts[i + 1]):
                last = end - (starts[i + 1] - t)
                lo = max(0, last + 1 - s["window"]) if s["window"] else 0
                z = s["q"][t, heads].double() @ k[lo:last + 1].t() * d ** -0.5
                lse[t, heads] = torch.logsumexp(z, 1)
                out[t, heads] = torch.softmax(z, 1) @ v[lo:last + 1]
    return out, lse


def exact_fork(s):
    """The scales after the copies (the rest are whole numbers)."""
    table, lens, parents = (s[x].tolist() for x in ("table", "lens", "parents"))
    rows = [table[p][:pages_of(lens[p])] if p >= 0 else [] for p in parents]
    held = [x for row in rows for x in row]
    free = iter(sorted(set(range(s["ck"].shape[1])) - set(held)))
    ks, vs = s["ks"].double(), s["vs"].double()
    begun = set()
    for p, row in zip(parents, rows):
        if p < 0:
            continue
        if lens[p] % PAGE == 0:
            next(free)
        elif row[-1] in begun:
            to = next(free)
            ks[:, to], vs[:, to] = ks[:, row[-1]], vs[:, row[-1]]
        else:
            begun.add(row[-1])
    return *[None] * 6, ks, vs


def exact_comp(s):
    used = set(s["table"].flatten().tolist()) - {-1}
    ks, vs = s["ks"].double(), s["vs"].double()
    free = sorted(set(range(s["pages"])) - used)
    for to, at in zip(free, sorted(used, reverse=True)):
        if to < at:
            ks[:, to], vs[:, to] = ks[:, at], vs[:, at]
    return *[None] * 5, ks, vs


EXACT = {"rot": exact_rot, "app": exact_app, "att": exact_att, "fork": exact_fork,
         "comp": exact_comp}
