"""The operators of a second pass over decoded words, as cases that can be timed.

A second pass runs a small language model beside the decoder: for each lane it
reads the first-pass words and answers one token at a time.  Four operators
make up its step: products with 4-bit weights, the heads' norm and rotation
with the write into the paged cache, attention of the new token over that
cache, and the draw of the next token.

``run`` computes a case in elementary torch operations while ``own`` is false
and through the package's entry points while it is true; ``exact`` gives the
same outputs from the definitions in 64 bits.
"""
from __future__ import annotations

import math
import random

import torch

own = False

DEV = "cuda"
TYPES = {"bf16": torch.bfloat16, "f16": torch.float16, "f32": torch.float32}
FIXED = 43                      # sampling weights are whole multiples of 2^-43 of the largest one


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # one lane's square projection: the latency of a single stream
        dict(name="matvec-1x4096x4096", op="matvec", rows=1, n=4096, k=4096, group=128, zeros=False, bias=False,
             type="bf16"),
        # the output layer over this decoder's 5000 labels for its 64 lanes, odd model width, zero points
        dict(name="matvec-64x5000x1056", op="matvec", rows=64, n=5000, k=1056, group=32, zeros=True, bias=True,
             type="f16"),
        # a large word vocabulary for eight streaming channels
        dict(name="matvec-8x131072x4096", op="matvec", rows=8, n=131072, k=4096, group=128, zeros=False, bias=False,
             type="bf16"),
        # one new token of one stream
        dict(name="rotate-1", op="rotate", tokens=1, hq=32, hkv=8, d=128, rot=128, page=16, inter=False, type="bf16"),
        # one new token of each of 64 lanes; half of a head turned, in neighbouring pairs
        dict(name="rotate-64", op="rotate", tokens=64, hq=16, hkv=16, d=64, rot=32, page=48, inter=True, type="f16"),
        # the first-pass words of all lanes, read at once
        dict(name="rotate-16000", op="rotate", tokens=16000, hq=32, hkv=8, d=128, rot=128, page=16, inter=False,
             type="bf16"),
        # one lane a few hundred words in: latency
        dict(name="attend-1x500", op="attend", lanes=1, lo=500, hi=500, hq=16, hkv=16, d=64, page=16, window=0,
             sinks=0, type="f16"),
        # 64 lanes of very different lengths
        dict(name="attend-64x8192", op="attend", lanes=64, lo=1, hi=8192, hq=32, hkv=8, d=128, page=16, window=0,
             sinks=0, type="bf16"),
        # two long documents: few rows, the cache's length is split
        dict(name="attend-2x131072", op="attend", lanes=2, lo=100000, hi=131072, hq=64, hkv=8, d=128, page=64,
             window=0, sinks=0, type="bf16"),
        # 128 channels of hour-long audio: the last 2047 tokens and the first 4 stay, pages between are gone
        dict(name="attend-128x90000-window", op="attend", lanes=128, lo=500, hi=90000, hq=32, hkv=8, d=128, page=48,
             window=2047, sinks=4, type="bf16"),
        # one lane over this decoder's 5000 labels
        dict(name="sample-1x5000", op="sample", lanes=1, vocab=5000, temp=0.8, top_k=40, top_p=0.95, min_p=0.0,
             type="f32"),
        # 64 lanes over a large word vocabulary
        dict(name="sample-64x131071", op="sample", lanes=64, vocab=131071, temp=1.0, top_k=0, top_p=0.9, min_p=0.02,
             type="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["matvec", "rotate", "attend", "sample"])
    if op == "matvec":
        group = rng.choice([32, 64, 128])
        rows, n = _log(rng, 1, 64), _log(rng, 256, 65536)
        k = group * max(1, _log(rng, 512, 8192) // group)
        return dict(op=op, rows=rows, n=n, k=k, group=group, zeros=rng.random() < 0.5, bias=rng.random() < 0.5,
                    type=rng.choice(["bf16", "f16"]))
    if op == "rotate":
        hkv, d = rng.choice([1, 2, 4, 8]), rng.choice([64, 128, 256])
        return dict(op=op, tokens=_log(rng, 1, 8000), hq=hkv * rng.choice([1, 2, 3, 4]), hkv=hkv, d=d,
                    rot=rng.choice([d, d // 2]), page=rng.choice([16, 17, 48, 64]), inter=rng.random() < 0.5,
                    type=rng.choice(["bf16", "f16"]))
    if op == "attend":
        hkv, d, lanes = rng.choice([1, 2, 5, 8]), rng.choice([64, 128, 256]), _log(rng, 1, 96)
        hi = _log(rng, 16, min(60000, 200_000_000 // (lanes * hkv * d)))
        window = rng.choice([0, 0, _log(rng, 8, 4000)])
        return dict(op=op, lanes=lanes, lo=rng.choice([1, max(1, hi // 2), hi]), hi=hi,
                    hq=hkv * rng.choice([1, 3, 4, 8, 12]), hkv=hkv, d=d, page=rng.choice([1, 16, 48, 64, 100]),
                    window=window, sinks=rng.choice([0, 1, 4, 20]) if window else 0, type=rng.choice(["bf16", "f16"]))
    return dict(op=op, lanes=_log(rng, 1, 64), vocab=_log(rng, 1000, 131072), temp=round(rng.uniform(0.5, 1.5), 3),
                top_k=rng.choice([0, _log(rng, 1, 1000)]), top_p=rng.choice([1.0, round(rng.uniform(0.3, 0.99), 3)]),
                min_p=rng.choice([0.0, round(rng.uniform(0.001, 0.2), 4)]), type=rng.choice(["bf16", "f16", "f32"]))


# ------------------------------------------------------------------ the inputs

def _visible(c, length):
    """(first, window start) of a lane: tokens [0, first) and [start, length) are seen."""
    if not c["window"]:
        return 0, 0
    start = max(0, length - c["window"])
    return min(c["sinks"], start), start


def _lengths(c, seed):
    rng = random.Random(seed * 7919 + 13)
    n = [rng.randint(c["lo"], c["hi"]) for _ in range(c["lanes"])]
    n[0] = c["hi"]
    return n


def prepare(case, seed):
    c = dict(case)
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    t = TYPES[c["type"]]

    def normal(*shape, scale=1.0, dtype=t):
        return (torch.randn(*shape, generator=g, device=DEV, dtype=torch.float32) * scale).to(dtype)

    def uniform(*shape, lo=0.0, hi=1.0, dtype=torch.float32):
        return (torch.rand(*shape, generator=g, device=DEV, dtype=torch.float32) * (hi - lo) + lo).to(dtype)

    s = dict(c)
    if c["op"] == "matvec":
        n, k, groups = c["n"], c["k"], c["k"] // c["group"]
        s["x"] = normal(c["rows"], k)
        # two codes to a byte, the lower code in the lower half
        s["codes"] = torch.randint(0, 256, (n, k // 2), generator=g, device=DEV, dtype=torch.uint8)
        s["scales"] = uniform(n, groups, lo=0.2, hi=1.8, dtype=torch.float32).mul_(0.2 / math.sqrt(k)).to(t)
        s["zp"] = torch.randint(5, 11, (n, groups), generator=g, device=DEV).to(t) if c["zeros"] else None
        s["b"] = normal(n, scale=0.5) if c["bias"] else None
        if own:
            import wfst_beam_search_gb300 as W
            s["W"], s["weights"] = W, W.pack_quant(s["codes"], s["scales"], s["zp"])
    elif c["op"] == "rotate":
        tok, d = c["tokens"], c["d"]
        # one projection's output holds q, k and v of a token side by side
        qkv = normal(tok, (c["hq"] + 2 * c["hkv"]) * d, scale=1.5)
        heads = qkv.view(tok, -1, d)
        s["q"], s["k"], s["v"] = heads.split([c["hq"], c["hkv"], c["hkv"]], 1)
        s["qw"], s["kw"] = uniform(d, lo=0.5, hi=1.5, dtype=t), uniform(d, lo=0.5, hi=1.5, dtype=t)
        ctx = 4096
        freq = 10000.0 ** (-torch.arange(0, c["rot"], 2, device=DEV, dtype=torch.float64) / c["rot"])
        ang = torch.arange(ctx, device=DEV, dtype=torch.float64)[:, None] * freq
        s["table"] = torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()
        s["pos"] = torch.randint(0, ctx, (tok,), generator=g, device=DEV, dtype=torch.int32)
        pages = -(-tok // c["page"]) + 3
        s["kc"] = torch.zeros(pages, c["page"], c["hkv"], d, device=DEV, dtype=t)
        s["vc"] = torch.zeros_like(s["kc"])
        s["slots"] = torch.randperm(pages * c["page"], generator=g, device=DEV)[:tok].to(torch.int32)
        if own:
            import wfst_beam_search_gb300 as W
            s["W"] = W
    elif c["op"] == "attend":
        lens = _lengths(c, seed)
        width = -(-max(lens) // c["page"])
        table = torch.full((c["lanes"], width), -1, dtype=torch.int32)
        need = []
        for b, n in enumerate(lens):
            first, start = _visible(c, n)
            ids = sorted({j // c["page"] for j in range(first)} | set(range(start // c["page"], -(-n // c["page"]))))
            need += [(b, i) for i in ids]
        order = list(range(len(need)))
        random.Random(seed).shuffle(order)             # pages of a lane lie anywhere in the pool
        at = torch.tensor(need, dtype=torch.int64)
        table[at[:, 0], at[:, 1]] = torch.tensor(order, dtype=torch.int32)
        s["table"] = table.to(DEV)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        shape = (len(need), c["page"], c["hkv"], c["d"])
        s["q"] = normal(c["lanes"], c["hq"], c["d"], scale=1.5)
        s["kc"] = torch.empty(shape, dtype=t, device=DEV).normal_(generator=g)
        s["vc"] = torch.empty(shape, dtype=t, device=DEV).normal_(generator=g)
        s["most"] = max(lens)
        s["scale"] = 1.0 / math.sqrt(c["d"])
        if own:
            import wfst_beam_search_gb300 as W
            s["W"], s["ws"] = W, W.attend_workspace(DEV)
    else:
        # a peaked head over a broad tail, as trained models answer
        x = normal(c["lanes"], c["vocab"], scale=2.0, dtype=torch.float32)
        few = torch.randint(0, c["vocab"], (c["lanes"], 32), generator=g, device=DEV)
        x.scatter_add_(1, few, uniform(c["lanes"], 32, lo=0.0, hi=8.0))
        s["logits"] = x.to(t)
        s["u"] = uniform(c["lanes"])
        if own:
            import wfst_beam_search_gb300 as W
            s["W"] = W
    return s


# ------------------------------------------------------------------ one pass

def _unpack(codes, dtype):
    return torch.stack([codes & 15, codes >> 4], 2).reshape(codes.shape[0], -1).to(dtype)


def _dequant(s, dtype):
    n, k = s["n"], s["k"]
    c = _unpack(s["codes"], dtype).view(n, k // s["group"], s["group"])
    z = 8.0 if s["zp"] is None else s["zp"].to(dtype)[:, :, None]
    return ((c - z) * s["scales"].to(dtype)[:, :, None]).view(n, k)


def _rotate_heads(x, w, table, pos, rot, inter, dtype, eps=1e-6):
    x = x.to(dtype)
    x = x / torch.sqrt((x * x).mean(-1, keepdim=True) + eps) * w.to(dtype)
    cs = table.to(dtype)[pos.long()][:, None, :]
    cos, sin = cs[..., : rot // 2], cs[..., rot // 2:]
    a, b = (x[..., 0:rot:2], x[..., 1:rot:2]) if inter else (x[..., : rot // 2], x[..., rot // 2: rot])
    y, z = a * cos - b * sin, a * sin + b * cos
    turned = torch.stack([y, z], -1).flatten(-2) if inter else torch.cat([y, z], -1)
    return torch.cat([turned, x[..., rot:]], -1)


def _plain_rotate(s, dtype):
    q = _rotate_heads(s["q"], s["qw"], s["table"], s["pos"], s["rot"], s["inter"], dtype)
    k = _rotate_heads(s["k"], s["kw"], s["table"], s["pos"], s["rot"], s["inter"], dtype)
    return q, k


def _plain_attend(s):
    lanes, hkv, d, page, most = s["lanes"], s["hkv"], s["d"], s["page"], s["most"]
    lens = s["lens"][:, None]
    j = torch.arange(most, device=DEV)[None, :]
    if s["window"]:
        # the visible tokens alone, side by side: the first ones, then the window
        start = (lens - s["window"]).clamp_min(0)
        first = torch.minimum(start, torch.full_like(start, s["sinks"]))
        j = torch.arange(min(most, s["window"] + s["sinks"]), device=DEV)[None, :]
        j = torch.where(j < first, j, j - first + start)
    seen = j < lens
    j = torch.where(seen, j, 0)
    rows = s["table"].gather(1, (j // page).long()).long().clamp_min(0) * page + j % page
    k = s["kc"].view(-1, hkv, d)[rows].float()
    v = s["vc"].view(-1, hkv, d)[rows].float()
    q = s["q"].float().view(lanes, hkv, -1, d)
    x = torch.einsum("bhgd,bjhd->bhgj", q, k) * s["scale"]
    x = x.masked_fill(~seen[:, None, None, :], -math.inf)
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    total = e.sum(-1, keepdim=True)
    o = torch.einsum("bhgj,bjhd->bhgd", e / total, v)
    return o.reshape(lanes, -1, d).to(s["q"].dtype), (m + torch.log(total)).reshape(lanes, -1)


def _plain_sample(s):
    x = s["logits"].float()
    y = (x - x.amax(1, keepdim=True)) * torch.reciprocal(torch.full((), s["temp"], device=DEV))
    w = torch.exp(y)
    # whole numbers: their sums have one value in any order
    fixed = (w.double() * 2.0 ** FIXED).long()
    order = torch.sort(x, dim=1, descending=True, stable=True).indices
    ranked = fixed.gather(1, order)
    place = torch.arange(x.shape[1], device=DEV).expand_as(x)
    keep = place < (s["top_k"] or x.shape[1])
    if s["top_p"] < 1.0:
        ranked_k = torch.where(keep, ranked, 0)
        want = torch.ceil(ranked_k.sum(1, keepdim=True).double() * _single(s["top_p"])).long().clamp_min(1)
        keep = keep & (ranked_k.cumsum(1) - ranked_k < want)
    if s["min_p"] > 0.0:
        keep = keep & (w.gather(1, order) >= _single(s["min_p"]))
    kept = keep.sum(1, dtype=torch.int32)
    fixed = torch.where(torch.zeros_like(keep).scatter_(1, order, keep), fixed, 0)
    total = fixed.sum(1, keepdim=True)
    aim = torch.minimum((s["u"].double()[:, None] * total.double()).long(), total - 1)
    token = (fixed.cumsum(1) <= aim).sum(1, keepdim=True)
    logprob = y.gather(1, token) - torch.log(total.double() * 2.0 ** -FIXED).float()
    return token[:, 0].to(torch.int32), logprob[:, 0], kept


def _single(v):
    """The value of a number once held in 32 bits."""
    return float(torch.tensor(v, dtype=torch.float32))


def run(s):
    op = s["op"]
    if own:
        W = s["W"]
        if op == "matvec":
            return W.matvec_quant(s["x"], s["weights"], bias=s["b"])
        if op == "rotate":
            q = W.norm_rotate(s["q"], s["k"], s["v"], s["pos"], s["table"], s["qw"], s["kw"], s["kc"], s["vc"],
                              s["slots"], eps=1e-6, interleaved=s["inter"])
            return q, s["kc"], s["vc"]
        if op == "attend":
            return W.attend_paged(s["q"], s["kc"], s["vc"], s["table"], s["lens"], scale=s["scale"],
                                  window=s["window"], sinks=s["sinks"], workspace=s["ws"], with_lse=True)
        return W.sample_tokens(s["logits"], s["u"], temperature=s["temp"], top_k=s["top_k"], top_p=s["top_p"],
                               min_p=s["min_p"])
    if op == "matvec":
        y = s["x"].float() @ _dequant(s, torch.float32).t()
        if s["b"] is not None:
            y = y + s["b"].float()
        return y.to(s["x"].dtype)
    if op == "rotate":
        q, k = _plain_rotate(s, torch.float32)
        at = s["slots"].long()
        s["kc"].view(-1, s["hkv"], s["d"])[at] = k.to(s["kc"].dtype)
        s["vc"].view(-1, s["hkv"], s["d"])[at] = s["v"]
        return q.to(s["q"].dtype), s["kc"], s["vc"]
    if op == "attend":
        return _plain_attend(s)
    return _plain_sample(s)


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op, f = case["op"], torch.float64
    if op == "matvec":
        out = []
        x, step = s["x"].to(f), max(1, (1 << 26) // case["k"])
        for lo in range(0, case["n"], step):
            hi = min(case["n"], lo + step)
            low, high = s["codes"][lo:hi].to(f) % 16, torch.div(s["codes"][lo:hi], 16, rounding_mode="floor").to(f)
            w = torch.empty(hi - lo, case["k"], dtype=f, device=DEV)
            w[:, 0::2], w[:, 1::2] = low, high
            w -= 8 if s["zp"] is None else s["zp"][lo:hi].to(f).repeat_interleave(case["group"], 1)
            w *= s["scales"][lo:hi].to(f).repeat_interleave(case["group"], 1)
            out.append(x @ w.t())
        y = torch.cat(out, 1)
        return y if s["b"] is None else y + s["b"].to(f)
    if op == "rotate":
        rot, half = case["rot"], case["rot"] // 2

        def turned(x, w):
            x = x.to(f)
            x = x * w.to(f) * (x.pow(2).sum(-1, keepdim=True) / case["d"] + 1e-6).rsqrt()
            cs = s["table"].to(f)[s["pos"].long()]
            z = torch.complex(cs[:, None, :half], cs[:, None, half:])
            i = torch.arange(half, device=DEV)
            re, im = (2 * i, 2 * i + 1) if case["inter"] else (i, i + half)
            p = torch.complex(x[..., re], x[..., im]) * z
            x[..., re], x[..., im] = p.real, p.imag
            return x

        kc, vc = s["kc"].to(f), s["vc"].to(f)
        at = s["slots"].long()
        kc[at // case["page"], at % case["page"]] = turned(s["k"], s["kw"])
        vc[at // case["page"], at % case["page"]] = s["v"].to(f)
        return turned(s["q"], s["qw"]), kc, vc
    if op == "attend":
        o = torch.zeros(case["lanes"], case["hq"], case["d"], dtype=f, device=DEV)
        lse = torch.zeros(case["lanes"], case["hq"], dtype=f, device=DEV)
        share = case["hq"] // case["hkv"]
        for b, n in enumerate(s["lens"].tolist()):
            first, start = _visible(case, n)
            j = torch.cat([torch.arange(first, device=DEV), torch.arange(start, n, device=DEV)])
            page = s["table"][b][j // case["page"]].long()
            k, v = (s[name][page, j % case["page"]] for name in ("kc", "vc"))
            for h in range(case["hkv"]):
                heads = slice(h * share, (h + 1) * share)
                x = s["q"][b, heads].to(f) @ k[:, h].to(f).t() * s["scale"]
                lse[b, heads] = torch.logsumexp(x, 1)
                o[b, heads] = torch.softmax(x, 1) @ v[:, h].to(f)
        return o, lse
    tokens, logprobs, counts = [], [], []
    for x, u in zip(s["logits"].to(f), s["u"].tolist()):
        p = torch.softmax(x / _single(case["temp"]), 0)
        top, at = torch.sort(p, dim=0, descending=True, stable=True)
        n = case["top_k"] or len(x)
        if case["top_p"] < 1.0:
            c = top[:n].cumsum(0)
            n = 1 + int((c[:-1] < _single(case["top_p"]) * c[-1]).sum())
        if case["min_p"] > 0.0:
            n = min(n, int((top >= _single(case["min_p"]) * top[0]).sum()))
        some = at[:n].sort().values
        c = p[some].cumsum(0)
        i = min(int((c <= u * c[-1]).sum()), n - 1)
        tokens.append(int(some[i]))
        logprobs.append(float(torch.log(p[some[i]] / c[-1])))
        counts.append(n)
    return (torch.tensor(tokens, dtype=torch.int32), torch.tensor(logprobs, dtype=f),
            torch.tensor(counts, dtype=torch.int32))


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c, size = case, 4 if case["type"] == "f32" else 2
    if c["op"] == "matvec":
        groups = c["n"] * (c["k"] // c["group"])
        return {"bytes": c["n"] * c["k"] // 2 + groups * size * (2 if c["zeros"] else 1)
                + (c["rows"] * (c["k"] + c["n"]) + (c["n"] if c["bias"] else 0)) * size,
                "flops": 2 * c["rows"] * c["n"] * c["k"]}
    if c["op"] == "rotate":
        values = c["tokens"] * (c["hq"] + 2 * c["hkv"]) * c["d"]
        rows = min(c["tokens"], 4096) * c["rot"] * 4
        return {"bytes": 2 * values * size + rows + 8 * c["tokens"] + 2 * c["d"] * size,
                "flops": 8 * c["tokens"] * (c["hq"] + c["hkv"]) * c["d"]}
    if c["op"] == "attend":
        # the lengths of a middling seed; another seed's differ by a few percent
        seen = 0
        for n in _lengths(c, 1):
            first, start = _visible(c, n)
            seen += first + n - start
        return {"bytes": 2 * seen * c["hkv"] * c["d"] * size + c["lanes"] * c["hq"] * (2 * c["d"] * size + 4),
                "flops": 4 * seen * c["hq"] * c["d"]}
    return {"bytes": c["lanes"] * (c["vocab"] * size + 16), "flops": 6 * c["lanes"] * c["vocab"]}
