"""The operators of a second pass that rescores hypotheses, as cases that can be timed.

Many hypotheses are read by one language model after the same long context, and
each one's words are scored.  Three operators are met there beside those of a
plain step: attention of lanes that share a long prefix, low-rank adapters of
many requests beside a shared projection, and the log probabilities of given
tokens with entropy and the likeliest alternatives.

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


# ------------------------------------------------------------------ the cases

def listed():
    return [
        # eight hypotheses of one utterance after a short instruction: latency
        dict(name="prefix-8x500", op="prefix", lanes=8, prefix=500, lo=1, hi=64, hq=16, hkv=16, d=64, page=16,
             type="f16"),
        # 64 lanes, a long instruction before all of them, their own words behind it
        dict(name="prefix-64x8192", op="prefix", lanes=64, prefix=8192, lo=1, hi=256, hq=32, hkv=8, d=128, page=64,
             type="bf16"),
        # few hypotheses after the transcript of hours: the cache is what has to be read
        dict(name="prefix-16x131072", op="prefix", lanes=16, prefix=131072, lo=100, hi=500, hq=32, hkv=8, d=128, page=64,
             type="bf16"),
        # 128 channels after one long document, pages that end inside a tile: the products count
        dict(name="prefix-128x32767", op="prefix", lanes=128, prefix=32767, lo=1, hi=500, hq=64, hkv=8, d=128, page=48,
             type="bf16"),
        # one hypothesis' word over this decoder's 5000 labels
        dict(name="score-1x5000", op="score", rows=1, vocab=5000, top=5, masked=0.0, type="f32"),
        # one word of each of 64 lanes over a large word vocabulary
        dict(name="score-64x131071", op="score", rows=64, vocab=131071, top=8, masked=0.0, type="bf16"),
        # the first-pass words of 64 lanes at once, those that a grammar forbids masked
        dict(name="score-2000x20000", op="score", rows=2000, vocab=20000, top=0, masked=0.3, type="f16"),
        # the words of many hypotheses over a large word vocabulary
        dict(name="score-2048x131072", op="score", rows=2048, vocab=131072, top=20, masked=0.0, type="bf16"),
        # one lane with its speaker's adapter beside a square projection: latency
        dict(name="lowrank-1x4096x4096", op="lowrank", rows=1, n=4096, k=4096, adapters=4, rank=16, run=1, none=0.0,
             type="bf16"),
        # 64 lanes of eight domains, some without one, at the output layer of 5000 labels
        dict(name="lowrank-64x5000x1056", op="lowrank", rows=64, n=5000, k=1056, adapters=8, rank=8, run=1, none=0.2,
             type="f16"),
        # 64 lanes of 40 speakers with large adapters
        dict(name="lowrank-64x8192x8192", op="lowrank", rows=64, n=8192, k=8192, adapters=40, rank=64, run=1, none=0.0,
             type="bf16"),
        # the words of all lanes at once, a lane's words side by side
        dict(name="lowrank-4096x6144x4096", op="lowrank", rows=4096, n=6144, k=4096, adapters=16, rank=16, run=64,
             none=0.1, type="bf16"),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng: random.Random):
    op = rng.choice(["prefix", "score", "lowrank"])
    if op == "prefix":
        hkv, d = rng.choice([1, 2, 5, 8]), rng.choice([64, 128, 256])
        share, lanes = rng.choice([1, 3, 4, 8]), _log(rng, 1, 128)
        most = min(131072, 2 ** 38 // (4 * lanes * share * hkv * d), 2 ** 29 // (lanes * share * hkv), 2 ** 28 // (hkv * d))
        hi = _log(rng, 1, min(1000, 2 ** 28 // (lanes * hkv * d)))
        return dict(op=op, lanes=lanes, prefix=_log(rng, 100, most), lo=rng.choice([0, 1, hi]), hi=hi, hq=hkv * share,
                    hkv=hkv, d=d, page=rng.choice([1, 16, 48, 64, 100]), type=rng.choice(["bf16", "f16"]))
    if op == "score":
        vocab = _log(rng, 1000, 131072)
        return dict(op=op, rows=_log(rng, 1, min(4096, 2 ** 28 // vocab)), vocab=vocab,
                    top=rng.choice([0, 1, rng.randint(2, 32)]), masked=rng.choice([0.0, 0.0, round(rng.uniform(0.05, 0.9), 2)]),
                    type=rng.choice(["bf16", "f16", "f32"]) if vocab < 65536 else rng.choice(["bf16", "f16"]))
    rows, rank = _log(rng, 1, 4096), rng.choice([8, 16, 24, 32, 64])
    return dict(op=op, rows=rows, n=_log(rng, 256, 8192), k=8 * _log(rng, 32, 1024),
                adapters=_log(rng, 1, 40 if rows < 256 else 16), rank=rank, run=rng.choice([1, _log(rng, 1, 100)]),
                none=rng.choice([0.0, 0.3]), type=rng.choice(["bf16", "f16"]))


# ------------------------------------------------------------------ the inputs

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
    if c["op"] == "prefix":
        page, lens = c["page"], _lengths(c, seed)
        width = -(-c["hi"] // page)
        shared = -(-c["prefix"] // page)
        need = [-(-n // page) for n in lens]
        order = torch.randperm(shared + sum(need), generator=g, device=DEV).to(torch.int32)  # pages lie anywhere
        s["shared"] = order[:shared].clone()
        i = torch.arange(width)[None, :] < torch.tensor(need)[:, None]
        table = torch.full((c["lanes"], width), -1, dtype=torch.int32)
        table[i] = order[shared:].cpu()
        s["table"] = table.to(DEV)
        s["lens"] = torch.tensor(lens, dtype=torch.int32, device=DEV)
        s["plen"] = torch.tensor([c["prefix"]], dtype=torch.int32, device=DEV)
        shape = (len(order), page, c["hkv"], c["d"])
        s["q"] = normal(c["lanes"], c["hq"], c["d"], scale=1.5)
        s["kc"] = torch.empty(shape, dtype=t, device=DEV).normal_(generator=g)
        s["vc"] = torch.empty(shape, dtype=t, device=DEV).normal_(generator=g)
        s["scale"] = 1.0 / math.sqrt(c["d"])
        if own:
            import wfst_beam_search_gb300 as W
            s["W"], s["ws"] = W, W.attend_prefix_workspace(c["lanes"], c["hq"], c["hkv"], c["d"], DEV)
    elif c["op"] == "score":
        # a peaked head over a broad tail, as trained models answer; what is scored is often likely
        x = normal(c["rows"], c["vocab"], scale=2.0, dtype=torch.float32)
        few = torch.randint(0, c["vocab"], (c["rows"], 32), generator=g, device=DEV)
        x.scatter_add_(1, few, uniform(c["rows"], 32, lo=0.0, hi=8.0))
        if c["masked"]:
            x.masked_fill_(torch.rand(x.shape, generator=g, device=DEV) < c["masked"], -math.inf)
        s["logits"] = x.to(t)
        del x
        drawn = torch.randint(0, c["vocab"], (c["rows"],), generator=g, device=DEV)
        s["tokens"] = torch.where(uniform(c["rows"]) < 0.7, few[:, 0], drawn).to(torch.int32)
        if own:
            import wfst_beam_search_gb300 as W
            s["W"] = W
    else:
        rows, n, k, rank = c["rows"], c["n"], c["k"], c["rank"]
        s["x"], s["y"] = normal(rows, k), normal(rows, n)
        s["shrink"] = normal(c["adapters"], rank, k, scale=k ** -0.5)
        s["expand"] = normal(c["adapters"], n, rank, scale=0.5 * rank ** -0.5)
        s["scales"] = uniform(c["adapters"], lo=0.5, hi=2.0)
        lanes = -(-rows // c["run"])
        which = torch.randint(0, c["adapters"], (lanes,), generator=g, device=DEV)
        which = torch.where(uniform(lanes) < c["none"], -1, which)
        s["which"] = which.repeat_interleave(c["run"])[:rows].to(torch.int32)
        if own:
            import wfst_beam_search_gb300 as W
            s["W"] = W
    return s


# ------------------------------------------------------------------ one pass

def _plain_prefix(s):
    lanes, hkv, d, page = s["lanes"], s["hkv"], s["d"], s["page"]
    pools = [s[name].view(-1, hkv, d) for name in ("kc", "vc")]
    j = torch.arange(s["prefix"], device=DEV)
    rows = s["shared"][j // page].long() * page + j % page
    kp, vp = (p[rows].float() for p in pools)
    j = torch.arange(s["hi"], device=DEV)[None, :]
    seen = j < s["lens"][:, None]
    rows = s["table"].gather(1, (j // page).expand(lanes, -1)).long().clamp_min(0) * page + j % page
    ko, vo = (p[rows].float() for p in pools)
    q = s["q"].float().view(lanes, hkv, -1, d)
    shared = torch.einsum("bhgd,jhd->bhgj", q, kp) * s["scale"]
    mine = torch.einsum("bhgd,bjhd->bhgj", q, ko) * s["scale"]
    x = torch.cat([shared, mine.masked_fill(~seen[:, None, None, :], -math.inf)], -1)
    del shared, mine
    m = x.amax(-1, keepdim=True)
    e = torch.exp(x - m)
    del x
    total = e.sum(-1, keepdim=True)
    p = e / total
    o = torch.einsum("bhgj,jhd->bhgd", p[..., :s["prefix"]], vp) + torch.einsum("bhgj,bjhd->bhgd", p[..., s["prefix"]:], vo)
    return o.reshape(lanes, -1, d).to(s["q"].dtype), (m + torch.log(total)).reshape(lanes, -1)


def _plain_score(s):
    x = s["logits"].float()
    m = x.amax(1, keepdim=True)
    y = x - m
    e = torch.exp(y)
    total = e.sum(1, keepdim=True)
    log_total = torch.log(total)
    entropy = log_total - (e * torch.where(e > 0, y, 0.0)).sum(1, keepdim=True) / total
    logprob = y.gather(1, s["tokens"].long()[:, None]) - log_total
    at = torch.sort(x, dim=1, descending=True, stable=True).indices[:, :s["top"]]
    return logprob[:, 0], entropy[:, 0], at.to(torch.int32), y.gather(1, at) - log_total


def _plain_lowrank(s):
    rows, a, rank = s["rows"], s["adapters"], s["rank"]
    # every adapter for every row, and the others' parts taken out
    t = (s["x"].float() @ s["shrink"].float().view(a * rank, -1).t()).view(rows, a, rank)
    mine = s["which"][:, None] == torch.arange(a, device=DEV)
    t = torch.where(mine[:, :, None], t * s["scales"][None, :, None], 0.0)
    more = t.reshape(rows, -1) @ s["expand"].float().transpose(1, 2).reshape(a * rank, -1)
    return (s["y"].float() + more).to(s["y"].dtype)


def run(s):
    op = s["op"]
    if own:
        W = s["W"]
        if op == "prefix":
            return W.attend_prefix(s["q"], s["kc"], s["vc"], s["shared"], s["plen"], s["table"], s["lens"],
                                   scale=s["scale"], workspace=s["ws"], with_lse=True)
        if op == "score":
            return W.score_tokens(s["logits"], s["tokens"], top=s["top"])
        return W.add_lowrank(s["y"], s["x"], s["shrink"], s["expand"], s["which"], scales=s["scales"])
    if op == "prefix":
        return _plain_prefix(s)
    if op == "score":
        return _plain_score(s)
    return _plain_lowrank(s)


# ------------------------------------------------------------------ 64 bits

def exact(case, seed):
    s = prepare(case, seed)
    op, f = case["op"], torch.float64
    if op == "prefix":
        lanes, share, page = case["lanes"], case["hq"] // case["hkv"], case["page"]
        o = torch.zeros(lanes, case["hq"], case["d"], dtype=f, device=DEV)
        lse = torch.zeros(lanes, case["hq"], dtype=f, device=DEV)
        jp = torch.arange(case["prefix"], device=DEV)
        page_p = s["shared"][jp // page].long()
        for h in range(case["hkv"]):
            heads = slice(h * share, (h + 1) * share)
            # the prefix' and the lane's own sums, each with its own largest score, put together at the end
            k, v = (s[name][page_p, jp % page, h].to(f) for name in ("kc", "vc"))
            step = max(1, (1 << 27) // (case["prefix"] * share))
            for b0 in range(0, lanes, step):
                x = torch.einsum("bgd,jd->bgj", s["q"][b0:b0 + step, heads].to(f), k) * s["scale"]
                lse[b0:b0 + step, heads] = torch.logsumexp(x, 2)
                o[b0:b0 + step, heads] = torch.softmax(x, 2) @ v
            for b, n in enumerate(s["lens"].tolist()):
                if not n:
                    continue
                j = torch.arange(n, device=DEV)
                at = s["table"][b][j // page].long()
                k1, v1 = (s[name][at, j % page, h].to(f) for name in ("kc", "vc"))
                x = s["q"][b, heads].to(f) @ k1.t() * s["scale"]
                one = torch.logsumexp(x, 1)
                both = torch.logaddexp(lse[b, heads], one)
                o[b, heads] = (o[b, heads] * torch.exp(lse[b, heads] - both)[:, None]
                               + torch.softmax(x, 1) @ v1 * torch.exp(one - both)[:, None])
                lse[b, heads] = both
        return o, lse
    if op == "score":
        logprob, entropy, tokens, top = [], [], [], []
        step = max(1, (1 << 26) // case["vocab"])
        for r in range(0, case["rows"], step):
            x = torch.log_softmax(s["logits"][r:r + step].to(f), 1)
            logprob.append(x.gather(1, s["tokens"][r:r + step].long()[:, None])[:, 0])
            entropy.append(torch.special.entr(torch.exp(x)).sum(1))
            # (the widened logits themselves: differences of them could make ties)
            order = torch.sort(s["logits"][r:r + step].to(f), dim=1, descending=True, stable=True).indices[:, :case["top"]]
            tokens.append(order.to(torch.int32))
            top.append(x.gather(1, order))
        return torch.cat(logprob), torch.cat(entropy), torch.cat(tokens), torch.cat(top)
    z = s["y"].to(f)
    which = s["which"].long()
    for a in range(case["adapters"]):
        rows = torch.nonzero(which == a)[:, 0]
        t = torch.einsum("rk,jk->rj", s["x"][rows].to(f), s["shrink"][a].to(f))
        z[rows] += s["scales"][a].to(f) * torch.einsum("rj,nj->rn", t, s["expand"][a].to(f))
    return z


# ------------------------------------------------------------------ what a pass cannot do without

def work(case):
    c, size = case, 4 if case["type"] == "f32" else 2
    if c["op"] == "prefix":
        # the lengths of a middling seed; another seed's differ by a few percent
        mine = sum(_lengths(c, 1))
        return {"bytes": 2 * (c["prefix"] + mine) * c["hkv"] * c["d"] * size + c["lanes"] * c["hq"] * (2 * c["d"] * size + 4),
                "flops": 4 * (c["lanes"] * c["prefix"] + mine) * c["hq"] * c["d"]}
    if c["op"] == "score":
        return {"bytes": c["rows"] * (c["vocab"] * size + 12 + 8 * c["top"]), "flops": 5 * c["rows"] * c["vocab"]}
    # adapters that some row uses, as many as the rows' lanes hit on average
    lanes = -(-c["rows"] // c["run"]) * (1 - c["none"])
    used = c["adapters"] * (1 - (1 - 1 / c["adapters"]) ** lanes)
    rows = c["rows"] * (1 - c["none"])
    return {"bytes": int(used * c["rank"] * (c["k"] + c["n"]) * size + (rows * c["k"] + 2 * c["rows"] * c["n"]) * size),
            "flops": int(2 * rows * c["rank"] * (c["k"] + c["n"]))}
