"""Rescoring: the operators together, against the same model in 64 bits.

Tolerance, of a row of logits by its norm: as for a plain pass (14 roundings by
u = 2^-11 of a layer's vector), with four more where an adapter's part is added
to a product that has been rounded, and q and k off by one u more each: a
weight of the softmax moves by 128 u instead of 96.  150 u for each of two
layers, doubled for what later layers make of it.  A wrong head, place, page,
prefix or adapter is off by the whole norm."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

LIMIT = 2 * 2 * 150 * 2.0 ** -11


@pytest.fixture(scope="module")
def P():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import wfst_beam_search_gb300 as W
    W.load()
    from wfst_beam_search_gb300 import second_pass
    return second_pass


def shape(P, **more):
    return P.Shape(**{**dict(vocab=777, width=128, layers=2, q_heads=6, kv_heads=2, head_dim=64, hidden=160, group=32),
                      **more})


def adapters_of(s, count, seed):
    """Adapters of some matrices, of several ranks, as large as the matrices themselves."""
    g = torch.Generator().manual_seed(seed)
    heads, t = s.q_heads * s.head_dim, {}
    for i, m, rank, n, k in ((0, "qkv", 16, heads + 2 * s.kv_heads * s.head_dim, s.width), (0, "down", 8, s.width, s.hidden),
                             (1, "out", 24, s.width, heads), (1, "up", 16, 2 * s.hidden, s.width)):
        t[f"{i}.{m}.shrink"] = torch.randn(count, rank, k, generator=g) * k ** -0.5
        t[f"{i}.{m}.expand"] = torch.randn(count, n, rank, generator=g) * rank ** -0.5
    return t


def norm(x, eps):
    return x / (x.square().mean(-1, keepdim=True) + eps).sqrt()


def plain(P, s, tensors, tokens, adapted=None, bare=0):
    """Logits in 64 bits of one lane's tokens; ``adapted``: (tensors, scale, adapter),
    from token ``bare`` on."""
    def take(name):
        t = tensors[name]
        if t.dim() == 1 or name == "embed":
            return t.half().double()
        codes, scales = P.quantize(t, s.group, torch.float16)
        c = torch.stack([codes & 15, codes >> 4], 2).reshape(t.shape).double()
        return (c - 8) * scales.double().repeat_interleave(s.group, 1)

    n, d, hq, hkv = len(tokens), s.head_dim, s.q_heads, s.kv_heads
    angle = torch.arange(n).double()[:, None] * s.base ** (-torch.arange(0, d, 2).double() / d)

    def product(x, name):
        y = x @ take(name).t()
        if adapted and f"{name}.shrink" in adapted[0]:
            a, scale, which = adapted
            shrink, expand = (a[f"{name}.{part}"][which].half().double() for part in ("shrink", "expand"))
            y[bare:] += scale * (x[bare:] @ shrink.t()) @ expand.t()
        return y

    def turn(x):
        a, b = x[..., :d // 2], x[..., d // 2:]
        c, t = angle.cos()[:, None], angle.sin()[:, None]
        return torch.cat([a * c - b * t, b * c + a * t], -1)

    i = torch.arange(n)
    sees = i[:, None] >= i
    if s.window:
        sees &= (i[:, None] - i < s.window) | (i < s.sinks)
    x = take("embed")[tokens]
    for layer in range(s.layers):
        h = product(norm(x, s.eps) * take(f"{layer}.gain1"), f"{layer}.qkv").view(n, hq + 2 * hkv, d)
        q = turn(norm(h[:, :hq], s.eps) * take(f"{layer}.q_gain"))
        k = turn(norm(h[:, hq:hq + hkv], s.eps) * take(f"{layer}.k_gain")).repeat_interleave(hq // hkv, 1)
        v = h[:, hq + hkv:].repeat_interleave(hq // hkv, 1)
        scores = torch.einsum("ihd,jhd->hij", q, k) * d ** -0.5
        p = scores.masked_fill(~sees, float("-inf")).softmax(-1)
        x = x + product(torch.einsum("hij,jhd->ihd", p, v).reshape(n, -1), f"{layer}.out")
        h = product(norm(x, s.eps) * take(f"{layer}.gain2"), f"{layer}.up")
        x = x + product(torch.nn.functional.silu(h[:, :s.hidden]) * h[:, s.hidden:], f"{layer}.down")
    return (norm(x, s.eps) * take("gain")) @ take("head").t()


def read(second, words, adapters=None):
    """Each lane's logits for its words."""
    out = [[] for _ in words]
    for lanes, targets, logits in second._read(words, adapters):
        for b, target, row in zip(lanes, targets.tolist(), logits.double().cpu()):
            assert target == words[b][len(out[b])]
            out[b].append(row)
    return out


@pytest.mark.parametrize("prefix,rows,page", [(0, 16, 4), (0, 256, 16), (1, 7, 4), (16, 12, 4), (61, 16, 4), (150, 64, 16)])
@pytest.mark.parametrize("with_adapters", [False, True])
def test_against_64_bits(P, prefix, rows, page, with_adapters):
    """Words of several lanes, one of them without any, read many at a time
    behind a prefix and with adapters of their own; then the same lanes step by
    step."""
    s = shape(P)
    tensors = P.random_tensors(s, 1)
    g = torch.Generator().manual_seed(prefix + 3)
    words = [torch.randint(0, s.vocab, (n,), generator=g).tolist() for n in (9, 0, 21, 1, 30)]
    before = torch.randint(0, s.vocab, (prefix,), generator=g).tolist()
    lm = P.LanguageModel(s, tensors, torch.float16)
    extra, scales, which = adapters_of(s, 3, 5), [0.5, 1.0, -0.75], [2, 0, None, 1, 2]
    if with_adapters:
        lm.adapt(extra, scales)
    second = P.SecondPass(lm, 5, 40, page_size=page, pages=5 * -(-40 // page) + -(-prefix // page), rows=rows)
    second.read_prefix(before)
    which = which if with_adapters else None
    got = read(second, words, which)
    scores = second.score(words, top=3, adapters=which)
    for b, w in enumerate(words):
        a = which and which[b]
        ref = plain(P, s, tensors, [*before, s.start, *w], None if a is None else (extra, scales[a], a), prefix)[prefix:]
        assert len(got[b]) == len(w) == len(scores[b]["logprobs"])
        if not w:
            continue
        mine, ref = torch.stack(got[b]), ref[:-1]
        assert bool(((mine - ref).norm(dim=1) <= LIMIT * ref.norm(dim=1)).all()), b
        lp = mine.log_softmax(1)                   # of the logits that were scored
        at = torch.tensor(w)[:, None]
        assert (torch.tensor(scores[b]["logprobs"]) - lp.gather(1, at)[:, 0]).abs().max() < 2e-5
        assert (torch.tensor(scores[b]["entropy"]) - torch.special.entr(lp.exp()).sum(1)).abs().max() < 1e-4
        order = torch.sort(mine, dim=1, descending=True, stable=True).indices[:, :3].tolist()
        assert [[t for t, _ in row] for row in scores[b]["alternatives"]] == order
    # step by step, as ``run`` does
    plan, table = second.plan_lanes(words, 1)
    second.table.copy_(torch.from_numpy(table))
    second.which.copy_(torch.tensor([-1 if a is None else a for a in which or [None] * 5]))
    steps = torch.stack([second.logits(*torch.from_numpy(row).cuda().unbind()).double().cpu() for row in plan])
    for b, w in enumerate(words):
        a = which and which[b]
        ref = plain(P, s, tensors, [*before, s.start, *w], None if a is None else (extra, scales[a], a), prefix)[prefix:]
        mine = steps[:len(w) + 1, b]
        assert bool(((mine - ref).norm(dim=1) <= LIMIT * ref.norm(dim=1)).all()), b


def test_runs_behind_a_prefix(P):
    """Graph and single steps agree; another prefix is another pass; none is
    the pass without; adapters belong to their lanes."""
    s = shape(P)
    lm = P.LanguageModel.random(s)
    lm.adapt(adapters_of(s, 2, 7))
    words = [[1, 2, 3], [], list(range(20, 50)), [700]]
    second = P.SecondPass(lm, 5, 64, page_size=16, pages=25)
    bare = second.run(words, 12, top_p=0.9, seed=4)
    second.read_prefix(range(100))
    first = second.run(words, 12, top_p=0.9, seed=4)
    assert first != bare and second.run(words, 12, top_p=0.9, seed=4) == first
    assert second.run(words, 12, top_p=0.9, seed=4, graph=False) == first
    second.read_prefix(range(100, 190))
    assert second.run(words, 12, top_p=0.9, seed=4) != first
    second.read_prefix(list(range(100)))
    assert second.run(words, 12, top_p=0.9, seed=4) == first
    mixed = second.run(words, 12, top_p=0.9, seed=4, adapters=[None, 1, None, 0])
    assert mixed[0] == first[0] and mixed[2] == first[2] and mixed[1] != first[1] and mixed[3] != first[3]
    assert second.run(words, 12, top_p=0.9, seed=4) == first
    second.read_prefix(None)
    assert second.run(words, 12, top_p=0.9, seed=4) == bare
    # what is likely scores higher than what is not
    best = second.run([[5]], 8, temperature=0.0)[0]["tokens"]
    good, bad = second.score([[5, *best], [5, *[(t + 300) % s.vocab for t in best]]])
    assert sum(good["logprobs"][1:]) > sum(bad["logprobs"][1:])
    assert all(v >= 0 for a in (good, bad) for v in a["entropy"])
    assert second.score([[], []]) == [{"logprobs": [], "entropy": []}] * 2 and second.score([]) == []


def test_other_adapters_after_a_pass(P):
    """A step that was captured with other adapters, or with none, is not run again."""
    s = shape(P)
    words, which = [[1, 2, 3], list(range(20, 50)), [700]], [1, None, 0]
    lm = P.LanguageModel.random(s)
    second = P.SecondPass(lm, 3, 64, page_size=16)
    seen = [second.run(words, 12, top_p=0.9, seed=4)]
    for seed in (7, 8):
        lm.adapt(adapters_of(s, 2, seed))
        seen.append(second.run(words, 12, top_p=0.9, seed=4, adapters=which))
        assert second.run(words, 12, top_p=0.9, seed=4, adapters=which, graph=False) == seen[-1]
        assert seen[-1][1] == seen[0][1] and seen[-1][0] != seen[0][0]
    assert seen[1][0] != seen[2][0]


def test_windows_score_too(P):
    s = shape(P, window=7, sinks=2)
    tensors = P.random_tensors(s, 2)
    second = P.SecondPass(P.LanguageModel(s, tensors, torch.float16), 2, 40, page_size=4, rows=11)
    words = [list(range(5, 35)), list(range(300, 318))]
    for b, rows in enumerate(read(second, words)):
        ref, mine = plain(P, s, tensors, [s.start, *words[b]])[:-1], torch.stack(rows)
        assert bool(((mine - ref).norm(dim=1) <= LIMIT * ref.norm(dim=1)).all())
    with pytest.raises(ValueError, match="window"):
        second.read_prefix([1])


def test_refusals(P):
    s = shape(P)
    lm = P.LanguageModel.random(s)
    second = P.SecondPass(lm, 2, 32, page_size=16, pages=5)
    for bad in ([777], [-1], [1] * 81):
        with pytest.raises(ValueError):
            second.read_prefix(bad)
    second.read_prefix([1] * 40)                     # three of the five pages
    with pytest.raises(ValueError, match="pool has 2"):
        second.run([[1] * 10, [1] * 20], 2)
    for change in (dict(top=-1), dict(top=65), dict(adapters=[0, 0]), dict(adapters=[None])):
        with pytest.raises(ValueError):
            second.score([[1], [2]], **change)
    with pytest.raises(ValueError):
        second.score([[777], [2]])
    extra = adapters_of(s, 2, 1)
    for change in ({"0.qkv.shrink": None}, {"5.qkv.shrink": extra["0.qkv.shrink"]}, {"0.qkv.expand": extra["0.qkv.expand"][:1]},
                   {"0.qkv.expand": extra["0.qkv.expand"][:, :, :8]}, {"0.qkv.shrink": extra["0.qkv.shrink"][:, :12],
                                                                        "0.qkv.expand": extra["0.qkv.expand"][:, :, :12]}):
        with pytest.raises(ValueError):
            lm.adapt({k: v for k, v in {**extra, **change}.items() if v is not None})
    with pytest.raises(ValueError):
        lm.adapt({})
    with pytest.raises(ValueError):
        lm.adapt(extra, [1.0])
    lm.adapt(extra, [1.0, math.pi])
    with pytest.raises(ValueError):
        second.run([[1]], 1, adapters=[2])
