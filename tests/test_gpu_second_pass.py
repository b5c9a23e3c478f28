"""The second pass: the operators together, against the same model in 64 bits.

Tolerance, of a row of logits by its norm: with u = 2^-11 a layer rounds some
14 times by u of its vector; q and k, off by 3 u each, move a score (at most
sqrt(d) in size times the gains, d = 64, the heads being normed) by 6 u sqrt(d)
and a weight of the softmax by twice that, 96 u.  110 u for each of two layers, doubled for what
later layers make of it.  A wrong head, place or page is off by the whole
norm."""
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

LIMIT = 2 * 2 * 110 * 2.0 ** -11


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


def norm(x, eps):
    return x / (x.square().mean(-1, keepdim=True) + eps).sqrt()


def plain(P, s, tensors, tokens):
    """Logits in 64 bits of one lane's tokens, one after the other."""
    def take(name):
        t = tensors[name]
        if t.dim() == 1 or name == "embed":
            return t.half().double()
        codes, scales = P.quantize(t, s.group, torch.float16)
        c = torch.stack([codes & 15, codes >> 4], 2).reshape(t.shape).double()
        return (c - 8) * scales.double().repeat_interleave(s.group, 1)

    n, d, hq, hkv = len(tokens), s.head_dim, s.q_heads, s.kv_heads
    angle = torch.arange(n).double()[:, None] * s.base ** (-torch.arange(0, d, 2).double() / d)

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
        def w(name):
            return take(f"{layer}.{name}")
        h = ((norm(x, s.eps) * w("gain1")) @ w("qkv").t()).view(n, hq + 2 * hkv, d)
        q = turn(norm(h[:, :hq], s.eps) * w("q_gain"))
        k = turn(norm(h[:, hq:hq + hkv], s.eps) * w("k_gain")).repeat_interleave(hq // hkv, 1)
        v = h[:, hq + hkv:].repeat_interleave(hq // hkv, 1)
        scores = torch.einsum("ihd,jhd->hij", q, k) * d ** -0.5
        p = scores.masked_fill(~sees, float("-inf")).softmax(-1)
        x = x + torch.einsum("hij,jhd->ihd", p, v).reshape(n, -1) @ w("out").t()
        h = (norm(x, s.eps) * w("gain2")) @ w("up").t()
        x = x + (torch.nn.functional.silu(h[:, :s.hidden]) * h[:, s.hidden:]) @ w("down").t()
    return (norm(x, s.eps) * take("gain")) @ take("head").t()


@pytest.mark.parametrize("window,sinks,lanes", [(0, 0, 3), (7, 2, 3), (5, 0, 20)])
def test_against_64_bits(P, window, sinks, lanes):
    """Lanes of several lengths, one of them without words, in one pool of
    small pages: every step's logits."""
    s = shape(P, window=window, sinks=sinks)
    tensors = P.random_tensors(s, 1)
    tensors = {n: t * (0.5 + torch.rand(t.shape, generator=torch.Generator().manual_seed(2))) if "gain" in n else t
               for n, t in tensors.items()}
    g = torch.Generator().manual_seed(3)
    words = [torch.randint(0, s.vocab, (n % 29,), generator=g).tolist() for n in range(0, 9 * lanes, 9)]
    second = P.SecondPass(P.LanguageModel(s, tensors, torch.float16), lanes, 40, page_size=4)
    plan, table = second.plan_lanes(words, 1)
    second.table.copy_(torch.from_numpy(table))
    got = torch.stack([second.logits(*torch.from_numpy(row).cuda().unbind()).double().cpu() for row in plan])
    for b, w in enumerate(words):
        ref = plain(P, s, tensors, [s.start, *w])
        mine = got[:len(w) + 1, b]
        assert bool(((mine - ref).norm(dim=1) <= LIMIT * ref.norm(dim=1)).all())


def test_graph_and_steps_agree(P):
    lm = P.LanguageModel.random(shape(P))
    second = P.SecondPass(lm, 5, 64, page_size=16, pages=14)
    words = [[1, 2, 3], [], list(range(20, 50)), [700]]
    first = second.run(words, 12, top_p=0.9, seed=4)
    assert [len(a["tokens"]) for a in first] == [12] * 4
    assert all(0 <= t < 777 for a in first for t in a["tokens"])
    assert all(v <= 0 for a in first for v in a["logprobs"])
    assert second.run(words, 12, top_p=0.9, seed=4, graph=False) == first
    assert second.run(words, 12, top_p=0.9, seed=5) != first
    assert second.run(words, 12, top_p=0.9, seed=4) == first
    # the largest logit needs no random number
    assert second.run(words, 12, temperature=0.0, seed=1) == second.run(words, 12, temperature=0.0, seed=2)
    assert second.run([], 3) == []


def test_logits_without_a_number_end_an_answer(P):
    """A lane that reads a token whose embedding is not finite has no logits
    from there on: its answer is -1, its neighbours' answers stay, and the
    model goes on being of use."""
    s = shape(P)
    tensors = P.random_tensors(s)
    clean = [[1, 2], [3, 4, 5], [6]]
    want = P.SecondPass(P.LanguageModel(s, tensors), 3, 32).run(clean, 9, top_p=0.9, seed=4)
    drawn = {t for a in want for t in a["tokens"]}
    bad = next(t for t in range(7, s.vocab) if t not in drawn)
    tensors["embed"][bad] = float("nan")
    for graph in (True, False):
        second = P.SecondPass(P.LanguageModel(s, tensors), 3, 32)
        got = second.run([clean[0], [3, bad, 5], clean[2]], 9, top_p=0.9, seed=4, graph=graph)
        assert got[0] == want[0] and got[2] == want[2]
        assert got[1] == {"tokens": [-1] * 9, "logprobs": [-float("inf")] * 9}
        assert second.run(clean, 9, top_p=0.9, seed=4, graph=graph) == want


def test_refusals(P):
    lm = P.LanguageModel.random(shape(P))
    second = P.SecondPass(lm, 2, 32, page_size=16, pages=3)
    for words, new in (([[1]] * 3, 4), ([[1]], 0), ([[1] * 30], 3), ([[1] * 20, [1] * 20], 4), ([[777]], 1), ([[-1]], 1)):
        with pytest.raises(ValueError):
            second.run(words, new)
    tensors = P.random_tensors(shape(P))
    del tensors["1.up"]
    with pytest.raises(ValueError):
        P.LanguageModel(shape(P), tensors)


def test_after_a_first_pass(P):
    import synth
    import wfst_beam_search_gb300 as W
    wl, g = synth.workload(0), synth.make_graph(0)
    dec = W.Decoder(W.Graph(g, device=0), W.make_params(wl.search_beam, wl.output_beam, wl.min_active, wl.max_active, True),
                    max_lanes=wl.B, max_frames=wl.T)
    before = dec.decode(torch.from_numpy(synth.make_log_probs(0)).cuda(), synth.make_lens(0))
    words = [[int(w) for w in r["words"]] for r in before]
    lm = P.LanguageModel.random(shape(P, vocab=int(g["olabel"].max()) + 1))
    second = P.SecondPass(lm, len(words), max(map(len, words)) + 8)
    assert all(len(a["tokens"]) == 8 for a in second.run(words, 8))
    after = dec.decode(torch.from_numpy(synth.make_log_probs(0)).cuda(), synth.make_lens(0))
    assert [list(r["words"]) for r in after] == [list(r["words"]) for r in before]


@pytest.mark.parametrize("scale", [0.0055, 0.0012])     # values that leave fp16's range, ones that stay
@pytest.mark.parametrize("lanes", [3, 40])
def test_calls_follow_each_other(P, lanes, scale):
    """A chain of calls that read what the one before wrote, in buffers that
    are used again, gives the same bits as with a wait after each call."""
    import wfst_beam_search_gb300 as W
    g = torch.Generator(device="cuda")
    g.manual_seed(6)
    hq, hkv, d, page, steps = 24, 8, 64, 16, 60

    def matrix(n, k):
        codes = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
        return W.pack_quant(codes, torch.full((n, k // 128), scale, device="cuda").half())

    up, down = matrix((hq + 2 * hkv) * d, hq * d), matrix(hq * d, hq * d)
    start = torch.randn(lanes, hq * d, generator=g, device="cuda").half()
    uniform = torch.rand(steps, lanes, generator=g, device="cuda")
    angle = torch.rand(steps, d // 2, generator=g, device="cuda") * 6
    rotary = torch.cat([angle.cos(), angle.sin()], 1)
    width = -(-steps // page)
    table = torch.randperm(lanes * width, generator=g, device="cuda").int().view(lanes, width)
    at = torch.arange(steps, device="cuda")
    slots = (table[:, at // page] * page + at % page).t().int().contiguous()
    lengths = (at + 1).int()[:, None].repeat(1, lanes)
    positions = at.int()[:, None].repeat(1, lanes)
    ws = W.attend_workspace()

    def chain(wait):
        x, h, o = start.clone(), start.new_empty(lanes, (hq + 2 * hkv) * d), start.new_empty(lanes, hq, d)
        cache = torch.zeros(2, lanes * width, page, hkv, d, device="cuda").half()
        tokens = []
        torch.cuda.synchronize()
        for i in range(steps):
            W.matvec_quant(x, up, out=h)
            wait()
            heads = h.view(lanes, -1, d)
            W.norm_rotate(heads[:, :hq], heads[:, hq:hq + hkv], heads[:, hq + hkv:], positions[i], rotary, None, None,
                          cache[0], cache[1], slots[i], out=heads[:, :hq])
            wait()
            W.attend_paged(heads[:, :hq], cache[0], cache[1], table, lengths[i], workspace=ws, out=o)
            wait()
            W.matvec_quant(o.view(lanes, -1), down, out=x)
            wait()
            tokens.append(W.sample_tokens(x, uniform[i], top_p=0.9)[0])
            wait()
        assert bool(x.isfinite().all()) == (scale < 0.002)
        return x.view(torch.int16), cache.view(torch.int16), torch.stack(tokens)

    want = chain(torch.cuda.synchronize)
    for _ in range(5):
        got = chain(lambda: None)
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_gradients_are_refused_and_writes_are_known(P):
    """No operator gives a gradient, so none cuts one off in silence; what is
    written in place counts as changed."""
    import wfst_beam_search_gb300 as W
    dev = dict(device="cuda")
    x = torch.randn(2, 64, **dev).half()
    w = W.pack_quant(torch.zeros(64, 32, dtype=torch.uint8, **dev), torch.ones(64, 1, **dev).half())
    i, one = torch.zeros(2, dtype=torch.int32, **dev), torch.ones(2, dtype=torch.int32, **dev)
    pages, rotary = torch.zeros(2, 2, 16, 1, 64, **dev).half(), torch.zeros(4, 64, **dev)
    slots = torch.arange(2, dtype=torch.int32, **dev)

    def calls(x, out, kc, vc):
        h = x[:, None]
        yield lambda: W.matvec_quant(x, w, out=out)
        yield lambda: W.norm_rotate(h, h, h, i, rotary, None, None, kc, vc, slots, out=out[:, None])
        yield lambda: W.attend_paged(h, kc, vc, i[:, None], one, out=out[:, None])
        yield lambda: W.sample_tokens(x, torch.zeros(2, **dev))

    asks = x.clone().requires_grad_()
    out, kc, vc = torch.empty_like(x), pages[0].clone(), pages[1].clone()
    for call in calls(asks, out, kc, vc):
        with pytest.raises(ValueError, match="gradient"):
            call()
        with torch.no_grad():
            call()
    for call, (of_out, of_cache) in zip(calls(x, out, kc, vc), [(1, 0), (1, 1), (1, 0), (0, 0)]):
        before = out._version, kc._version, vc._version
        call()
        assert (out._version, kc._version, vc._version) == (before[0] + of_out, before[1] + of_cache, before[2] + of_cache)
    with torch.inference_mode():
        for call in calls(x.clone(), torch.empty_like(x), *pages.clone()):
            call()
    with pytest.raises(ValueError, match="gradient"):
        W.pack_quant(torch.zeros(64, 32, dtype=torch.uint8, **dev), torch.ones(64, 1, **dev).half().requires_grad_())
    # weights that are parameters
    s = shape(P)
    tensors = {n: torch.nn.Parameter(t) for n, t in P.random_tensors(s).items()}
    want = P.SecondPass(P.LanguageModel.random(s), 1, 16).run([[1, 2]], 3)
    assert P.SecondPass(P.LanguageModel(s, tensors), 1, 16).run([[1, 2]], 3) == want
