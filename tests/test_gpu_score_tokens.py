"""Scores of given tokens against the definition in 64 bits.

Tolerance: with y = x - max (one rounding, 2^-24 |y|), exp is off by a few
2^-23 and by |y| 2^-22 (the rounding of y and of its product with log2 e),
relative; a thread adds up to V / 256 of the weights after one another and some
30 sums are put together, each 2^-24.  Since |y| e^y < 0.4, log Z is off by at
most z = (V / 256 + 64) 2^-23, a log probability by that and two roundings of
its parts, the entropy by z for either of its sums, relative to sum p |y|.
Alternatives are whole numbers and have to be equal."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

TYPES = [torch.float32, torch.float16, torch.bfloat16]


@pytest.fixture(scope="module")
def W():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import wfst_beam_search_gb300 as W
    W.load()
    return W


def logits(seed, rows, vocab, dtype, spread=2.0, masked=0.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(rows, vocab, generator=g, device="cuda") * spread
    if masked:
        x.masked_fill_(torch.rand(rows, vocab, generator=g, device="cuda") < masked, -math.inf)
    return x.to(dtype), torch.randint(0, vocab, (rows,), generator=g, device="cuda").int()


def check(got, x, tokens, top):
    logprobs, entropy, at, alt = got
    rows, vocab = x.shape
    assert logprobs.shape == entropy.shape == (rows,) and at.shape == alt.shape == (rows, top)
    assert logprobs.dtype == entropy.dtype == alt.dtype == torch.float32 and at.dtype == torch.int32
    d = x.double()
    some = (d > -math.inf).any(1)
    m = torch.where(some, d.amax(1), 0.0)[:, None]
    y = d - m
    e = torch.exp(y)
    total = e.sum(1)
    log_z = torch.log(total)
    far = torch.where(e > 0, e * y.abs(), 0.0).sum(1) / total
    z = (vocab / 256 + 64) * 2.0 ** -23
    # log probabilities
    lp = torch.where(tokens < 0, 0.0, y.gather(1, tokens.clamp(0, vocab - 1).long()[:, None])[:, 0] - log_z)
    lp = torch.where(tokens >= vocab, math.nan, lp)
    lp = torch.where(some | (tokens < 0) | (tokens >= vocab), lp, -math.inf)

    def near(a, b, bound):
        a, b = a.double(), b.float().double()      # (a log probability below fp32's range is -inf)
        same = (a == b) | (a.isnan() & b.isnan())
        return bool((same | ((a - b).abs() <= bound)).all())

    assert near(logprobs, lp, z + 2.0 ** -22 * (lp.abs() + log_z.abs() + 1))
    assert near(entropy, torch.where(some, log_z + far, 0.0), z * (1 + 2 * far) + 2.0 ** -22 * (log_z + far + 1))
    # alternatives
    if top:
        order = torch.sort(d, dim=1, descending=True, stable=True).indices[:, :top]
        best = y.gather(1, order)
        want = torch.where(best > -math.inf, order, -1)
        best = torch.where(best > -math.inf, best - log_z[:, None], -math.inf)
        want = torch.nn.functional.pad(want, (0, top - want.shape[1]), value=-1)
        best = torch.nn.functional.pad(best, (0, top - best.shape[1]), value=-math.inf)
        assert torch.equal(at.long(), want)
        assert near(alt, best, z + 2.0 ** -22 * (best.abs() + log_z.abs()[:, None] + 1))


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("vocab", [1, 2, 3, 7, 8, 9, 31, 63, 64, 65, 100, 255, 257, 1000, 2047, 2049, 5000, 8191, 20000, 65537])
def test_vocabularies(W, vocab, dtype):
    for rows, top, masked in ((5, 0, 0.0), (3, 1, 0.0), (4, 5, 0.5), (33, 64, 0.0)):
        x, t = logits(vocab + rows, rows, vocab, dtype, masked=masked)
        check(W.score_tokens(x, t, top=top), x, t, top)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab,top", [(1, 131071, 20), (2, 1 << 20, 64), (1, 1 << 20, 0), (7, 131072, 1), (64, 131071, 8),
                                            (200, 40000, 33), (700, 20001, 3), (3000, 1500, 64), (1, 40000, 7)])
def test_many_logits_and_rows(W, rows, vocab, top, dtype):
    x, t = logits(rows + top, rows, vocab, dtype)
    check(W.score_tokens(x, t, top=top), x, t, top)


@pytest.mark.parametrize("rows", [1, 40, 600])
@pytest.mark.parametrize("vocab", [1000, 30011])
def test_orders_and_equal_logits(W, rows, vocab):
    """Rows that rise, fall, hold one value, two values, a few among many equal
    ones, the largest at their ends."""
    i = torch.arange(vocab, device="cuda").float()
    kinds = [i / vocab, -i / vocab, i * 0, (i % 2), (i // 37 % 5) * -1, torch.where(i % 501 == 7, 3.0, 1.0),
             torch.where(i == vocab - 1, 5.0, -(i % 3)), torch.where(i == 0, 5.0, i % 3), torch.where(i < 20, -math.inf, 0.0),
             torch.where(i < 20, 0.0, -math.inf), torch.where(i >= vocab - 70, i - vocab, -math.inf)]
    x = torch.stack([kinds[r % len(kinds)] for r in range(max(rows, len(kinds)))])
    for dtype in TYPES:
        z = x.to(dtype)
        for first in range(0, len(x), rows):
            part = z[first:first + rows].contiguous()
            t = (torch.arange(len(part), device="cuda") * 31 % vocab).int()
            for top in (1, 20, 64):
                check(W.score_tokens(part, t, top=top), part, t, top)


@pytest.mark.parametrize("dtype", TYPES)
def test_large_and_far_apart(W, dtype):
    """Logits of one large size, ones that leave one token all the weight, and the type's extremes."""
    big = 60000.0 if dtype == torch.float16 else 3e38
    for x in (logits(1, 6, 3001, dtype, spread=30.0)[0], (logits(2, 6, 3001, torch.float32)[0] + 1000.0).to(dtype),
              logits(3, 6, 3001, dtype, spread=3000.0)[0], torch.where(logits(4, 6, 3001, torch.float32)[0] > 0, big, -big).to(dtype)):
        t = torch.tensor([0, 5, 3000, 7, 8, 9], device="cuda").int()
        check(W.score_tokens(x, t, top=10), x, t, 10)


@pytest.mark.parametrize("rows", [6, 400])
@pytest.mark.parametrize("vocab", [50, 4000, 50000])
def test_rows_without_logits_and_tokens_outside(W, rows, vocab):
    x, t = logits(rows, rows, vocab, torch.bfloat16)
    x[1] = -math.inf
    x[2, 1:] = -math.inf
    x[3] = -math.inf
    x[3, vocab - 1] = -5.0
    t[0], t[1], t[2], t[3], t[4], t[5] = -1, 3, 0, 0, vocab, 2 ** 31 - 1
    check(W.score_tokens(x, t, top=3), x, t, 3)
    t[1], t[2] = -2 ** 31, 1
    check(W.score_tokens(x, t, top=3), x, t, 3)


@pytest.mark.parametrize("rows", [4, 400])
@pytest.mark.parametrize("vocab", [50, 4000, 50000])
def test_nan_and_infinite_logits_stay_in_their_row(W, rows, vocab):
    for bad in (math.nan, math.inf):
        for at in (0, vocab // 2, vocab - 1):
            x, t = logits(rows, rows, vocab, torch.float32)
            clean = W.score_tokens(x, t, top=4)
            x[1, at] = bad
            got = W.score_tokens(x, t, top=4)
            assert all(bool(g[1].isnan().all()) for g in (got[0], got[1], got[3]))
            want = torch.sort(torch.where(x[1].isnan(), -math.inf, x[1]), descending=True, stable=True).indices[:4]
            assert torch.equal(got[2][1].long(), want)
            for g, c in zip(got, clean):
                g[1] = c[1] = 0
                assert torch.equal(g, c)


@pytest.mark.parametrize("dtype", TYPES)
@pytest.mark.parametrize("rows,vocab", [(5, 5000), (300, 777), (2, 60001)])
def test_strides_and_boundaries(W, rows, vocab, dtype):
    """Rows that begin anywhere, in longer rows whose rest is never counted; the same bits each time."""
    x, t = logits(vocab, rows, vocab, dtype)
    for shift, more in ((1, 0), (3, 5), (0, 8), (5, 1), (7, 6)):
        room = torch.full((rows * (vocab + more) + 16,), 1e4, device="cuda", dtype=dtype)
        part = room[shift:shift + rows * (vocab + more)].view(rows, -1)[:, :vocab]
        part.copy_(x)
        got = W.score_tokens(part, t, top=9)
        check(got, x, t, 9)
        assert all(torch.equal(a, b) for a, b in zip(got, W.score_tokens(part, t, top=9)))


def test_offsets_past_32_bits(W):
    rows, vocab = 5, 2 ** 20
    x, t = logits(3, rows, vocab, torch.bfloat16)
    room = torch.empty(5 * 2 ** 29, device="cuda", dtype=torch.bfloat16).view(5, -1)[:, :vocab]
    room.copy_(x)
    check(W.score_tokens(room, t, top=5), x, t, 5)


def test_streams_and_graphs(W):
    x, t = logits(5, 40, 30000, torch.bfloat16)
    want = W.score_tokens(x, t, top=6)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = W.score_tokens(x, t, top=6, stream=side)
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        outs = [W.score_tokens(x, t, top=6) for _ in range(2)]
    y, t2 = logits(6, 40, 30000, torch.bfloat16)
    x.copy_(y), t.copy_(t2)
    graph.replay()
    want = W.score_tokens(y, t2, top=6)
    for got in outs:
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_refusals(W):
    x, t = logits(7, 4, 50, torch.float16)
    assert [tuple(v.shape) for v in W.score_tokens(x[:0], t[:0], top=3)] == [(0,), (0,), (0, 3), (0, 3)]
    for error, change in [
            (TypeError, dict(logits=x.double())), (TypeError, dict(logits=x.int())), (TypeError, dict(tokens=t.long())),
            (TypeError, dict(tokens=[1, 2, 3, 4])), (TypeError, dict(top=1.5)), (TypeError, dict(top=None)),
            (ValueError, dict(tokens=t[:3])), (ValueError, dict(tokens=t.repeat(2)[::2])), (ValueError, dict(tokens=t.cpu())),
            (ValueError, dict(logits=x[0])), (ValueError, dict(logits=x.t().contiguous().t())),
            (ValueError, dict(top=-1)), (ValueError, dict(top=65)), (ValueError, dict(top=2 ** 40)),
            (ValueError, dict(logits=x.clone().requires_grad_())),
            (W.WfstError, dict(logits=x[:, :0])),
            (W.WfstError, dict(logits=torch.zeros(1, 1, device="cuda").expand(4, 2 ** 20 + 1).half()))]:
        with pytest.raises(error):
            W.score_tokens(**{**dict(logits=x, tokens=t, top=2), **change})


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rows,vocab", [(5, 3001), (700, 3001), (700, 70001)])
def test_what_16_bits_hold(W, rows, vocab, dtype):
    """NaN and +inf among 16-bit logits, and rows whose logits are all near the
    type's lowest number, masked and not: two by two they are treated otherwise
    than in fp32."""
    low = -65504.0 if dtype == torch.float16 else -3.3895313892515355e38
    x, t = logits(rows + vocab, rows, vocab, dtype, masked=0.3)
    x[0, 1::2], x[0, ::2] = low, -math.inf
    x[1] = low
    x[2, :] = low
    x[2, vocab // 2] = low * 0.5
    x[3, 5:] = low
    check(W.score_tokens(x, t, top=20), x, t, 20)
    for bad in (math.nan, math.inf):
        for at in (0, 1, vocab - 1):
            y = x.clone()
            y[4, at] = bad
            got, clean = W.score_tokens(y, t, top=4), W.score_tokens(x, t, top=4)
            assert all(bool(g[4].isnan().all()) for g in (got[0], got[1], got[3]))
            want = torch.sort(torch.where(y[4].isnan(), -math.inf, y[4].float()), descending=True, stable=True).indices[:4]
            assert torch.equal(got[2][4].long(), want)
            for g, c in zip(got, clean):
                g[4] = c[4] = 0
                assert torch.equal(g, c)
