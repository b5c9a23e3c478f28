"""The draw of the next token against the definition in 64 bits.

A token, a count and a logprob follow from sums of weights whose fp32 values
are off by a few units (exp of an fp32 difference times an fp32 reciprocal:
relative at most (|y| + 4) 2^-23, below 1e-5 wherever a weight is not zero).
So they are checked as decisions: where the returned token's share of the
cumulative weight, widened by 1e-5 of the total, holds u, and where the
returned count's prefix reaches its bounds within 1e-5."""
import math

import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

SLACK = 1e-5


@pytest.fixture(scope="module")
def W():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import wfst_beam_search_gb300 as W
    W.load()
    return W


def check_lane(x, u, temp, k, p, min_p, token, logprob, kept):
    x = np.where(np.isnan(x), -np.inf, x.astype(np.float64))
    top = x.max()
    if top == -np.inf:
        assert (token, logprob, kept) == (-1, -math.inf, 0)
        return
    temp, p, min_p = (float(np.float32(v)) for v in (temp, p, min_p))
    if temp == 0:
        assert (token, logprob, kept) == (int(x.argmax()), 0.0, 1)
        return
    with np.errstate(invalid="ignore"):
        w = np.exp(np.where(x == top, 0.0, (x - top) / temp))
    order = np.argsort(-x, kind="stable")
    n = len(x) if k <= 0 or k >= len(x) else k
    assert 1 <= kept <= n
    c = w[order[:n]].cumsum()
    total = c[-1]
    lo, hi = n, n                      # the prefixes that could be the kept one
    if p < 1:
        lo = 1 + int((c[:-1] < (p - SLACK) * total).sum())
        hi = 1 + int((c[:-1] < (p + SLACK) * total).sum())
    if min_p > 0:
        lo = min(lo, int((w >= min_p * (1 + SLACK)).sum()) or 1)
        hi = min(hi, int((w >= min_p * (1 - SLACK)).sum()))
    assert lo <= kept <= hi, (lo, kept, hi)
    mine = np.zeros(len(x), bool)
    mine[order[:kept]] = True
    assert mine[token] and w[token] > 0
    cum = np.where(mine, w, 0.0).cumsum()
    aim = u * cum[-1]
    assert cum[token] - w[token] <= aim + SLACK * cum[-1] and cum[token] >= aim - SLACK * cum[-1]
    assert abs(logprob - math.log(w[token] / cum[-1])) <= SLACK * (2 + abs(math.log(w[token] / cum[-1])))


def check(W, x, u, temp=1.0, k=0, p=1.0, min_p=0.0):
    got = W.sample_tokens(x, u, temperature=temp, top_k=k, top_p=p, min_p=min_p)
    assert [g.dtype for g in got] == [torch.int32, torch.float32, torch.int32]
    lanes = len(x)

    def each(v):
        return v.tolist() if isinstance(v, torch.Tensor) else [v] * lanes

    host = x.float().cpu().numpy()
    for b, args in enumerate(zip(u.tolist(), each(temp), each(k), each(p), each(min_p),
                                 *(g.tolist() for g in got))):
        check_lane(host[b], *args)
    return got


def logits(seed, lanes, vocab, dtype, scale=2.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    x = torch.randn(lanes, vocab, generator=g, device="cuda") * scale
    x[:, :: max(1, vocab // 20)] += torch.rand(lanes, len(range(0, vocab, max(1, vocab // 20))), generator=g,
                                               device="cuda") * 6
    return x.to(dtype), torch.rand(lanes, generator=g, device="cuda")


@pytest.mark.parametrize("dtype", [torch.float32, torch.float16, torch.bfloat16])
@pytest.mark.parametrize("vocab", [1, 2, 3, 31, 100, 1023, 5000, 8193, 32000, 131071, 300000])
def test_against_64_bits(W, vocab, dtype):
    x, u = logits(vocab, 6, vocab, dtype)
    for temp, k, p, min_p in [(1.0, 0, 1.0, 0.0), (0.7, 0, 0.9, 0.0), (1.3, 40, 1.0, 0.0), (1.0, 1, 1.0, 0.0),
                              (1.0, 7, 0.5, 0.0), (0.9, 500, 0.99, 0.01), (1.0, 0, 1.0, 0.05), (0.0, 5, 0.5, 0.1),
                              (5.0, vocab, 0.3, 0.0), (1.0, vocab + 1, 1e-6, 1.0), (100.0, vocab - 1, 0.999, 0.0)]:
        check(W, x, u, temp, max(k, 0), p, min_p)


def test_settings_for_each_lane(W):
    x, u = logits(1, 8, 2000, torch.bfloat16)
    dev = dict(device="cuda")
    check(W, x, u, torch.tensor([1.0, 0.5, 0.0, 2.0, 1.0, 0.8, 1.0, 1e-3], **dev),
          torch.tensor([0, 10, 3, 1999, 2000, -4, 1, 50], dtype=torch.int32, **dev),
          torch.tensor([1.0, 0.9, 0.5, 0.7, 1.0, 0.2, 1.0, 0.95], **dev),
          torch.tensor([0.0, 0.1, 0.0, 0.01, 0.5, 0.0, 1.0, 0.2], **dev))


def test_settings_of_a_lane_that_are_out_of_range(W):
    """Nothing is refused on the device: they count as the nearest ones in range."""
    vocab = 3000
    x, _ = logits(7, 12, vocab, torch.float32)
    x[:] = x[0].clone()
    x[:, 5::7] = -math.inf
    u = torch.full((12,), 0.37, device="cuda")
    inf, nan = math.inf, math.nan
    rows = [(inf, 0, 1.0, 0.0), (3e38, 0, 1.0, 0.0), (-1.0, 0, 1.0, 0.0), (nan, 0, 1.0, 0.0), (0.0, 0, 1.0, 0.0),
            (1.0, -7, 2.0, -0.5), (1.0, 0, 1.0, 0.0), (1.0, 50, -0.3, 0.0), (1.0, 50, nan, 0.0), (1.0, 1, 1.0, 0.0),
            (1.0, 0, 1.0, 7.0), (1.0, 0, 1.0, nan)]
    temp, k, p, min_p = zip(*rows)
    got = W.sample_tokens(x, u, temperature=torch.tensor(temp, device="cuda"),
                          top_k=torch.tensor(k, device="cuda", dtype=torch.int32),
                          top_p=torch.tensor(p, device="cuda"), min_p=torch.tensor(min_p, device="cuda"))
    got = list(zip(*(t.tolist() for t in got)))
    assert got[0] == got[1] and got[2] == got[3] == got[4] and got[5] == got[6]
    assert got[7] == got[8] == got[9] == got[10] == got[11] == got[4]
    host = x[0].cpu().numpy()
    for b in (0, 1, 4, 6):
        check_lane(host, float(u[0]), *((3e38,) + rows[b][1:] if b == 0 else rows[b]), *got[b])


def test_ends_of_the_uniform_range(W):
    x, _ = logits(2, 4, 999, torch.float32)
    u = torch.tensor([0.0, 1.0 - 2.0 ** -24, 0.5, 2.0 ** -40], device="cuda")
    check(W, x, u)
    tokens, _, kept = check(W, x, u, k=20)
    for b in (0, 1):                     # the first and the last index of the kept ones
        best = torch.topk(x[b], 20).indices
        assert int(tokens[b]) == int(best.min() if b == 0 else best.max()) and int(kept[b]) == 20


def test_ties_go_to_the_lowest_index(W):
    for dtype in (torch.float32, torch.bfloat16):
        x = torch.zeros(3, 10000, device="cuda", dtype=dtype)
        x[1, 5000:] = 1.0
        x[2] = -0.0
        x[2, ::2] = 0.0
        u = torch.tensor([0.999999, 0.999999, 0.999999], device="cuda")
        tokens, _, kept = check(W, x, u, k=100)
        assert tokens.tolist() == [99, 5099, 99] and kept.tolist() == [100] * 3
        tokens, _, kept = check(W, x, u, p=0.25)
        assert kept.tolist()[0] == 2500 and tokens.tolist()[0] == 2499
        assert W.sample_tokens(x, u, temperature=0.0)[0].tolist() == [0, 5000, 0]


def test_masked_and_infinite_logits(W):
    x, u = logits(3, 8, 777, torch.float32)
    x[0] = -math.inf
    x[1] = math.nan
    x[2, :] = -math.inf
    x[2, 345] = -3e38
    x[3, 100:] = -math.inf
    x[4, ::2] = math.nan
    x[5, 10] = x[5, 700] = math.inf
    x[6] = torch.finfo(torch.float32).min
    x[7, 3:] = torch.finfo(torch.float32).min
    for kw in (dict(), dict(k=50), dict(p=0.9), dict(k=200, p=0.5, min_p=0.1), dict(temp=0.0), dict(k=776)):
        tokens = check(W, x, u, **kw)[0].tolist()
        assert tokens[0] == tokens[1] == -1 and tokens[2] == 345 and tokens[5] in (10, 700)
    check(W, x[:, :3], u, p=0.5)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
@pytest.mark.parametrize("vocab", [8200, 40001, 131071])
def test_masked_rows_of_a_cluster(W, vocab, dtype):
    """Rows that several CTAs share, with masks that leave nothing, one logit,
    fewer than k of them, those of one CTA, or every other one."""
    x, u = logits(vocab, 8, vocab, dtype)
    x[0] = -math.inf
    x[1] = math.nan
    x[2, :] = -math.inf
    x[2, vocab - 3] = -5.0
    few = torch.randperm(vocab, generator=torch.Generator().manual_seed(1))[:30].cuda()
    some = x[3, few].clone()
    x[3] = -math.inf
    x[3, few] = some
    x[4, 700:] = -math.inf
    x[5, ::2] = math.nan
    x[6, :vocab - 900] = -math.inf
    x[7, [5, vocab // 2, vocab - 1]] = math.inf
    for kw in (dict(), dict(k=50), dict(p=0.9), dict(k=200, p=0.5, min_p=0.1), dict(p=0.95, min_p=0.02),
               dict(temp=0.0), dict(k=vocab - 1)):
        tokens = check(W, x, u, **kw)[0].tolist()
        assert tokens[0] == tokens[1] == -1 and tokens[2] == vocab - 3 and tokens[7] in (5, vocab // 2, vocab - 1)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("vocab", [900, 60000, 1000000])
def test_infinite_logits_leave_no_weight_to_others(W, vocab, dtype):
    """At any temperature, beside logits next to the type's largest number."""
    x, u = logits(9, 4, vocab, dtype)
    large = float(torch.tensor(torch.finfo(dtype).max, dtype=dtype).view(torch.int16 if dtype != torch.float32 else
                                                                         torch.int32).sub(1).view(dtype))
    x[1:, ::3] = large
    x[:2, [17, vocab - 2]] = math.inf
    for temp in (1.0, 5000.0, 3e38):
        for kw in (dict(), dict(k=2), dict(p=0.9), dict(k=700, p=0.999, min_p=1e-6), dict(min_p=1e-7)):
            tokens = check(W, x[:2], u[:2], temp, **kw)[0].tolist()
            assert tokens[0] in (17, vocab - 2) and tokens[1] in (17, vocab - 2)
    check(W, x[2:], u[2:], 5000.0, p=0.9)


def test_strides_alignment_streams_and_repeats(W):
    """Rows at every alignment, rows of a wider tensor, another stream; the same answer every time."""
    for dtype in (torch.float32, torch.float16):
        wide, u = logits(4, 5, 40100, dtype)
        for off in range(9):
            check(W, wide[:, off: off + 40001 + off % 3], u, p=0.95, k=300)
    x = wide[:, 3:39999]
    want = [t.clone() for t in W.sample_tokens(x, u, top_p=0.9)]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        got = W.sample_tokens(x, u, top_p=0.9, stream=side)
        side.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want))


def test_shares_follow_the_weights(W):
    """Over a comb of uniform numbers every token comes up as often as its weight says."""
    lanes, vocab = 4096, 50
    x = torch.randn(1, vocab, device="cuda", generator=torch.Generator("cuda").manual_seed(5)) * 1.5
    u = (torch.arange(lanes, device="cuda") + 0.5) / lanes
    tokens, logprobs, _ = W.sample_tokens(x.expand(lanes, vocab).contiguous(), u)
    share = torch.bincount(tokens.long(), minlength=vocab).double() / lanes
    assert bool(((share - torch.softmax(x[0].double(), 0)).abs() <= 1.01 / lanes).all())
    assert bool((tokens[1:] >= tokens[:-1]).all())


def test_no_lanes_and_refusals(W):
    x, u = logits(6, 3, 100, torch.float32)
    assert [t.shape for t in W.sample_tokens(x[:0], u[:0])] == [(0,)] * 3
    for error, kw in [(TypeError, dict(logits=x.double())), (TypeError, dict(uniform=u.double())),
                      (ValueError, dict(logits=x.cpu())), (ValueError, dict(uniform=u[:2])),
                      (ValueError, dict(logits=x.t().contiguous().t())),
                      (TypeError, dict(top_k=torch.ones(3, device="cuda"))),
                      (ValueError, dict(temperature=torch.ones(2, device="cuda"))),
                      (W.WfstError, dict(temperature=-1.0)), (W.WfstError, dict(temperature=math.nan)),
                      (W.WfstError, dict(temperature=math.inf)), (W.WfstError, dict(top_k=-1)),
                      (W.WfstError, dict(top_p=0.0)), (W.WfstError, dict(min_p=1.5)),
                      (W.WfstError, dict(min_p=-0.1)), (W.WfstError, dict(logits=x[:, :0]))]:
        with pytest.raises(error):
            W.sample_tokens(**{**dict(logits=x, uniform=u), **kw})
