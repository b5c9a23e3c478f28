"""Attention of one new token over a paged cache against the formula in 64
bits.

Tolerance: o is rounded once (u of it); in front of that, scores are fp32 sums
of d products, off by at most (d + 8) * 2^-23 of the terms' size (for a score:
scale * sum |q k|, here called r), which changes a weight by that much,
relative; the weights add up in fp32 in any split.  So o is off by at most
u |o| + (2 r (d + 8) + n / 8 + 64) 2^-23 sum p |v|, and the 16-bit halves of P
leave 2^-16 (bf16: two times 8 bits) of sum p |v| at most."""
import math

import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")

UNIT = {torch.float16: 2.0 ** -11, torch.bfloat16: 2.0 ** -8}


@pytest.fixture(scope="module")
def W():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import wfst_beam_search_gb300 as W
    W.load()
    return W


@pytest.fixture(scope="module")
def ws(W):
    return W.attend_workspace("cuda")


def visible(n, window, sinks):
    start = max(0, n - window) if window else 0
    return list(range(min(sinks, start) if window else 0)) + list(range(start, n))


def make(seed, lens, hq, hkv, d, page, dtype, window=0, sinks=0, spread=1.5):
    """Inputs whose pages lie anywhere; what no lane sees is NaN, pages and table entries alike."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    width = max(1, -(-max(lens) // page)) + 1
    table = torch.full((len(lens), width), -7, dtype=torch.int32)
    ids = [(b, i) for b, n in enumerate(lens) for i in sorted({j // page for j in visible(n, window, sinks)})]
    order = torch.randperm(len(ids) + 2, generator=g, device="cuda").cpu()[: len(ids)]
    shape = (len(ids) + 2, page, hkv, d)
    kc, vc = (torch.full(shape, math.nan, device="cuda", dtype=dtype) for _ in range(2))
    for (b, i), o in zip(ids, order.tolist()):
        table[b, i] = o
    table = table.cuda()
    for b, n in enumerate(lens):
        j = torch.tensor(visible(n, window, sinks), dtype=torch.long, device="cuda")
        if len(j):
            at = (table[b][j // page].long(), j % page)
            kc[at] = torch.randn(len(j), hkv, d, generator=g, device="cuda").to(dtype)
            vc[at] = torch.randn(len(j), hkv, d, generator=g, device="cuda").to(dtype)
    q = (torch.randn(len(lens), hq, d, generator=g, device="cuda") * spread).to(dtype)
    return q, kc, vc, table, torch.tensor(lens, dtype=torch.int32, device="cuda")


def check(o, lse, q, kc, vc, table, lens, scale, window=0, sinks=0, seen=None):
    page, hkv, d = kc.shape[1:]
    share = q.shape[1] // hkv
    for b, n in enumerate(lens.tolist()):
        j = torch.tensor(seen[b] if seen else visible(n, window, sinks), dtype=torch.long, device="cuda")
        if not len(j):
            assert bool((o[b] == 0).all()) and bool((lse[b] == -math.inf).all())
            continue
        at = (table[b][j // page].long(), j % page)
        k, v = (c[at].double().repeat_interleave(share, 1) for c in (kc, vc))
        x = torch.einsum("hd,jhd->hj", q[b].double(), k) * scale
        r = (torch.einsum("hd,jhd->hj", q[b].double().abs(), k.abs()) * abs(scale)).amax(1)
        p = torch.softmax(x, 1)
        ref, size = torch.einsum("hj,jhd->hd", p, v), torch.einsum("hj,jhd->hd", p, v.abs())
        fp = (2 * r * (d + 8) + len(j) / 8 + 64)[:, None] * 2.0 ** -23
        bound = UNIT[o.dtype] * ref.abs() + (fp + 2.0 ** -16) * size + 2.0 ** -24
        assert bool(((o[b].double() - ref).abs() <= bound).all()), (b, n)
        assert bool(((lse[b].double() - torch.logsumexp(x, 1)).abs() <= fp[:, 0]).all()), (b, n)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 4), (6, 2), (8, 1), (18, 2), (16, 1), (40, 2)])
def test_head_layouts(W, ws, hq, hkv, d, dtype):
    a = make(hq * d, [1, 0, 17, 64, 65, 333], hq, hkv, d, 16, dtype)
    check(*W.attend_paged(*a, workspace=ws, with_lse=True), *a, d ** -0.5)


@pytest.mark.parametrize("page", [1, 7, 16, 64, 100])
@pytest.mark.parametrize("window,sinks", [(0, 0), (1, 0), (1, 3), (63, 1), (64, 4), (200, 40), (5000, 4)])
def test_lengths_pages_and_windows(W, ws, page, window, sinks):
    lens = [0, 1, 2, 3, 4, 5, 15, 16, 31, 63, 64, 65, 67, 68, 69, 127, 128, 129, 200, 240, 241, 1000, 3001]
    a = make(page + window, lens, 4, 2, 64, page, torch.bfloat16, window, sinks)
    check(*W.attend_paged(*a, window=window, sinks=sinks, workspace=ws, with_lse=True), *a, 0.125, window, sinks)


@pytest.mark.parametrize("lens", [[40000], [20000, 1, 30011], [1] * 700, [0] * 5, [0, 9000, 0, 0, 129], [130] * 331])
def test_splits(W, ws, lens):
    """One lane over all CTAs, lanes that share CTAs, more lanes than threads of one."""
    a = make(len(lens), lens, 8, 2, 128, 32, torch.bfloat16)
    check(*W.attend_paged(*a, workspace=ws, with_lse=True), *a, 128 ** -0.5)


def test_a_workspace_whose_parts_hold_anything(W):
    """Only its first bytes have to be zeros; the parts are written before they are read."""
    a = make(3, [20000, 1, 30011, 0, 700], 24, 2, 128, 32, torch.bfloat16)
    ws = W.attend_workspace("cuda")
    ws[W.WFST_ATTEND_ZEROED:] = 255                      # NaN
    for _ in range(2):
        check(*W.attend_paged(*a, workspace=ws, with_lse=True), *a, 128 ** -0.5)
        assert not bool(ws[:W.WFST_ATTEND_ZEROED].any())


def test_large_scores_and_other_scale(W, ws):
    """Weights that are nearly all on one key, and a negative scale."""
    a = make(5, [700, 64, 33], 8, 4, 64, 16, torch.float16, spread=30.0)
    check(*W.attend_paged(*a, workspace=ws, with_lse=True), *a, 0.125)
    check(*W.attend_paged(*a, scale=-0.02, workspace=ws, with_lse=True), *a, -0.02)


@pytest.mark.parametrize("d,hq,hkv", [(64, 2, 2), (128, 12, 1), (256, 8, 1)])
@pytest.mark.parametrize("gap", [8.0, 12.0, 14.0, 16.0, 17.0, 17.4, 20.0])
def test_weights_far_below_the_largest_fp16(W, ws, gap, d, hq, hkv):
    """One key `gap` above thousands of others, whose value is zero: what o
    holds comes from the others alone.  Here P's halves have to hold small
    weights: each is rounded twice to 11 bits, 2^-24 of it, or by half a step
    below fp16's smallest exponent, 2^-25 where the largest weight is 2^15.
    (No slack of 2^-16.)"""
    n, page = 20011, 64
    g = torch.Generator(device="cuda")
    g.manual_seed(int(gap * 10) + d)
    pages = -(-n // page)
    table = torch.randperm(pages, generator=g, device="cuda").int()[None]
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    for peak in (0, 7000, n - 1):
        kc = torch.zeros(pages, page, hkv, d, device="cuda").half()
        vc = ((torch.rand(pages, page, hkv, d, generator=g, device="cuda") + 0.5) * 4096).half()
        q = torch.zeros(1, hq, d, device="cuda").half()
        q[..., 3] = 1.0
        kc[..., 3] = (torch.rand(pages, page, hkv, generator=g, device="cuda") * 0.5).half()
        at = int(table[0, peak // page])
        kc[at, peak % page, :, 3] = gap
        vc[at, peak % page] = 0
        o, lse = W.attend_paged(q, kc, vc, table, lens, scale=1.0, workspace=ws, with_lse=True)
        j = torch.arange(n, device="cuda")
        k, v = (c[table[0][j // page].long(), j % page].double().repeat_interleave(hq // hkv, 1) for c in (kc, vc))
        x = torch.einsum("hd,jhd->hj", q[0].double(), k)
        p = torch.softmax(x, 1)
        ref = torch.einsum("hj,jhd->hd", p, v)
        fp = (2 * gap * (d + 8) + n / 8 + 64) * 2.0 ** -23
        lost = 2.0 ** -40 * v.sum(0) / torch.exp(x - x.amax(1, keepdim=True)).sum(1)[:, None]
        assert bool(((o[0].double() - ref).abs() <= (2.0 ** -11 + fp + 2.0 ** -23) * ref + lost + 2.0 ** -24).all()), peak
        assert bool(((lse[0].double() - torch.logsumexp(x, 1)).abs() <= fp).all())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_weights_keep_their_fp32_value(W, ws, dtype):
    """Values that cancel all but the last bits of a weight: three keys of
    weight 1 hold p = exp(-x) in three parts of the type, the fourth, of weight
    p, holds -1.  What is left is the error of p itself: exp2 (2^-22), the
    score's three roundings (3 times 2^-24 of at most 4) and the sums (a few
    2^-24), below 2^-20 of the terms; p in 16 bits would leave up to 2^-19."""
    lanes, d = 3000, 64
    x = torch.linspace(0.02, 2.7, lanes, device="cuda").to(dtype).double()
    p, parts = torch.exp(-x), []
    rest = p.clone()
    for _ in range(3):
        parts.append(rest.to(dtype))
        rest = rest - parts[-1].double()
    kc = torch.zeros(lanes, 4, 1, d, device="cuda", dtype=dtype)
    kc[:, 3, 0, 0] = -x.to(dtype)
    vc = torch.stack([*parts, -torch.ones_like(parts[0])], 1)[:, :, None, None].expand(lanes, 4, 1, d).contiguous()
    q = torch.zeros(lanes, 1, d, device="cuda", dtype=dtype)
    q[..., 0] = 1.0
    table = torch.arange(lanes, device="cuda").int()[:, None]
    lens = torch.full((lanes,), 4, device="cuda").int()
    o = W.attend_paged(q, kc, vc, table, lens, scale=1.0, workspace=ws)[:, 0].double()
    w = torch.stack([torch.ones_like(p)] * 3 + [p], 1) / (3 + p)[:, None]
    ref, size = (w * vc[:, :, 0, 0].double()).sum(1), (w * vc[:, :, 0, 0].double().abs()).sum(1)
    bound = UNIT[dtype] * ref.abs() + 2.0 ** -20 * size + (2.0 ** -25 if dtype == torch.float16 else 0)
    assert bool(((o - ref[:, None]).abs() <= bound[:, None]).all())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("power", range(8, 31, 2))
def test_huge_scores(W, ws, power, dtype):
    """Scores of up to 2^30 whose differences leave one key all the weight: o
    is its value to the bit, lse its score to the roundings of a product."""
    n, d, page = 1500, 64, 16
    g = torch.Generator(device="cuda")
    g.manual_seed(power)
    pages = -(-n // page)
    table = torch.randperm(pages, generator=g, device="cuda").int()[None]
    kc = torch.zeros(pages, page, 1, d, device="cuda", dtype=dtype)
    vc = torch.randn(pages, page, 1, d, generator=g, device="cuda").to(dtype)
    size = 2.0 ** (power // 2)                     # of q's one element and of the keys'
    q = torch.zeros(1, 3, d, device="cuda", dtype=dtype)
    q[0, 0, 7], q[0, 1, 7], q[0, 2, 7] = size, -size, size * 0.75
    score = torch.linspace(-0.5, 0.5, n, device="cuda", dtype=torch.float64)[torch.randperm(n, generator=g, device="cuda")] * size
    best, worst = 777, 40
    score[best], score[worst] = size, -size
    j = torch.arange(n, device="cuda")
    at = table[0][j // page].long(), j % page
    kc[at[0], at[1], 0, 7] = score.to(dtype)
    lens = torch.tensor([n], dtype=torch.int32, device="cuda")
    o, lse = W.attend_paged(q, kc, vc, table, lens, scale=1.0, workspace=ws, with_lse=True)
    v = vc[at][:, 0]
    assert torch.equal(o[0], torch.stack([v[best], v[worst], v[best]]))
    want = torch.tensor([1.0, 1.0, 0.75], device="cuda", dtype=torch.float64) * 4.0 ** (power // 2)
    assert bool(((lse[0].double() - want).abs() <= 8 * 2.0 ** -24 * want).all())


def test_missing_pages_and_long_lengths(W, ws):
    """Tokens of pages outside the pool are not seen; a length past the table ends with it."""
    lens = [100, 100, 64]
    q, kc, vc, table, n = make(6, lens, 2, 1, 64, 16, torch.bfloat16)
    table = table[:, :6].contiguous()            # 96 tokens
    table[0, 2], table[1, 0], table[1, 5], table[2] = -1, kc.shape[0], 2 ** 31 - 1, -2 ** 31
    seen = [[j for j in range(96) if j // 16 != 2], list(range(16, 80)), []]
    big = torch.tensor([100, 2 ** 31 - 1, 64], dtype=torch.int32, device="cuda")
    o, lse = W.attend_paged(q, kc, vc, table, big, workspace=ws, with_lse=True)
    check(o, lse, q, kc, vc, table, n, 0.125, seen=seen)
    n[:] = -5
    o, lse = W.attend_paged(q, kc, vc, table, n, workspace=ws, with_lse=True)
    assert bool((o == 0).all()) and bool((lse == -math.inf).all())


def test_infinities_and_nan_in_seen_places(W, ws):
    """What is seen counts as the formula says: a NaN spreads to its own lane
    and heads alone, a key of weight zero (-inf score) weighs nothing."""
    q, kc, vc, table, n = make(7, [50, 50], 4, 2, 64, 16, torch.float16)
    clean = W.attend_paged(q, kc, vc, table, n, workspace=ws)
    vc2 = vc.clone()
    vc2[table[1, 1].long(), 3, 1, 5] = math.nan
    o = W.attend_paged(q, kc, vc2, table, n, workspace=ws)
    assert torch.equal(o[0], clean[0]) and torch.equal(o[1, :2], clean[1, :2])
    assert bool(o[1, 2:, 5].isnan().all()) and int(o[1, 2:].isnan().sum()) == 2
    q[:] = 1.0
    kc2 = kc.clone()
    kc2[table[0, 0].long(), 2] = -65504.0
    kc2[table[0, 0].long(), 2, :, 0] = -math.inf
    o, lse = W.attend_paged(q, kc2, vc, table, n, workspace=ws, with_lse=True)
    seen = [[j for j in range(50) if j != 2], list(range(50))]
    check(o, lse, q, kc2, vc, table, n, 0.125, seen=seen)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("lens,hq,hkv,d", [([30000], 16, 2, 64), ([9000, 1, 0, 20011, 3], 40, 2, 128), ([130] * 331, 6, 2, 256),
                                           ([70, 64, 5000], 4, 4, 64)])
def test_into_the_queries_themselves(W, ws, lens, hq, hkv, d, dtype):
    """Lanes that many CTAs share, and many lanes of one CTA: all have read a
    head's query before its result is written."""
    q, kc, vc, table, n = make(len(lens), lens, hq, hkv, d, 32, dtype)
    for shift in (0, 8):                # heads on cache lines of their own, and across them
        for _ in range(5):
            room = torch.zeros(len(lens) * hq * d + 8, device="cuda", dtype=dtype)
            x = room[shift:shift + q.numel()].view(q.shape).copy_(q)
            want = W.attend_paged(x, kc, vc, table, n, workspace=ws, with_lse=True)
            got = W.attend_paged(x, kc, vc, table, n, workspace=ws, with_lse=True, out=x)
            assert got[0] is x and torch.equal(x, want[0]) and torch.equal(got[1], want[1])


def test_an_infinite_value_stays_in_its_element(W, ws):
    q, kc, vc, table, n = make(12, [50, 3000], 4, 2, 64, 16, torch.bfloat16)
    clean = W.attend_paged(q, kc, vc, table, n, workspace=ws)
    vc[table[1, 1].long(), 3, 1, 5] = math.inf
    o = W.attend_paged(q, kc, vc, table, n, workspace=ws)
    assert not bool(o[1, 2:, 5].isfinite().any())
    o[1, 2:, 5] = clean[1, 2:, 5]
    assert torch.equal(o, clean)


def test_layouts_streams_and_repeats(W, ws):
    """Heads before places, q and o as parts of wider tensors, a table with
    longer rows, another stream with a workspace of its own; the same bits
    every time."""
    q, kc, vc, table, n = make(8, [5000, 300, 1, 77], 12, 4, 128, 16, torch.bfloat16)
    kc, vc = (c.transpose(1, 2).contiguous().transpose(1, 2) for c in (kc, vc))
    wide = torch.zeros(4, 20, 128, device="cuda", dtype=torch.bfloat16)
    wide[:, 4:16] = q
    q = wide[:, 4:16]
    long = torch.zeros(4, table.shape[1] + 9, dtype=torch.int32, device="cuda")
    long[:, : table.shape[1]] = table
    table = long[:, : table.shape[1]]
    room = torch.full((4, 14, 130), 3.0, device="cuda", dtype=torch.bfloat16)
    out = room[:, 1:13, :128]
    first, lse = W.attend_paged(q, kc, vc, table, n, workspace=ws, with_lse=True, out=out)
    assert first is out
    check(out, lse, q, kc, vc, table, n, 128 ** -0.5)
    assert bool((room[:, 0] == 3).all()) and bool((room[:, 13] == 3).all()) and bool((room[..., 128:] == 3).all())
    want = out.clone()
    torch.cuda.synchronize()
    side, ws2 = torch.cuda.Stream(), W.attend_workspace("cuda")
    torch.cuda.synchronize()
    for _ in range(3):
        again = W.attend_paged(q, kc, vc, table, n, workspace=ws2, stream=side)
        side.synchronize()
        assert torch.equal(again, want)
    assert torch.equal(W.attend_paged(q, kc, vc, table, n), want)      # a workspace made by the call


def test_offsets_past_32_bits(W, ws):
    """A pool of more than 2^31 elements, its last pages in use."""
    hkv, d, page = 8, 128, 16
    pages = 2 ** 31 // (hkv * d * page) + 50
    pool = torch.empty(pages, page, hkv, d, device="cuda", dtype=torch.bfloat16)
    q, kc, vc, table, n = make(9, [300], 8, hkv, d, page, torch.bfloat16)
    used = table[0, :19].long()
    for c in (kc, vc):
        pool[pages - 40: pages - 21] = c[used]
        table2 = table.clone()
        table2[0, :19] = torch.arange(pages - 40, pages - 21, device="cuda")
    o, lse = W.attend_paged(q, pool, pool, table2, n, workspace=ws, with_lse=True)
    check(o, lse, q, pool, pool, table2, n, 128 ** -0.5)


def test_no_lanes(W, ws):
    q, kc, vc, table, n = make(10, [5], 4, 2, 64, 16, torch.float16)
    assert W.attend_paged(q[:0], kc, vc, table[:0], n[:0], workspace=ws).shape == (0, 4, 64)


def test_refusals(W, ws):
    q, kc, vc, table, n = make(11, [40, 50], 4, 2, 64, 16, torch.float16)
    ok = dict(q=q, k_pages=kc, v_pages=vc, page_table=table, lengths=n, workspace=ws)
    W.attend_paged(**ok)
    for error, change in [
            (TypeError, dict(q=q.float())), (TypeError, dict(k_pages=kc.bfloat16())),
            (TypeError, dict(lengths=n.long())), (TypeError, dict(page_table=table.long())),
            (ValueError, dict(q=q.cpu())), (ValueError, dict(lengths=n[:1])), (ValueError, dict(v_pages=vc[:1])),
            (ValueError, dict(page_table=table[:1])), (ValueError, dict(workspace=ws[:100])),
            (ValueError, dict(page_table=table.t().contiguous().t())),
            (ValueError, dict(q=torch.zeros(2, 64, 4, device="cuda").half().transpose(1, 2))),
            (ValueError, dict(out=torch.zeros(2, 4, 65, device="cuda").half())),
            (W.WfstError, dict(q=torch.zeros(2, 5, 64, device="cuda").half())),    # 5 heads over 2
            (W.WfstError, dict(q=q[..., :32], k_pages=kc[..., :32], v_pages=vc[..., :32])),
            (W.WfstError, dict(window=-1)), (W.WfstError, dict(sinks=-1)), (W.WfstError, dict(scale=math.nan))]:
        with pytest.raises(error):
            W.attend_paged(**{**ok, **change})
