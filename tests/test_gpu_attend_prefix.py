"""Attention behind a shared prefix against the formula in 64 bits.

Tolerance: o is rounded once (u of it); in front of that, scores are fp32 sums
of d products, off by at most (d + 8) * 2^-23 of the terms' size (for a score:
scale * sum |q k|, here called r), which changes a weight by that much,
relative, and its distance to the largest one by as much again; the weighted
values add up in fp32, 16 at a time on the tensor cores, where each of them may
be cut off at 2^-24 of the sum: n / 2 * 2^-23; and the prefix' weights are held
in two 16-bit parts, each half a step off: 2^-16 (bf16: twice 2^-8), with fp16
also 2^-35 of the largest weight (its smallest exponent)."""
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


def make(seed, prefix, lens, hq, hkv, d, page, dtype, spread=1.5):
    """Inputs whose pages lie anywhere; what no lane sees is NaN, pages and table entries alike."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    width, shared = max(1, -(-max(lens, default=1) // page)) + 1, -(-prefix // page)
    ids = [(b, i) for b, n in enumerate(lens) for i in range(-(-n // page))]
    count = shared + len(ids) + 2
    order = torch.randperm(count, generator=g, device="cuda").int()
    ptable = torch.full((shared + 2,), -3, dtype=torch.int32, device="cuda")
    ptable[:shared] = order[:shared]
    table = torch.full((len(lens), width), -7, dtype=torch.int32)
    for (b, i), o in zip(ids, order[shared:].tolist()):
        table[b, i] = o
    table = table.cuda()
    kc, vc = (torch.full((count, page, hkv, d), math.nan, device="cuda", dtype=dtype) for _ in range(2))
    for row, n in [(ptable, prefix), *((table[b], n) for b, n in enumerate(lens))]:
        j = torch.arange(n, device="cuda")
        at = (row[j // page].long(), j % page)
        kc[at] = torch.randn(n, hkv, d, generator=g, device="cuda").to(dtype)
        vc[at] = torch.randn(n, hkv, d, generator=g, device="cuda").to(dtype)
    q = (torch.randn(len(lens), hq, d, generator=g, device="cuda") * spread).to(dtype)
    i32 = dict(dtype=torch.int32, device="cuda")
    return q, kc, vc, ptable, torch.tensor([prefix], **i32), table, torch.tensor(lens, **i32)


def check(o, lse, q, kc, vc, ptable, plen, table, lens, scale, seen=None):
    """``seen``: per lane (tokens of the prefix, tokens of its own)."""
    page, hkv, d = kc.shape[1:]
    share, p16 = q.shape[1] // hkv, 2.0 ** -16 if q.dtype == torch.bfloat16 else 2.0 ** -22
    for b, n in enumerate(lens.tolist()):
        first, mine = seen[b] if seen else (range(int(plen)), range(n))
        ks, vs = [], []
        for row, j in ((ptable, first), (table[b], mine)):
            j = torch.tensor(list(j), dtype=torch.long, device="cuda")
            at = (row[j // page].long(), j % page)
            ks.append(kc[at].double()), vs.append(vc[at].double())
        k, v = torch.cat(ks), torch.cat(vs)
        if not len(k):
            assert bool((o[b] == 0).all()) and bool((lse[b] == -math.inf).all())
            continue
        x = torch.einsum("gsd,jgd->gsj", q[b].double().view(hkv, share, d), k) * scale
        r = (torch.einsum("gsd,jgd->gsj", q[b].double().abs().view(hkv, share, d), k.abs()) * abs(scale)).amax(2)
        p = torch.softmax(x, 2)
        ref, size = torch.einsum("gsj,jgd->gsd", p, v), torch.einsum("gsj,jgd->gsd", p, v.abs())
        fp = (2 * r * (d + 8) + len(k) / 2 + 64)[:, :, None] * 2.0 ** -23
        low = 2.0 ** -35 * v.abs().sum(0)[:, None, :] if q.dtype == torch.float16 else 0.0
        bound = UNIT[o.dtype] * ref.abs() + (fp + p16) * size + low + 2.0 ** -24
        assert bool(((o[b].double().view(hkv, share, d) - ref).abs() <= bound).all()), (b, n)
        assert bool(((lse[b].double().view(hkv, share) - torch.logsumexp(x, 2)).abs() <= fp[..., 0]).all()), (b, n)


def attend(W, a, **more):
    q, kc = a[0], a[1]
    ws = W.attend_prefix_workspace(q.shape[0], q.shape[1], kc.shape[2], q.shape[2])
    return W.attend_prefix(*a, workspace=ws, with_lse=True, **more)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("hq,hkv", [(1, 1), (4, 4), (6, 2), (8, 1), (18, 2), (16, 1), (66, 2)])
def test_head_layouts(W, hq, hkv, d, dtype):
    a = make(hq * d, 333, [1, 0, 17, 64, 65, 200], hq, hkv, d, 16, dtype)
    check(*attend(W, a), *a, d ** -0.5)


@pytest.mark.parametrize("page", [1, 7, 16, 48, 64, 100])
@pytest.mark.parametrize("d,dtype", [(64, torch.bfloat16), (128, torch.float16), (256, torch.bfloat16)])
def test_lengths_and_pages(W, page, d, dtype):
    for prefix in (0, 1, 2, 15, 16, 63, 64, 65, 100, 127, 128, 129, 191, 193, 255, 256, 257, 383, 385, 1000, 3001):
        a = make(page + prefix, prefix, [0, 1, 5, 130], 4, 2, d, page, dtype)
        check(*attend(W, a), *a, d ** -0.5)


@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("lanes,hq,hkv", [(32, 4, 1), (33, 8, 2), (64, 4, 1), (65, 4, 1), (40, 24, 3), (130, 5, 1), (3, 129, 1),
                                          (2, 257, 1), (300, 12, 4)])
def test_many_rows(W, lanes, hq, hkv, d):
    """Rows of a key-value head that end inside a tile of rows, at its end and behind it."""
    for prefix, dtype in ((700, torch.bfloat16), (130, torch.float16)):
        a = make(lanes + hq, prefix, [n % 23 for n in range(lanes)], hq, hkv, d, 32, dtype)
        check(*attend(W, a), *a, d ** -0.5)


@pytest.mark.parametrize("prefix,lens,hq,hkv,d", [(40000, [3], 4, 1, 128), (20011, [0, 700], 8, 2, 64), (9000, [1] * 5, 64, 64, 64),
                                                  (513, [2] * 3, 200, 200, 64), (150, [9], 170, 170, 128),
                                                  (2000, [400] * 70, 8, 2, 256), (1, [0] * 9, 8, 8, 128),
                                                  (300, [1] * 140, 160, 20, 64)])
def test_splits(W, prefix, lens, hq, hkv, d):
    """One head's prefix over all CTAs; several heads' prefixes in one CTA; parts of two of them."""
    a = make(len(lens), prefix, lens, hq, hkv, d, 32, torch.bfloat16)
    check(*attend(W, a), *a, d ** -0.5)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("d", [64, 128, 256])
@pytest.mark.parametrize("share", [1, 50])
def test_long_runs(W, share, d, dtype):
    """Many tiles of keys for each CTA, with one tile of rows and with two."""
    for prefix in (20011, 7100):
        a = make(prefix + share, prefix, [70, 0, 5], 8 * share, 8, d, 48, dtype)
        check(*attend(W, a), *a, d ** -0.5)


def test_a_workspace_whose_parts_hold_anything(W):
    a = make(3, 3000, [2000, 1, 0, 700], 24, 2, 128, 32, torch.bfloat16)
    ws = W.attend_prefix_workspace(4, 24, 2, 128)
    assert ws.numel() == W.wfst_prefix_size(4, 24, 2, 128)
    ws[W.WFST_ATTEND_ZEROED:] = 255                      # NaN
    for _ in range(2):
        check(*W.attend_prefix(*a, workspace=ws, with_lse=True), *a, 128 ** -0.5)
        assert not bool(ws[:W.WFST_ATTEND_ZEROED].any())


def test_a_workspace_of_more_lanes(W):
    ws = W.attend_prefix_workspace(300, 8, 2, 128)
    for lanes, prefix in ((300, 100), (1, 5000), (64, 700), (65, 700), (7, 0)):
        a = make(lanes, prefix, [n % 40 for n in range(lanes)], 8, 2, 128, 16, torch.bfloat16)
        check(*W.attend_prefix(*a, workspace=ws, with_lse=True), *a, 128 ** -0.5)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
def test_large_scores_and_other_scales(W, dtype):
    """Weights that are nearly all on one key, and a negative scale."""
    a = make(5, 900, [700, 64, 33, 0], 8, 4, 64, 16, dtype, spread=30.0)
    for scale in (0.125, -0.02, 0.0):
        check(*attend(W, a, scale=scale), *a, scale)


@pytest.mark.parametrize("d,hq,hkv", [(64, 2, 2), (128, 12, 1), (256, 8, 1)])
@pytest.mark.parametrize("gap", [3.0, 8.0, 12.0, 14.0, 16.0, 17.4, 20.0])
def test_weights_far_below_the_largest_fp16(W, gap, d, hq, hkv):
    """One key of the prefix `gap` above thousands of others, whose value is
    zero: what o holds comes from the others alone.  (Largest first, last and
    between, so that the sums are rescaled or not.)"""
    n = 20011
    for peak in (0, 7000, n - 1):
        q, kc, vc, ptable, plen, table, lens = make(int(gap * 10) + d, n, [0, 3], hq, hkv, d, 64, torch.float16)
        g = torch.Generator(device="cuda")
        g.manual_seed(peak)
        kc.zero_(), q.zero_()
        vc.copy_(((torch.rand(vc.shape, generator=g, device="cuda") + 0.5) * 4096).half())
        q[..., 3] = 1.0
        kc[..., 3] = (torch.rand(kc.shape[:3], generator=g, device="cuda") * 0.5).half()
        at = int(ptable[peak // 64])
        kc[at, peak % 64, :, 3] = gap
        vc[at, peak % 64] = 0
        a = q, kc, vc, ptable, plen, table, lens
        check(*attend(W, a, scale=1.0), *a, 1.0)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("power", range(8, 31, 2))
@pytest.mark.parametrize("best_in_prefix", [True, False])
def test_huge_scores(W, power, dtype, best_in_prefix):
    """Scores of up to 2^30 whose differences leave one key all the weight: o
    is its value to the bit, lse its score to the roundings of a product."""
    n, d, page, mine = 1500, 64, 16, 300
    g = torch.Generator(device="cuda")
    g.manual_seed(power)
    q, kc, vc, ptable, plen, table, lens = make(power, n, [mine], 3, 1, d, page, dtype)
    kc.zero_(), q.zero_()
    size = 2.0 ** (power // 2)                     # of q's one element and of the keys'
    q[0, 0, 7], q[0, 1, 7], q[0, 2, 7] = size, -size, size * 0.75
    total = n + mine
    score = torch.linspace(-0.5, 0.5, total, device="cuda", dtype=torch.float64)[torch.randperm(total, generator=g, device="cuda")] * size
    best, worst = (777, n + 40) if best_in_prefix else (n + 7, 40)
    score[best], score[worst] = size, -size
    j = torch.arange(n, device="cuda")
    one = torch.arange(mine, device="cuda")
    page_of = torch.cat([ptable[j // page].long(), table[0][one // page].long()])
    place = torch.cat([j % page, one % page])
    kc[page_of, place, 0, 7] = score.to(dtype)
    o, lse = attend(W, (q, kc, vc, ptable, plen, table, lens), scale=1.0)
    v = vc[page_of, place][:, 0]
    assert torch.equal(o[0], torch.stack([v[best], v[worst], v[best]]))
    want = torch.tensor([1.0, 1.0, 0.75], device="cuda", dtype=torch.float64) * 4.0 ** (power // 2)
    assert bool(((lse[0].double() - want).abs() <= 8 * 2.0 ** -24 * want).all())


def test_missing_pages_and_long_lengths(W):
    """Tokens of pages outside the pool are not seen; a length past the table ends with it."""
    q, kc, vc, ptable, plen, table, n = make(6, 400, [100, 100, 64], 2, 1, 64, 16, torch.bfloat16)
    ptable, table = ptable[:25].contiguous(), table[:, :6].contiguous()            # 400 and 96 tokens
    ptable[3], ptable[8:16], ptable[24] = -1, kc.shape[0], 2 ** 31 - 1
    table[0, 2], table[1, 0], table[1, 5], table[2] = -1, kc.shape[0], 2 ** 31 - 1, -2 ** 31
    first = [j for j in range(384) if j // 16 not in (3, *range(8, 16))]
    seen = [(first, [j for j in range(96) if j // 16 != 2]), (first, range(16, 80)), (first, ())]
    big = torch.tensor([100, 2 ** 31 - 1, 64], dtype=torch.int32, device="cuda")
    plen[:] = 2 ** 31 - 1
    a = q, kc, vc, ptable, plen, table, big
    check(*attend(W, a), q, kc, vc, ptable, plen, table, n, 0.125, seen=seen)
    n[:] = -5
    check(*attend(W, (*a[:6], n)), q, kc, vc, ptable, plen, table, n, 0.125, seen=[(first, ())] * 3)
    for change in (-9, 0):
        plen[:] = change
        o, lse = attend(W, (*a[:6], n))
        assert bool((o == 0).all()) and bool((lse == -math.inf).all())
    plen[:], ptable[:] = 400, -1
    o, lse = attend(W, (*a[:6], n))
    assert bool((o == 0).all()) and bool((lse == -math.inf).all())


def test_infinities_and_nan_in_seen_places(W):
    """What is seen counts as the formula says: a lane's own NaN stays in it, a
    query's in its head, a value's of the prefix in its element; a key of weight
    zero (-inf score) weighs nothing."""
    a = q, kc, vc, ptable, plen, table, n = make(7, 300, [50, 50, 0], 4, 2, 64, 16, torch.float16)
    clean, lse0 = attend(W, a)
    q2, vc2 = q.clone(), vc.clone()
    vc2[table[1, 1].long(), 3, 1, 5] = math.nan
    o, _ = attend(W, (q, kc, vc2, *a[3:]))
    assert torch.equal(o[::2], clean[::2]) and torch.equal(o[1, :2], clean[1, :2])
    assert bool(o[1, 2:, 5].isnan().all()) and int(o[1, 2:].isnan().sum()) == 2
    q2[1, 3, 7] = math.nan
    o, lse = attend(W, (q2, *a[1:]))
    assert bool(o[1, 3].isnan().all()) and bool(lse[1, 3].isnan()) and int(o.isnan().sum()) == 64
    o[1, 3] = clean[1, 3]
    assert torch.equal(o, clean)
    vc2 = vc.clone()
    vc2[ptable[2].long(), 3, 0, 9] = math.inf
    o, lse = attend(W, (q, kc, vc2, *a[3:]))
    assert not bool(o[:, :2, 9].isfinite().any()) and torch.equal(lse, lse0)
    o[:, :2, 9] = clean[:, :2, 9]
    assert torch.equal(o, clean)
    q2 = torch.ones_like(q)
    kc2 = kc.clone()
    kc2[ptable[0].long(), 2], kc2[ptable[18].long(), 1] = -65504.0, -65504.0
    kc2[ptable[0].long(), 2, :, 0] = kc2[ptable[18].long(), 1, :, 0] = -math.inf
    seen = [([j for j in range(300) if j not in (2, 18 * 16 + 1)], range(m)) for m in (50, 50, 0)]
    check(*attend(W, (q2, kc2, *a[2:])), q2, kc2, *a[2:], 0.125, seen=seen)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("prefix,lens,hq,hkv,d", [(30000, [3, 100], 16, 2, 64), (900, [9000, 1, 0], 40, 2, 128),
                                                  (400, [30] * 131, 6, 2, 256), (70, [64, 5000], 4, 4, 64)])
def test_into_the_queries_themselves(W, prefix, lens, hq, hkv, d, dtype):
    """A head's query is read before its result is written."""
    a = make(len(lens), prefix, lens, hq, hkv, d, 32, dtype)
    for _ in range(5):
        x = a[0].clone()
        want = attend(W, (x, *a[1:]))
        got = attend(W, (x, *a[1:]), out=x)
        assert got[0] is x and torch.equal(x, want[0]) and torch.equal(got[1], want[1])


def test_layouts_streams_and_repeats(W):
    """Heads before places, q and o as parts of wider tensors, tables with
    longer rows, another stream with a workspace of its own; the same bits
    every time."""
    q, kc, vc, ptable, plen, table, n = make(8, 3000, [5000, 300, 1, 77], 12, 4, 128, 16, torch.bfloat16)
    kc, vc = (c.transpose(1, 2).contiguous().transpose(1, 2) for c in (kc, vc))
    wide = torch.zeros(4, 20, 128, device="cuda", dtype=torch.bfloat16)
    wide[:, 4:16] = q
    q = wide[:, 4:16]
    long = torch.zeros(4, table.shape[1] + 9, dtype=torch.int32, device="cuda")
    long[:, : table.shape[1]] = table
    table = long[:, : table.shape[1]]
    room = torch.full((4, 14, 130), 3.0, device="cuda", dtype=torch.bfloat16)
    out = room[:, 1:13, :128]
    a = q, kc, vc, ptable, plen, table, n
    first, lse = attend(W, a, out=out)
    assert first is out
    check(out, lse, *a, 128 ** -0.5)
    assert bool((room[:, 0] == 3).all()) and bool((room[:, 13] == 3).all()) and bool((room[..., 128:] == 3).all())
    want = out.clone()
    side, ws = torch.cuda.Stream(), W.attend_prefix_workspace(4, 12, 4, 128)
    torch.cuda.synchronize()
    for _ in range(3):
        again = W.attend_prefix(*a, workspace=ws, stream=side)
        side.synchronize()
        assert torch.equal(again, want)
    assert torch.equal(W.attend_prefix(*a), want)      # a workspace made by the call


def test_in_a_graph_whose_lengths_change(W):
    a = make(13, 2000, [300, 40, 0, 7] * 9, 16, 2, 128, 16, torch.bfloat16)
    ws, ws2 = (W.attend_prefix_workspace(36, 16, 2, 128) for _ in range(2))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    W.attend_prefix(*a, workspace=ws, stream=side)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        outs = [W.attend_prefix(*a, workspace=ws, with_lse=True) for _ in range(3)]
    lens = a[6].clone()
    for prefix, most in ((2000, 300), (1, 300), (0, 30), (777, 0), (1999, 1)):
        a[4].fill_(prefix)
        a[6].copy_(lens.clamp_max(most))
        graph.replay()
        want = W.attend_prefix(*a, workspace=ws2, with_lse=True)
        for got in outs:
            assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])


def test_calls_follow_each_other(W):
    """Each call's queries are the one's before it, in place; waits between the calls change nothing."""
    a = make(14, 1500, [100, 1, 0, 40] * 20, 8, 2, 128, 16, torch.bfloat16)
    ws = W.attend_prefix_workspace(80, 8, 2, 128)

    def chain(wait):
        x = a[0].clone()
        torch.cuda.synchronize()
        for _ in range(40):
            W.attend_prefix(x, *a[1:], scale=0.3, workspace=ws, out=x)
            x.add_(a[0])
            wait()
        return x

    want = chain(torch.cuda.synchronize)
    for _ in range(3):
        assert torch.equal(chain(lambda: None), want)


def test_offsets_past_32_bits(W):
    """A pool of more than 2^31 elements, its last pages in use."""
    hkv, d, page = 8, 128, 16
    pages = 2 ** 31 // (hkv * d * page) + 80
    pool = torch.empty(pages, page, hkv, d, device="cuda", dtype=torch.bfloat16)
    q, kc, vc, ptable, plen, table, n = make(9, 500, [70], 8, hkv, d, page, torch.bfloat16)
    pool[pages - len(kc):] = kc
    move = pages - len(kc)
    a = (q, pool, pool, torch.where(ptable >= 0, ptable + move, ptable), plen, torch.where(table >= 0, table + move, table), n)
    check(*attend(W, a), *a, 128 ** -0.5)


def test_no_lanes_and_no_pages(W):
    q, kc, vc, ptable, plen, table, n = make(10, 40, [5], 4, 2, 64, 16, torch.float16)
    ws = W.attend_prefix_workspace(1, 4, 2, 64)
    assert W.attend_prefix(q[:0], kc, vc, ptable, plen, table[:0], n[:0], workspace=ws).shape == (0, 4, 64)
    o = W.attend_prefix(q, kc[:0], vc[:0], ptable[:0], plen, table[:, :0], n, workspace=ws)
    assert bool((o == 0).all())
    # no table of its own: the prefix alone
    n.zero_()
    a = q, kc, vc, ptable, plen, table[:, :0], n
    check(*attend(W, a), *a, 0.125)


def test_refusals(W):
    q, kc, vc, ptable, plen, table, n = make(11, 40, [40, 50], 4, 2, 64, 16, torch.float16)
    ws = W.attend_prefix_workspace(2, 4, 2, 64)
    ok = dict(q=q, k_pages=kc, v_pages=vc, prefix_table=ptable, prefix_length=plen, page_table=table, lengths=n, workspace=ws)
    W.attend_prefix(**ok)
    for error, change in [
            (TypeError, dict(q=q.float())), (TypeError, dict(k_pages=kc.bfloat16())),
            (TypeError, dict(lengths=n.long())), (TypeError, dict(page_table=table.long())),
            (TypeError, dict(prefix_table=ptable.long())), (TypeError, dict(prefix_length=plen.long())),
            (TypeError, dict(prefix_length=40)), (ValueError, dict(prefix_length=n)), (ValueError, dict(prefix_table=table)),
            (ValueError, dict(prefix_table=ptable.repeat(2)[::2])),
            (ValueError, dict(q=q.cpu())), (ValueError, dict(lengths=n[:1])), (ValueError, dict(v_pages=vc[:1])),
            (ValueError, dict(page_table=table[:1])), (ValueError, dict(workspace=ws[:100])),
            (ValueError, dict(page_table=table.t().contiguous().t())),
            (ValueError, dict(q=torch.zeros(2, 64, 4, device="cuda").half().transpose(1, 2))),
            (ValueError, dict(out=torch.zeros(2, 4, 65, device="cuda").half())),
            (W.WfstError, dict(q=torch.zeros(2, 5, 64, device="cuda").half())),    # 5 heads over 2
            (W.WfstError, dict(q=q[..., :32], k_pages=kc[..., :32], v_pages=vc[..., :32])),
            (W.WfstError, dict(scale=math.nan))]:
        with pytest.raises(error):
            W.attend_prefix(**{**ok, **change})
    asks = q.clone().requires_grad_()
    with pytest.raises(ValueError, match="gradient"):
        W.attend_prefix(**{**ok, "q": asks})
    with torch.no_grad():
        W.attend_prefix(**{**ok, "q": asks})


def test_two_streams_at_once(W):
    """Calls on two streams with workspaces of their own, beside each other and
    beside products that use tensor memory too."""
    a = make(15, 3000, [100, 1, 0, 40] * 10, 8, 2, 64, 16, torch.bfloat16)
    b = make(16, 900, [30] * 64, 16, 4, 128, 48, torch.bfloat16)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    w = W.pack_quant(torch.randint(0, 256, (4096, 512), generator=g, device="cuda", dtype=torch.uint8),
                     torch.full((4096, 8), 0.01, device="cuda").bfloat16())
    x = torch.randn(64, 1024, generator=g, device="cuda").bfloat16()
    want = [attend(W, a)[0], attend(W, b)[0], W.matvec_quant(x, w)]
    ws = [W.attend_prefix_workspace(40, 8, 2, 64), W.attend_prefix_workspace(64, 16, 4, 128)]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    got = [[], [], []]
    for _ in range(20):
        for i, call in enumerate((lambda: W.attend_prefix(*a, workspace=ws[0]), lambda: W.attend_prefix(*b, workspace=ws[1]),
                                  lambda: W.matvec_quant(x, w))):
            with torch.cuda.stream(streams[i]):
                got[i].append(call())
    torch.cuda.synchronize()
    for mine, one in zip(got, want):
        assert all(torch.equal(m, one) for m in mine)


def test_a_pool_without_pages(W):
    """Tables that point into a pool that has none: nothing is seen."""
    q, kc, vc, ptable, plen, table, n = make(17, 300, [40, 5], 4, 2, 64, 16, torch.float16)
    o, lse = attend(W, (q, kc[:0], vc[:0], ptable, plen, table, n))
    assert bool((o == 0).all()) and bool((lse == -math.inf).all())
