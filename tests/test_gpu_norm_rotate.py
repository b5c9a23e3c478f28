"""The heads' norm, rotation and cache write against the formulas in 64 bits.

Tolerance: one rounding to the type (u of the value), and in front of it fp32
arithmetic of at most d + 16 operations on values of the pair's size."""
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


def make_table(contexts, rot):
    pos = torch.arange(contexts, device="cuda", dtype=torch.float64)[:, None]
    ang = pos * 500.0 ** (-torch.arange(0, rot, 2, device="cuda", dtype=torch.float64) / max(rot, 1))
    return torch.cat([ang.cos(), ang.sin()], 1).float().contiguous()


def reference(x, gain, table, pos, inter, eps):
    """(result, the size of the pair that each element comes from)"""
    rot = table.shape[1]
    x = x.double()
    x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt()
    if gain is not None:
        x = x * gain.double()
    size = x.abs()
    if rot:
        cs = table.double()[pos.long()][:, None]
        c, s = cs[..., : rot // 2], cs[..., rot // 2:]
        i = torch.arange(rot // 2, device="cuda")
        re, im = (2 * i, 2 * i + 1) if inter else (i, i + rot // 2)
        a, b = x[..., re], x[..., im]
        x, size = x.clone(), size.clone()
        x[..., re], x[..., im] = a * c - b * s, a * s + b * c
        size[..., re] = size[..., im] = a.abs() + b.abs()
    return x, size


def check(y, ref, size, d):
    bound = UNIT[y.dtype] * ref.abs() + (d + 16) * 2.0 ** -23 * size + 2.0 ** -24
    assert bool(((y.double() - ref).abs() <= bound).all())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("inter", [False, True])
@pytest.mark.parametrize("d,rot", [(64, 64), (64, 16), (64, 48), (128, 128), (128, 96), (128, 0), (256, 256), (256, 32)])
def test_against_64_bits(W, d, rot, inter, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(d + rot)
    table = make_table(300, rot)
    for tokens, hq, hkv, page in ((1, 1, 1, 16), (3, 5, 1, 7), (129, 8, 2, 16), (700, 3, 3, 1)):
        qkv = (torch.randn(tokens, (hq + 2 * hkv) * d, generator=g, device="cuda") * 3).to(dtype)
        q, k, v = qkv.view(tokens, -1, d).split([hq, hkv, hkv], 1)
        gains = [(torch.rand(d, generator=g, device="cuda") + 0.5).to(dtype) for _ in range(2)]
        if tokens == 3:
            gains = [None, None]
        pos = torch.randint(0, 300, (tokens,), generator=g, device="cuda", dtype=torch.int32)
        pages = -(-tokens // page) + 2
        slots = torch.randperm(pages * page, generator=g, device="cuda")[:tokens].int()
        kc, vc = (torch.full((pages, page, hkv, d), 9.0, device="cuda", dtype=dtype) for _ in range(2))
        eps = 1e-5
        out = W.norm_rotate(q, k, v, pos, table, *gains, kc, vc, slots, eps=eps, interleaved=inter)
        check(out, *reference(q, gains[0], table, pos, inter, eps), d)
        at = slots.long()
        check(kc.view(-1, hkv, d)[at], *reference(k, gains[1], table, pos, inter, eps), d)
        assert torch.equal(vc.view(-1, hkv, d)[at], v)
        rest = torch.ones(pages * page, dtype=torch.bool, device="cuda")
        rest[at] = False
        assert bool((kc.view(-1, hkv, d)[rest] == 9).all()) and bool((vc.view(-1, hkv, d)[rest] == 9).all())


def test_in_place_other_layouts_and_streams(W):
    """q turned in place, a cache with the heads before the places, k and v of
    their own, all on another stream."""
    tokens, hq, hkv, d, page = 37, 6, 3, 128, 8
    dtype = torch.bfloat16
    q, k, v = (torch.randn(tokens, h, d, device="cuda").to(dtype) for h in (hq, hkv, hkv))
    table, pos = make_table(64, d), torch.arange(tokens, device="cuda", dtype=torch.int32)
    slots = torch.arange(tokens, device="cuda", dtype=torch.int32) * 2
    pool = torch.zeros(2, 10, hkv, page, d, device="cuda", dtype=dtype)
    kc, vc = pool[0].transpose(1, 2), pool[1].transpose(1, 2)
    ref = reference(q, None, table, pos, False, 1e-6)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    out = W.norm_rotate(q, k, v, pos, table, None, None, kc, vc, slots, out=q, stream=side)
    side.synchronize()
    assert out is q
    check(q, *ref, d)
    at = slots.long()
    check(kc[at // page, at % page], *reference(k, None, table, pos, False, 1e-6), d)
    assert torch.equal(vc[at // page, at % page], v)


def test_tokens_that_are_not_kept_and_positions_out_of_range(W):
    tokens, d = 6, 64
    q = torch.randn(tokens, 2, d, device="cuda").half()
    k, v = torch.randn(2, tokens, 1, d, device="cuda").half()
    table = make_table(10, 32)
    pos = torch.tensor([0, 9, 10, -1, 3, 4], dtype=torch.int32, device="cuda")
    slots = torch.tensor([-1, 0, 5, 3, 12, 2 ** 31 - 1], dtype=torch.int32, device="cuda")   # 12: past the pool
    kc, vc = torch.zeros(2, 3, 4, 1, d, device="cuda").half()
    out = W.norm_rotate(q, k, v, pos, table, None, None, kc, vc, slots)
    assert bool(out[2, :, :32].isnan().all()) and bool(out[3, :, :32].isnan().all())
    assert not bool(out[2:4, :, 32:].isnan().any()) and not bool(out[[0, 1, 4, 5]].isnan().any())
    written = (vc.view(-1, d) != 0).any(1).nonzero().flatten().tolist()
    assert written == [0, 3, 5]


def test_zero_rows_and_no_tokens(W):
    d = 128
    table, z = make_table(4, d), torch.zeros(2, 2, d, device="cuda").half()
    kc, vc = torch.ones(2, 1, 2, 2, d, device="cuda").half()
    slots = torch.tensor([1, 0], dtype=torch.int32, device="cuda")
    pos = torch.zeros(2, dtype=torch.int32, device="cuda")
    assert bool((W.norm_rotate(z, z, z, pos, table, None, None, kc, vc, slots) == 0).all())
    assert bool((kc == 0).all()) and bool((vc == 0).all())
    e = z[:0]
    assert W.norm_rotate(e, e, e, pos[:0], table, None, None, kc, vc, slots[:0]).shape == (0, 2, d)


def test_a_pool_without_pages(W):
    """Nothing can be kept; q is turned all the same."""
    q, k = torch.randn(3, 2, 64, device="cuda").half(), torch.randn(3, 1, 64, device="cuda").half()
    table, i = make_table(4, 64), torch.arange(3, device="cuda", dtype=torch.int32)
    pages = torch.zeros(2, 16, 1, 64, device="cuda").half()
    want = W.norm_rotate(q, k, k, i, table, None, None, pages, pages.clone(), i)
    assert torch.equal(W.norm_rotate(q, k, k, i, table, None, None, pages[:0], pages[:0], i), want)
    none = torch.zeros(0, 16, 1, 64, device="cuda").half()
    assert torch.equal(W.norm_rotate(q, k, k, i, table, None, None, none, none, i), want)


def test_refusals(W):
    d = 64
    q = torch.randn(3, 2, d, device="cuda").half()
    table, i = make_table(8, 32), torch.zeros(3, dtype=torch.int32, device="cuda")
    kc = torch.zeros(2, 4, 2, d, device="cuda").half()
    vc = torch.zeros_like(kc)
    ok = dict(q=q, k=q, v=q, positions=i, table=table, q_gain=None, k_gain=None, k_pages=kc, v_pages=vc,
              slots=i + torch.arange(3, device="cuda", dtype=torch.int32))
    W.norm_rotate(**ok)
    wide = torch.randn(3, 2, 72, device="cuda").half()
    for error, change in [
            (TypeError, dict(q=q.float())), (TypeError, dict(k=q.bfloat16())), (TypeError, dict(positions=i.long())),
            (TypeError, dict(table=table.half())), (ValueError, dict(q=q.cpu())), (ValueError, dict(v=q[:2])),
            (ValueError, dict(slots=i[:2])), (ValueError, dict(q_gain=torch.ones(32, device="cuda").half())),
            (ValueError, dict(k_pages=kc[:, :, :1])), (ValueError, dict(q=q.transpose(1, 2))),
            (ValueError, dict(table=make_table(8, 64)[:, :32])),
            (W.WfstError, dict(table=make_table(8, 24))),                           # not a multiple of 16
            (W.WfstError, dict(table=make_table(8, 80))),                           # more than the head
            (W.WfstError, dict(q=wide[:, :, 4:68])),                                # off a 16-byte boundary
            (W.WfstError, dict(eps=-1.0)),
            (W.WfstError, dict(q=q[..., :32], k=q[..., :32], v=q[..., :32], k_pages=kc[..., :32], v_pages=vc[..., :32]))]:
        with pytest.raises(error):
            W.norm_rotate(**{**ok, **change})
