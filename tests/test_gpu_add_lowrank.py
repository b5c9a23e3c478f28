"""Low-rank adapters against the formula in 64 bits.

Tolerance: t is an fp32 sum of k products (off by at most (k / 2 + 8) 2^-23 of
their size: on the tensor cores each may be cut off at 2^-24 of the sum) and
goes on in two 16-bit parts (twice half a step: 2^-16 of it, bf16; with fp16 as
much is allowed); the second sum has rank products, twice; a factor and a sum
with y follow (16 more), and out is rounded once (u of it)."""
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


def make(seed, rows, n, k, rank, adapters, dtype, which=None):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)

    def normal(*shape, scale=1.0):
        return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)

    if which is None:
        which = torch.randint(-1, adapters + 1, (rows,), generator=g, device="cuda").int()
    return dict(y=normal(rows, n), x=normal(rows, k), shrink=normal(adapters, rank, k, scale=k ** -0.5),
                expand=normal(adapters, n, rank, scale=rank ** -0.5), adapters=which,
                scales=torch.rand(adapters, generator=g, device="cuda") * 2 + 0.2)


def check(out, y, x, shrink, expand, adapters, scales=None, **_):
    assert out.shape == y.shape and out.dtype == y.dtype
    (rows, k), rank = x.shape, shrink.shape[1]
    for a in range(-1, shrink.shape[0]):
        if a < 0:
            at = (adapters < 0) | (adapters >= shrink.shape[0])
            assert torch.equal(out[at], y[at])
            continue
        at = adapters == a
        xd, sd, ed = x[at].double(), shrink[a].double(), expand[a].double()
        s = 1.0 if scales is None else float(scales[a])
        t, size = xd @ sd.t(), xd.abs() @ sd.t().abs()
        ref = y[at].double() + s * (t @ ed.t())
        off = (size * (k / 2 + 8) * 2.0 ** -23 + t.abs() * (2.0 ** -16 + (rank + 16) * 2.0 ** -23)) @ ed.t().abs() * abs(s)
        bound = UNIT[y.dtype] * ref.abs() + off + y[at].double().abs() * 2.0 ** -23 + 2.0 ** -24
        assert bool(((out[at].double() - ref).abs() <= bound).all()), a


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rank", [8, 16, 24, 32, 40, 64, 72, 128])
@pytest.mark.parametrize("n,k", [(256, 512), (777, 1056), (1, 8), (33, 24), (4097, 2056), (1000, 40)])
def test_sizes(W, n, k, rank, dtype):
    for rows in (1, 2, 9, 33):
        a = make(n + rank, rows, n, k, rank, 3, dtype)
        check(W.add_lowrank(**a), **a)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rows", [1, 7, 8, 9, 16, 17, 31, 32, 33, 63, 64, 65, 127, 128, 200, 1000])
def test_rows_and_who_they_belong_to(W, rows, dtype):
    """All of one adapter, of none, each of its own, in runs, anyhow."""
    i = torch.arange(rows, device="cuda").int()
    for adapters, which in ((1, i * 0), (2, i * 0 - 1), (max(rows, 1), i), (5, i // 13 % 5), (70, i * 29 % 71 - 1), (3, i % 3),
                            (2, torch.where(i == rows - 1, 1, 7).int())):
        a = make(rows, rows, 200, 264, 16, adapters, dtype, which)
        check(W.add_lowrank(**a), **a)


@pytest.mark.parametrize("rows,n,k,rank,adapters", [(64, 8192, 4096, 64, 40), (2000, 1536, 1024, 16, 9), (300, 5000, 8192, 128, 2),
                                                    (1, 131071, 4096, 8, 2), (4, 64, 60000, 16, 2)])
def test_larger(W, rows, n, k, rank, adapters):
    a = make(rows, rows, n, k, rank, adapters, torch.bfloat16)
    check(W.add_lowrank(**a), **a)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rank", [16, 64])
@pytest.mark.parametrize("rows,adapters", [(13, 3), (100, 2)])
def test_rows_that_begin_anywhere(W, rows, adapters, rank, dtype):
    """y and out at every place between 16-byte boundaries, rows alike and
    each its own; the values are those of rows that begin at one, and nothing
    else is written."""
    n = 329
    a = make(rank + rows, rows, n, 264, rank, adapters, dtype)
    even, want = (torch.empty(rows, 336, device="cuda", dtype=dtype)[:, :n] for _ in range(2))
    even.copy_(a["y"])
    W.add_lowrank(**{**a, "y": even}, out=want)
    check(want, **a)
    for width in (344, 345, 347, 350):
        for shift in range(8):
            room = torch.full((rows, width), 7.0, device="cuda", dtype=dtype)
            y = room[:, shift:shift + n]
            y.copy_(a["y"])
            base = torch.full((rows, 351), 9.0, device="cuda", dtype=dtype)
            to = shift * 3 % 8
            out = base[:, to:to + n]
            W.add_lowrank(**{**a, "y": y}, out=out)
            assert torch.equal(out, want)
            assert bool((base[:, :to] == 9).all()) and bool((base[:, to + n:] == 9).all())
            W.add_lowrank(**{**a, "y": y}, out=y)
            assert torch.equal(y, want) and bool((room[:, :shift] == 7).all()) and bool((room[:, shift + n:] == 7).all())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("rows", [3, 70])
def test_strides_scales_and_places(W, rows, dtype):
    """Parts of wider tensors, rows that begin anywhere, out in place of y and
    elsewhere; nothing else is written."""
    a = make(rows, rows, 129, 264, 16, 4, dtype)
    wide = torch.zeros(rows, 304, device="cuda", dtype=dtype)
    wide[:, 8:272] = a["x"]
    a["x"] = wide[:, 8:272]
    for name, extra in (("shrink", (6, 24, 272)), ("expand", (6, 131, 24))):
        room = torch.full(extra, math.nan, device="cuda", dtype=dtype)
        part = room[1:5, 1:1 + a[name].shape[1], :a[name].shape[2]]
        part.copy_(a[name])
        a[name] = part
    want = W.add_lowrank(**a)
    check(want, **a)
    for shift, width in ((0, 129), (1, 131), (3, 136)):
        room = torch.full((rows, shift + width + 2), 7.0, device="cuda", dtype=dtype)
        y = room[:, shift:shift + 129]
        y.copy_(a["y"])
        base = torch.full_like(room, 9.0)
        out = base[:, shift + 1:shift + 130]
        assert W.add_lowrank(**{**a, "y": y}, out=out) is out
        assert torch.equal(out, want)
        assert bool((base[:, :shift + 1] == 9).all()) and bool((base[:, shift + 130:] == 9).all())
        version = y._version
        assert W.add_lowrank(**{**a, "y": y}, out=y) is y and y._version > version
        assert torch.equal(y, want) and bool((room[:, :shift] == 7).all()) and bool((room[:, shift + 129:] == 7).all())
    a["scales"] = None
    check(W.add_lowrank(**a), **a)
    a["scales"] = torch.tensor([0.0, -1.5, 1e4, 1.0], device="cuda")
    out = W.add_lowrank(**a)
    if dtype == torch.bfloat16:
        check(out, **a)
    assert torch.equal(out[a["adapters"] == 0], a["y"][a["adapters"] == 0])


@pytest.mark.parametrize("scale", [1e4, 1.0, 1e-3])
def test_sums_past_fp16(W, scale):
    """fp16: t beyond 65504 and far below its smallest number, which the factor brings back."""
    a = make(5, 20, 100, 512, 16, 3, torch.float16)
    a["x"], a["shrink"] = (a["x"].float() * scale).half().clamp(-60000, 60000), (a["shrink"].float() * scale).half()
    a["scales"] = torch.full((3,), scale ** -2, device="cuda")
    check(W.add_lowrank(**a), **a)


def test_what_is_not_finite_stays_in_its_row(W):
    a = make(6, 40, 100, 264, 16, 3, torch.bfloat16)
    clean = W.add_lowrank(**a)
    for name, bad in (("x", math.nan), ("x", math.inf), ("y", math.inf), ("y", math.nan)):
        b = {**a, name: a[name].clone()}
        b[name][17, 5] = bad
        b["adapters"] = a["adapters"].clone()
        for which in (1, -1):
            b["adapters"][17] = which
            out = W.add_lowrank(**b)
            keep = torch.arange(40, device="cuda") != 17
            assert torch.equal(out[keep], clean[keep])
            if which < 0:
                assert torch.equal(out[17].view(torch.int16), b["y"][17].view(torch.int16))
            else:
                assert not bool(out[17, 5 if name == "y" else slice(None)].isfinite().any())
    # an adapter that no row uses is not read
    b = {**a, "shrink": a["shrink"].clone(), "expand": a["expand"].clone(), "adapters": a["adapters"].clamp(0, 1)}
    b["shrink"][2], b["expand"][2] = math.nan, math.nan
    out = W.add_lowrank(**b)
    assert bool(out.isfinite().all())
    check(out, b["y"], b["x"], b["shrink"][:2], b["expand"][:2], b["adapters"], b["scales"])


def test_streams_graphs_and_repeats(W):
    a = make(8, 64, 1000, 512, 32, 6, torch.bfloat16)
    want = W.add_lowrank(**a)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    got = W.add_lowrank(**a, stream=side)
    side.synchronize()
    assert torch.equal(got, want)
    graph = torch.cuda.CUDAGraph()
    z = a["y"].clone()
    with torch.cuda.graph(graph):
        for _ in range(3):
            W.add_lowrank(**{**a, "y": z}, out=z)
    a["adapters"].copy_(a["adapters"].flip(0))
    z.copy_(a["y"])
    graph.replay()
    w = a["y"].clone()
    for _ in range(3):
        w = W.add_lowrank(**{**a, "y": w})
        torch.cuda.synchronize()
    assert torch.equal(z, w)


def test_offsets_past_32_bits(W):
    """Adapters that begin behind 2^31 elements."""
    a = make(9, 3, 64, 64, 16, 3, torch.bfloat16)
    for name in ("shrink", "expand"):
        room = torch.empty(3 * 2 ** 30, device="cuda", dtype=torch.bfloat16)
        part = room.view(3, -1)[:, :a[name][0].numel()].view(a[name].shape)
        part.copy_(a[name])
        a[name] = part
    a["adapters"] = torch.tensor([2, 1, 2], device="cuda").int()
    check(W.add_lowrank(**a), **a)


def test_refusals(W):
    a = make(10, 4, 64, 64, 16, 3, torch.float16)
    assert W.add_lowrank(**{**a, "y": a["y"][:0], "x": a["x"][:0], "adapters": a["adapters"][:0]}).shape == (0, 64)
    none = {**a, "shrink": a["shrink"][:0], "expand": a["expand"][:0], "scales": None}
    assert torch.equal(W.add_lowrank(**none), a["y"])
    x = a["x"]
    for error, change in [
            (TypeError, dict(y=a["y"].float())), (TypeError, dict(x=x.bfloat16())), (TypeError, dict(adapters=a["adapters"].long())),
            (TypeError, dict(scales=a["scales"].double())), (TypeError, dict(scales=2.0)), (TypeError, dict(shrink=None)),
            (ValueError, dict(x=x[:3])), (ValueError, dict(x=x[:, :56])), (ValueError, dict(expand=a["expand"][:2])),
            (ValueError, dict(expand=a["expand"][:, :, :8])), (ValueError, dict(adapters=a["adapters"][:3])),
            (ValueError, dict(scales=a["scales"][:2])), (ValueError, dict(x=x.cpu())), (ValueError, dict(y=a["y"].t())),
            (ValueError, dict(out=torch.zeros(4, 65, device="cuda").half())),
            (ValueError, dict(x=x.clone().requires_grad_())),
            (W.WfstError, dict(shrink=a["shrink"][:, :12], expand=a["expand"][:, :, :12])),
            (W.WfstError, dict(x=x[:, :60], shrink=a["shrink"][..., :60])),
            (W.WfstError, dict(x=torch.zeros(4, 72, device="cuda").half()[:, 4:68])),
            (W.WfstError, dict(x=torch.zeros(4, 68, device="cuda").half()[:, :64])),
            (W.WfstError, dict(shrink=torch.zeros(3, 136, 64, device="cuda").half(),
                               expand=torch.zeros(3, 64, 136, device="cuda").half()))]:
        with pytest.raises(error):
            W.add_lowrank(**{**a, **change})
