"""Products with 4-bit weights against the same product in 64 bits.

Tolerance: y is rounded once, by at most half a unit of its type (2^-11 or
2^-8 of it, relative: u), and its fp32 sums of K terms are off by at most K *
2^-23 of the sum of the terms' sizes, with zero points counted as the two
sums that they are computed as."""
import numpy as np
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


def matrix(seed, n, k, group, zeros, dtype):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    codes = torch.randint(0, 256, (n, k // 2), generator=g, device="cuda", dtype=torch.uint8)
    scales = (torch.rand(n, k // group, generator=g, device="cuda") * 0.1 + 0.01).to(dtype)
    z = (torch.rand(n, k // group, generator=g, device="cuda") * 15).to(dtype) if zeros else None
    return codes, scales, z


def reference(x, codes, scales, z, bias):
    """(y, the size of what its sums hold) in 64 bits."""
    k, group = 2 * codes.shape[1], 2 * codes.shape[1] // scales.shape[1]
    c = torch.stack([codes & 15, codes >> 4], 2).reshape(len(codes), k).double()
    s = scales.double().repeat_interleave(group, 1)
    zz = torch.full_like(s, 8.0) if z is None else z.double().repeat_interleave(group, 1)
    x = x.double()
    y, size = x @ (s * (c - zz)).t(), x.abs() @ (s * ((c - 8).abs() + (8 - zz).abs())).t()
    if bias is not None:
        y, size = y + bias.double(), size + bias.double().abs()
    return y, size


def check(y, ref, size, k):
    bound = UNIT[y.dtype] * ref.abs() + k * 2.0 ** -23 * size + 2.0 ** -24
    assert bool(((y.double() - ref).abs() <= bound).all())


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("zeros", [False, True])
@pytest.mark.parametrize("n,k,group", [(1, 32, 32), (15, 64, 64), (17, 96, 32), (33, 416, 32), (130, 256, 128),
                                       (64, 512, 256), (1000, 1056, 32), (257, 4096, 128), (5000, 640, 64)])
def test_against_64_bits(W, n, k, group, zeros, dtype):
    codes, scales, z = matrix(n + k, n, k, group, zeros, dtype)
    w = W.pack_quant(codes, scales, z)
    g = torch.Generator(device="cuda")
    g.manual_seed(1)
    bias = torch.randn(n, generator=g, device="cuda").to(dtype)
    for rows in (1, 2, 7, 8, 9, 16, 17, 31, 33, 64, 65, 130):
        x = torch.randn(rows, k, generator=g, device="cuda").to(dtype)
        for b in (None, bias):
            y = W.matvec_quant(x, w, bias=b)
            assert y.shape == (rows, n) and y.dtype == dtype
            check(y, *reference(x, codes, scales, z, b), k)


@pytest.mark.parametrize("dtype", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("zeros", ["none", "any", "whole"])
@pytest.mark.parametrize("n,k,group", [(2449, 96, 32), (2600, 1056, 32), (2449, 640, 64), (2560, 1152, 128),
                                       (3001, 768, 256)])
def test_many_rows(W, n, k, group, zeros, dtype):
    """Enough outputs and rows that the weights are widened once for all rows;
    rows that are not finite stay in their rows."""
    codes, scales, z = matrix(n + k, n, k, group, zeros != "none", dtype)
    if zeros == "whole":
        z = z.round()
    w = W.pack_quant(codes, scales, z)
    g = torch.Generator(device="cuda")
    g.manual_seed(2)
    for rows in (17, 32, 33, 50, 64, 65, 200):
        x = torch.randn(rows, k + 8, generator=g, device="cuda").to(dtype)[:, :k]
        y = W.matvec_quant(x, w)
        check(y, *reference(x, codes, scales, z, None), k)
        assert torch.equal(W.matvec_quant(x, w), y)
        x[rows // 2, k - 1] = float("inf")
        x[0, 0] = float("nan")
        other = W.matvec_quant(x, w)
        whole = [r for r in range(rows) if r not in (0, rows // 2)]
        assert torch.equal(other[whole], y[whole])
        assert bool(other[0].isnan().all())


def test_strides_streams_and_repeats(W):
    """Rows of a wider tensor in, rows of a wider tensor out, another stream,
    and the same bits every time."""
    codes, scales, z = matrix(3, 200, 256, 64, True, torch.bfloat16)
    side = torch.cuda.Stream()
    w = W.pack_quant(codes, scales, z)
    wide = torch.randn(24, 512, device="cuda").bfloat16()
    x = wide[::2, 128:384]
    ref, size = reference(x, codes, scales, z, None)
    out = torch.full((12, 333), 7.0, device="cuda", dtype=torch.bfloat16)
    assert W.matvec_quant(x, w, out=out[:, 50:250]) is not None
    check(out[:, 50:250], ref, size, 256)
    assert bool((out[:, :50] == 7).all()) and bool((out[:, 250:] == 7).all())
    torch.cuda.synchronize()
    first = W.matvec_quant(x, w, stream=side)
    side.synchronize()
    check(first, ref, size, 256)
    for _ in range(3):
        assert torch.equal(W.matvec_quant(x, w), first)


def test_non_finite_rows_stay_in_their_rows(W):
    codes, scales, _ = matrix(4, 40, 128, 128, False, torch.float16)
    w = W.pack_quant(codes, scales)
    x = torch.randn(3, 128, device="cuda").half()
    x[1] = float("nan")
    y = W.matvec_quant(x, w)
    ref, size = reference(x[[0, 2]], codes, scales, None, None)
    check(y[[0, 2]], ref, size, 128)
    assert bool(y[1].isnan().all())


def test_no_rows(W):
    codes, scales, _ = matrix(5, 40, 128, 128, False, torch.float16)
    y = W.matvec_quant(torch.empty(0, 128, device="cuda", dtype=torch.float16), W.pack_quant(codes, scales))
    assert y.shape == (0, 40)


def test_refusals(W):
    codes, scales, _ = matrix(6, 40, 128, 64, False, torch.float16)
    w = W.pack_quant(codes, scales)
    x = torch.randn(3, 128, device="cuda").half()
    with pytest.raises(TypeError):
        W.matvec_quant(x.bfloat16(), w)
    with pytest.raises(ValueError):
        W.matvec_quant(x[:, :64], w)
    with pytest.raises(ValueError):
        W.matvec_quant(x.cpu(), w)
    with pytest.raises(ValueError):
        W.matvec_quant(torch.randn(128, 3, device="cuda").half().t(), w)
    with pytest.raises(ValueError):
        W.matvec_quant(x, w, bias=torch.zeros(41, device="cuda").half())
    with pytest.raises(ValueError):
        W.matvec_quant(x, w, out=torch.empty(3, 41, device="cuda").half())
    with pytest.raises(W.WfstError):       # a row that starts off a 16-byte boundary
        W.matvec_quant(torch.randn(3, 136, device="cuda").half()[:, 1:129], w)
    with pytest.raises(W.WfstError):       # groups of 16
        W.pack_quant(codes, torch.ones(40, 8, device="cuda").half())
    with pytest.raises(ValueError):
        W.pack_quant(codes, torch.ones(40, 3, device="cuda").half())
    with pytest.raises(TypeError):
        W.pack_quant(codes, scales.float())
    with pytest.raises(TypeError):
        W.pack_quant(codes.int(), scales)
    with pytest.raises(ValueError):
        W.pack_quant(codes.cpu(), scales)
    from wfst_beam_search_gb300 import _ops
    host = np.zeros(1 << 16, np.uint8)      # host memory at the C entry, which has to ask
    with pytest.raises(W.WfstError):
        W.wfst_matvec_quant(_ops._MATVEC(w.ptr, (host.ctypes.data + 15) & ~15, 0, x.data_ptr(), 128, 40, -1, W.WFST_F16,
                                         40, 128, 64, 0, 1), None)
    y = torch.empty(1, 40, device="cuda").half()      # and device memory
    W.wfst_matvec_quant(_ops._MATVEC(w.ptr, x.data_ptr(), 0, y.data_ptr(), 128, 40, -1, W.WFST_F16, 40, 128, 64, 0, 1),
                        None)
    torch.cuda.synchronize()
    assert torch.equal(y, W.matvec_quant(x, w)[:1])
