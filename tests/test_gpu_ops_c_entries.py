"""The C entries of the second-pass operators by their own names: the argument
blocks as the header declares them, a device that the call has to ask for, and
host memory in the place of each array."""
import numpy as np
import pytest

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def W():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import wfst_beam_search_gb300 as W
    W.load()
    return W


def run(W, entry, pack, arrays, rest):
    """Calls once with the device known and once without, then with each array in host memory."""
    host = np.zeros(1 << 16, np.uint8)
    at_host = (host.ctypes.data + 15) & ~15
    i = [n for n, v in enumerate(rest) if v == "device"][0]
    for device in (0, -1):
        entry(pack(*(0 if a is None else a.data_ptr() for a in arrays), *rest[:i], device, *rest[i + 1:]), None)
    torch.cuda.synchronize()
    for n, a in enumerate(arrays):
        if a is not None:
            ptrs = [at_host if m == n else 0 if b is None else b.data_ptr() for m, b in enumerate(arrays)]
            with pytest.raises(W.WfstError, match="device memory"):
                entry(pack(*ptrs, *rest[:i], -1, *rest[i + 1:]), None)


def test_norm_rotate(W):
    from wfst_beam_search_gb300 import _ops
    q, k, v = torch.randn(5, 4, 64, device="cuda").half(), *torch.randn(2, 5, 2, 64, device="cuda").half()
    gains = torch.rand(2, 64, device="cuda").half()
    table = torch.rand(9, 32, device="cuda")
    pos, slots = torch.arange(5, device="cuda").int(), torch.tensor([7, 3, -1, 0, 12], device="cuda").int()
    pages = torch.zeros(2, 4, 4, 2, 64, device="cuda").half()
    want = W.norm_rotate(q, k, v, pos, table, *gains, *pages, slots, eps=1e-5, interleaved=True)
    out, mine = torch.empty_like(q), torch.zeros_like(pages)
    run(W, W.wfst_norm_rotate, _ops._ROTATE, [q, k, v, *gains, pos, slots, table, out, *mine],
        [*q.stride()[:2], *k.stride()[:2], *v.stride()[:2], *out.stride()[:2], *pages[0].stride()[:3], *pages[1].stride()[:3],
         "device", W.WFST_F16, 5, 4, 2, 64, 32, 1, 9, 4, 4, 1e-5])
    assert torch.equal(out, want) and torch.equal(mine, pages)


def test_attend_paged(W):
    from wfst_beam_search_gb300 import _ops
    q = torch.randn(3, 4, 64, device="cuda").bfloat16()
    pages = torch.randn(2, 40, 16, 2, 64, device="cuda").bfloat16()
    table = torch.randperm(39, device="cuda").int().view(3, 13)
    lens, ws = torch.tensor([200, 1, 77], device="cuda").int(), W.attend_workspace()
    want, lse = W.attend_paged(q, *pages, table, lens, scale=0.2, window=60, sinks=3, workspace=ws, with_lse=True)
    out, mine = torch.empty_like(q), torch.empty_like(lse)
    run(W, W.wfst_attend_paged, _ops._ATTEND, [q, *pages, table, lens, out, mine, ws],
        [*q.stride()[:2], *out.stride()[:2], 4, 13, *pages[0].stride()[:3], *pages[1].stride()[:3],
         "device", W.WFST_BF16, 3, 4, 2, 64, 13, 40, 16, 60, 3, 0.2])
    assert torch.equal(out, want) and torch.equal(mine, lse)


def test_sample_tokens(W):
    from wfst_beam_search_gb300 import _ops
    x, u = torch.randn(6, 9000, device="cuda"), torch.rand(6, device="cuda")
    temp, top_p, min_p = torch.rand(3, 6, device="cuda") * 0.5 + 0.4
    top_k = torch.tensor([0, 5, 300, 8999, 1, 40], device="cuda").int()
    want = W.sample_tokens(x, u, temp, top_k, top_p, min_p)
    mine = [torch.empty_like(t) for t in want]
    run(W, W.wfst_sample_tokens, _ops._SAMPLE, [x, u, temp, top_p, min_p, top_k, *mine],
        [9000, "device", W.WFST_F32, 6, 9000, 0, 1.0, 1.0, 0.0])
    assert all(torch.equal(a, b) for a, b in zip(mine, want))
    run(W, W.wfst_sample_tokens, _ops._SAMPLE, [x, u, None, None, None, None, *mine],
        [9000, "device", W.WFST_F32, 6, 9000, 50, 0.7, 0.9, 0.01])
    assert all(torch.equal(a, b) for a, b in zip(mine, W.sample_tokens(x, u, 0.7, 50, 0.9, 0.01)))
