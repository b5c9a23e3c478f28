"""The C entries of the rescoring operators by their own names: the argument
blocks as the header declares them, a device that the call has to ask for, and
host memory in the place of each array."""
import pytest

from tests.test_gpu_ops_c_entries import run

pytestmark = pytest.mark.gpu

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def W():
    if not torch.cuda.is_available():
        pytest.skip("no CUDA device")
    import wfst_beam_search_gb300 as W
    W.load()
    return W


def test_attend_prefix(W):
    from wfst_beam_search_gb300 import _ops
    q = torch.randn(3, 4, 64, device="cuda").bfloat16()
    pages = torch.randn(2, 60, 16, 2, 64, device="cuda").bfloat16()
    order = torch.randperm(60, device="cuda").int()
    shared, table = order[:20].contiguous(), order[20:59].view(3, 13)
    plen, lens = torch.tensor([311], device="cuda").int(), torch.tensor([200, 0, 77], device="cuda").int()
    ws = W.attend_prefix_workspace(3, 4, 2, 64)
    want, lse = W.attend_prefix(q, *pages, shared, plen, table, lens, scale=0.2, workspace=ws, with_lse=True)
    out, mine = torch.empty_like(q), torch.empty_like(lse)
    run(W, W.wfst_attend_prefix, _ops._PREFIX, [q, *pages, shared, plen, table, lens, out, mine, ws],
        [*q.stride()[:2], *out.stride()[:2], 4, 13, *pages[0].stride()[:3], *pages[1].stride()[:3],
         "device", W.WFST_BF16, 3, 4, 2, 64, 20, 13, 60, 16, 0.2])
    assert torch.equal(out, want) and torch.equal(mine, lse)


def test_score_tokens(W):
    from wfst_beam_search_gb300 import _ops
    x, t = torch.randn(6, 9000, device="cuda").half(), torch.arange(6, device="cuda").int()
    want = W.score_tokens(x, t, top=7)
    mine = [torch.empty_like(v) for v in want]
    run(W, W.wfst_score_tokens, _ops._SCORE, [x, t, *mine], [9000, "device", W.WFST_F16, 6, 9000, 7])
    assert all(torch.equal(a, b) for a, b in zip(mine, want))
    run(W, W.wfst_score_tokens, _ops._SCORE, [x, t, *mine[:2], None, None], [9000, "device", W.WFST_F16, 6, 9000, 0])
    assert all(torch.equal(a, b) for a, b in zip(mine, want))


def test_add_lowrank(W):
    from wfst_beam_search_gb300 import _ops
    y, x = torch.randn(9, 200, device="cuda").bfloat16(), torch.randn(9, 64, device="cuda").bfloat16()
    shrink, expand = torch.randn(3, 24, 64, device="cuda").bfloat16(), torch.randn(3, 200, 24, device="cuda").bfloat16()
    which, scales = torch.tensor([0, 1, 2, -1, 3, 1, 1, 0, 2], device="cuda").int(), torch.rand(3, device="cuda")
    for s in (scales, None):
        want, out = W.add_lowrank(y, x, shrink, expand, which, s), torch.empty_like(y)
        run(W, W.wfst_add_lowrank, _ops._LOWRANK, [y, x, shrink, expand, which, s, out],
            [200, 64, 200, 24 * 64, 64, 200 * 24, 24, "device", W.WFST_BF16, 9, 200, 64, 24, 3])
        assert torch.equal(out, want)
