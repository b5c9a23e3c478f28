"""What the second-pass operators refuse without a GPU: sizes and NULL
pointers at the C entries, host tensors and wrong types in the binding."""
import ctypes as C

import pytest

import wfst_beam_search_gb300 as W
from wfst_beam_search_gb300 import _build

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return W.load()


def test_sizes_of_a_packed_matrix(lib):
    # 128 outputs by 64 k are 4096 bytes of codes; a group's scales of a tile 256 bytes, with zero points 512
    assert W.wfst_quant_size(128, 64, 64, 0) == 4096 + 256
    assert W.wfst_quant_size(129, 64, 64, 1) == 2 * (4096 + 512)
    assert W.wfst_quant_size(1, 32, 32, 0) == 4096 + 2 * 256         # half a block is stored as a whole one
    assert W.wfst_quant_size(100000, 65536, 128, 0) == 782 * (1024 * 4096 + 512 * 256)   # past 2^31 bytes
    for n, k, group in ((0, 64, 64), (16, 0, 64), (16, 64, 16), (16, 96, 64), (16, 64, 0), (-1, 64, 64)):
        with pytest.raises(W.WfstError) as e:
            W.wfst_quant_size(n, k, group, 0)
        assert e.value.code == -1
    assert lib.wfst_quant_size(16, 64, 64, 0, None) == -1
    assert lib.wfst_quant_pack(None, None, None, W.WFST_F16, 16, 64, 64, None, None) == -1
    assert b"NULL" in lib.wfst_last_error()


def test_null_blocks(lib):
    for f in (lib.wfst_matvec_quant, lib.wfst_norm_rotate, lib.wfst_attend_paged, lib.wfst_sample_tokens):
        assert f(None, None) == -1 and b"NULL" in lib.wfst_last_error()
    assert lib.wfst_attend_size(None) == -1
    assert W.wfst_attend_size() > 0 and W.wfst_attend_size() % 16 == 0


def test_fields_are_checked_in_the_blocks(lib):
    from wfst_beam_search_gb300 import _ops

    def matvec(**kw):
        f = dict(sx=64, sy=16, device=-1, dtype=1, n=16, k=64, group=64, zeros=0, rows=1)
        f.update(kw)
        return lib.wfst_matvec_quant(_ops._MATVEC(*([0] * 4), *f.values()), None), lib.wfst_last_error()

    def rotate(**kw):
        f = dict(device=-1, dtype=1, tokens=1, hq=1, hkv=1, d=64, rot=64, inter=0, contexts=1, pages=1, page=16, eps=1e-6)
        f.update(kw)
        return lib.wfst_norm_rotate(_ops._ROTATE(*([0] * 25), *f.values()), None), lib.wfst_last_error()

    def attend(**kw):
        f = dict(device=-1, dtype=1, lanes=1, hq=2, hkv=1, d=64, width=1, pages=1, page=16, window=0, sinks=0, scale=1.0)
        f.update(kw)
        return lib.wfst_attend_paged(_ops._ATTEND(*([0] * 20), *f.values()), None), lib.wfst_last_error()

    def sample(**kw):
        f = dict(stride=10, device=-1, dtype=0, lanes=1, vocab=10, top_k=0, temp=1.0, top_p=1.0, min_p=0.0)
        f.update(kw)
        return lib.wfst_sample_tokens(_ops._SAMPLE(*([0] * 9), *f.values()), None), lib.wfst_last_error()

    assert matvec(rows=0)[0] == 0 and rotate(tokens=0)[0] == 0 and attend(lanes=0)[0] == 0 and sample(lanes=0)[0] == 0
    for call, word, change in [
            (matvec, b"NULL", {}), (matvec, b"dtype", dict(dtype=0)), (matvec, b"rows", dict(rows=-1)),
            (matvec, b"group", dict(group=16)), (matvec, b"multiple", dict(k=96)),
            (rotate, b"NULL", {}), (rotate, b"dtype", dict(dtype=0)), (rotate, b"head_dim", dict(d=80)),
            (rotate, b"rot", dict(rot=8)), (rotate, b"rot", dict(rot=128)), (rotate, b"eps", dict(eps=float("nan"))),
            (rotate, b"counts", dict(tokens=-1)),
            (attend, b"NULL", {}), (attend, b"dtype", dict(dtype=0)), (attend, b"head_dim", dict(d=32)),
            (attend, b"multiple", dict(hq=3, hkv=2)), (attend, b"page_size", dict(page=0)),
            (attend, b"2^31", dict(page=1 << 20, width=1 << 12)), (attend, b"window", dict(window=-1)),
            (attend, b"scale", dict(scale=float("nan"))),
            (sample, b"NULL", {}), (sample, b"dtype", dict(dtype=3)), (sample, b"vocab", dict(vocab=0)),
            (sample, b"vocab", dict(vocab=(1 << 20) + 1)), (sample, b"stride", dict(lanes=2, stride=9)),
            (sample, b"temperature", dict(temp=-1.0)), (sample, b"top_k", dict(top_k=-1)),
            (sample, b"top_p", dict(top_p=0.0)), (sample, b"min_p", dict(min_p=2.0))]:
        rc, said = call(**change)
        assert rc == -1 and word in said, (call.__name__, change, said)


def test_host_tensors_are_refused():
    h = torch.zeros(2, 64, dtype=torch.float16)
    i = torch.zeros(2, dtype=torch.int32)
    pages = torch.zeros(1, 16, 1, 64, dtype=torch.float16)
    with pytest.raises(ValueError):
        W.pack_quant(torch.zeros(4, 32, dtype=torch.uint8), torch.ones(4, 1).half())
    with pytest.raises(ValueError):
        W.sample_tokens(torch.zeros(2, 10), torch.zeros(2))
    with pytest.raises(ValueError):
        W.attend_paged(h[:, None], pages, pages, i[:, None], i)
    with pytest.raises(ValueError):
        W.norm_rotate(h[:, None], h[:, None], h[:, None], i, torch.zeros(4, 64), None, None, pages, pages, i)


def test_a_start_token_outside_the_vocabulary_is_refused():
    from wfst_beam_search_gb300 import second_pass as P
    for start in (-1, 50, 51):
        s = P.Shape(vocab=50, width=64, layers=1, start=start)
        with pytest.raises(ValueError, match="start token"):
            P.LanguageModel(s, P.random_tensors(s), device="cpu")


def test_a_pass_runs_on_its_models_device(monkeypatch):
    """With another device current, capture and replay are of the model's.
    torch.cuda is a stand-in that keeps count of what is current, so that no
    second GPU is needed."""
    import contextlib
    from types import SimpleNamespace

    from wfst_beam_search_gb300 import second_pass as P

    now = SimpleNamespace(device=0, stream=None, seen=[])

    class Stream:
        def __init__(self, device=None):
            self.device = now.device if device is None else torch.device(device).index

        def wait_stream(self, other):
            assert other.device == self.device

    class Graph:
        def replay(self):
            now.seen.append(("replay", now.device))

    @contextlib.contextmanager
    def use(**change):
        before = dict(vars(now))
        vars(now).update(change)
        yield
        vars(now).update({name: before[name] for name in ("device", "stream")})

    def graph(made, stream=None):
        stream = Stream() if stream is None else stream
        return use(device=stream.device, stream=stream)

    for name, fake in dict(Stream=Stream, CUDAGraph=Graph, graph=graph, device=lambda d: use(device=torch.device(d).index),
                           stream=lambda s: use(device=s.device, stream=s),
                           current_stream=lambda d=None: Stream(d)).items():
        monkeypatch.setattr(torch.cuda, name, fake)

    class Pass(P.SecondPass):
        def __init__(self):
            self.model = SimpleNamespace(device=torch.device("cuda", 1), shape=P.Shape(vocab=9))
            self.lanes, self.max_tokens, self.page, self.pages, self.graph = 2, 8, 4, 4, None
            self.table, self.plan = torch.zeros(2, 2, dtype=torch.int32), torch.zeros(8, 4, 2, dtype=torch.int32)
            self.uniform, self.logprobs, self.at = torch.zeros(8, 2), torch.zeros(8, 2), torch.zeros(1, dtype=torch.int64)
            self.settings = {n: torch.zeros(2) for n in ("temperature", "top_k", "top_p", "min_p")}
            self.drawn = torch.zeros(8, 2, dtype=torch.int32)

        def _step(self):
            now.seen.append(("step", now.device, now.stream and now.stream.device))

    second = Pass()
    assert len(second.run([[1, 2]], 2)) == 1
    assert now.seen == [("step", 1, 1), ("step", 1, 1)] + [("replay", 1)] * 4 and now.device == 0
    now.seen.clear()
    second.run([[1]], 1, graph=False)
    assert now.seen == [("step", 1, None)] * 2


def test_settings_of_a_pass_are_checked():
    from types import SimpleNamespace

    from wfst_beam_search_gb300 import second_pass as P
    second = P.SecondPass.__new__(P.SecondPass)
    second.model, second.lanes, second.max_tokens, second.page, second.pages = SimpleNamespace(shape=P.Shape(9)), 2, 8, 4, 4
    second.table = torch.zeros(2, 2, dtype=torch.int32)
    assert second.run([], 1, temperature=0, top_k=3, top_p=1.5, min_p=1.0) == []
    nan = float("nan")
    for name, values in dict(temperature=(-1.0, nan, float("inf")), top_k=(-1, 2 ** 31), top_p=(0.0, -0.5, nan),
                             min_p=(-0.1, 1.1, nan)).items():
        for value in values:
            with pytest.raises(ValueError, match=name):
                second.run([], 1, **{name: value})


def test_inputs_that_require_a_gradient_are_refused():
    h = torch.zeros(2, 64, dtype=torch.float16, requires_grad=True)
    i = torch.zeros(2, dtype=torch.int32)
    pages = torch.zeros(1, 16, 1, 64, dtype=torch.float16)
    with pytest.raises(ValueError, match="gradient"):
        W.sample_tokens(h, torch.zeros(2))
    with pytest.raises(ValueError, match="gradient"):
        W.attend_paged(h[:, None], pages, pages, i[:, None], i)
    with pytest.raises(ValueError, match="gradient"):
        W.norm_rotate(h[:, None], h[:, None], h[:, None], i, torch.zeros(4, 64), None, None, pages, pages, i)
    with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
        W.sample_tokens(h, torch.zeros(2))


def test_a_workspace_is_zeroed_where_it_has_to_be(monkeypatch):
    import os
    import re
    header = open(os.path.join(_build.INCLUDE, "wfst_gb300.h")).read()
    assert int(re.search(r"#define WFST_ATTEND_ZEROED (\d+)", header).group(1)) == W.WFST_ATTEND_ZEROED
    full = torch.full

    def garbage(size, dtype, device):
        return full((size,), 255, dtype=dtype, device=device)

    monkeypatch.setattr(torch, "empty", garbage)
    ws = W.attend_workspace("cpu")
    assert ws.shape == (W.wfst_attend_size(),)
    assert not bool(ws[:W.WFST_ATTEND_ZEROED].any()) and bool((ws[W.WFST_ATTEND_ZEROED:] == 255).all())


def test_what_is_no_tensor_is_a_type_error():
    h = torch.zeros(2, 1, 64, dtype=torch.float16)
    i = torch.zeros(2, dtype=torch.int32)
    pages, table = torch.zeros(1, 16, 1, 64, dtype=torch.float16), torch.zeros(4, 64)
    codes, scales = torch.zeros(4, 32, dtype=torch.uint8), torch.ones(4, 1).half()
    calls = [(W.pack_quant, dict(codes=codes, scales=scales)),
             (W.norm_rotate, dict(q=h, k=h, v=h, positions=i, table=table, q_gain=None, k_gain=None, k_pages=pages,
                                  v_pages=pages, slots=i)),
             (W.attend_paged, dict(q=h, k_pages=pages, v_pages=pages, page_table=i[:, None], lengths=i)),
             (W.sample_tokens, dict(logits=h[:, 0], uniform=torch.zeros(2)))]
    for call, args in calls:
        for name, value in args.items():
            if value is not None:
                for bad in (None, [1, 2], 3.0):
                    with pytest.raises(TypeError, match=name):
                        call(**{**args, name: bad})
        first = next(iter(args))
        with pytest.raises(TypeError, match=first):
            call(**{**args, first: None}, stream=0)
    with pytest.raises(TypeError, match="workspace"):
        W.attend_paged(**calls[2][1], workspace=7)
    for x, weights in ((None, None), (h[:, 0], None), (h[:, 0], codes)):
        with pytest.raises(TypeError):
            W.matvec_quant(x, weights)


def test_a_copied_matrix_points_to_its_own_memory():
    import copy
    import io
    import pickle
    w = W.QuantMatrix(torch.arange(64, dtype=torch.uint8), 16, 64, 64, 0, torch.float16)
    file = io.BytesIO()
    torch.save(w, file)
    file.seek(0)
    for other in (copy.deepcopy(w), pickle.loads(pickle.dumps(w)), torch.load(file, weights_only=False)):
        assert torch.equal(other.packed, w.packed) and other.packed.data_ptr() != w.packed.data_ptr()
        assert other.ptr == other.packed.data_ptr() and other.spec == (other.ptr, *w.spec[1:])
    assert copy.copy(w).packed is w.packed
