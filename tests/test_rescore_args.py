"""What the operators of a rescoring pass refuse without a GPU: sizes and NULL
pointers at the C entries, host tensors and wrong types in the binding."""
import os
import re

import pytest

import wfst_beam_search_gb300 as W
from wfst_beam_search_gb300 import _build

torch = pytest.importorskip("torch")


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return W.load()


def test_blocks_are_as_the_header_declares_them(lib, tmp_path):
    """Sizes of the argument blocks, asked of the C compiler."""
    import shutil
    import struct
    import subprocess
    from wfst_beam_search_gb300 import _ops
    cc = shutil.which("gcc") or shutil.which("cc")
    if not cc:
        pytest.skip("no C compiler")
    src = tmp_path / "sizes.c"
    src.write_text('#include "wfst_gb300.h"\n#include <stdio.h>\nint main(void) { printf("%zu %zu %zu\\n", '
                   "sizeof(wfst_prefix_args), sizeof(wfst_score_args), sizeof(wfst_lowrank_args)); return 0; }\n")
    subprocess.run([cc, "-I", _build.INCLUDE, str(src), "-o", str(tmp_path / "sizes")], check=True)
    said = subprocess.run([str(tmp_path / "sizes")], capture_output=True, text=True, check=True).stdout
    packs = (_ops._PREFIX, _ops._SCORE, _ops._LOWRANK)
    assert [int(v) for v in said.split()] == [p.__self__.size for p in packs]
    assert all(isinstance(p.__self__, struct.Struct) for p in packs)
    header = open(os.path.join(_build.INCLUDE, "wfst_gb300.h")).read()
    assert int(re.search(r"#define WFST_SCORE_TOP (\d+)", header).group(1)) == W.WFST_SCORE_TOP


def test_null_blocks(lib):
    for f in (lib.wfst_attend_prefix, lib.wfst_score_tokens, lib.wfst_add_lowrank):
        assert f(None, None) == -1 and b"NULL" in lib.wfst_last_error()
    assert lib.wfst_prefix_size(1, 1, 1, 64, None) == -1


def test_sizes_of_a_workspace(lib):
    for lanes, hq, hkv, d in ((1, 1, 1, 64), (64, 32, 8, 128), (128, 64, 8, 256), (0, 4, 2, 64), (3, 0, 1, 128)):
        size = W.wfst_prefix_size(lanes, hq, hkv, d)
        assert size >= W.wfst_attend_size() and size % 16 == 0
        assert W.wfst_prefix_size(lanes + 1, hq, hkv, d) >= size
    for bad in ((1, 1, 1, 80), (1, 3, 2, 64), (1, 1, 0, 64), (-1, 1, 1, 64), (1, -2, 1, 64), (2 ** 31 - 1, 2 ** 30, 1, 256)):
        with pytest.raises(W.WfstError) as e:
            W.wfst_prefix_size(*bad)
        assert e.value.code == -1


def test_fields_are_checked_in_the_blocks(lib):
    from wfst_beam_search_gb300 import _ops

    def prefix(**kw):
        f = dict(device=-1, dtype=1, lanes=1, hq=2, hkv=1, d=64, pwidth=1, width=1, pages=1, page=16, scale=1.0)
        f.update(kw)
        return lib.wfst_attend_prefix(_ops._PREFIX(*([0] * 22), *f.values()), None), lib.wfst_last_error()

    def score(**kw):
        f = dict(stride=10, device=-1, dtype=0, rows=1, vocab=10, top=0)
        f.update(kw)
        return lib.wfst_score_tokens(_ops._SCORE(*([0] * 6), *f.values()), None), lib.wfst_last_error()

    def lowrank(**kw):
        f = dict(sy=64, sx=64, so=64, ss_a=0, ss_j=64, se_a=0, se_n=16, device=-1, dtype=1, rows=1, n=64, k=64, rank=16, adapters=1)
        f.update(kw)
        return lib.wfst_add_lowrank(_ops._LOWRANK(*([0] * 7), *f.values()), None), lib.wfst_last_error()

    assert prefix(lanes=0)[0] == 0 and score(rows=0)[0] == 0 and lowrank(rows=0)[0] == 0 and lowrank(n=0)[0] == 0
    for call, word, change in [
            (prefix, b"NULL", {}), (prefix, b"dtype", dict(dtype=0)), (prefix, b"head_dim", dict(d=32)),
            (prefix, b"multiple", dict(hq=3, hkv=2)), (prefix, b"page_size", dict(page=0)), (prefix, b"page_size", dict(pwidth=-1)),
            (prefix, b"2^31", dict(page=1 << 20, width=1 << 12)), (prefix, b"2^31", dict(page=1 << 20, pwidth=1 << 12)),
            (prefix, b"scale", dict(scale=float("nan"))), (prefix, b"counts", dict(lanes=-1)),
            (score, b"NULL", {}), (score, b"dtype", dict(dtype=3)), (score, b"vocab", dict(vocab=0)), (score, b"rows", dict(rows=-1)),
            (score, b"vocab", dict(vocab=(1 << 20) + 1)), (score, b"stride", dict(rows=2, stride=9)),
            (score, b"top", dict(top=-1)), (score, b"top", dict(top=65)),
            (lowrank, b"NULL", {}), (lowrank, b"dtype", dict(dtype=0)), (lowrank, b"counts", dict(rows=-1)),
            (lowrank, b"multiple", dict(k=60)), (lowrank, b"multiple", dict(k=0)), (lowrank, b"rank", dict(rank=12)),
            (lowrank, b"rank", dict(rank=0)), (lowrank, b"rank", dict(rank=136))]:
        rc, said = call(**change)
        assert rc == -1 and word in said, (call.__name__, change, said)


def calls():
    h = torch.zeros(2, 1, 64, dtype=torch.float16)
    i = torch.zeros(2, dtype=torch.int32)
    pages = torch.zeros(1, 16, 1, 64, dtype=torch.float16)
    return [(W.attend_prefix, dict(q=h, k_pages=pages, v_pages=pages, prefix_table=i, prefix_length=i[:1],
                                   page_table=i[:, None], lengths=i)),
            (W.score_tokens, dict(logits=h[:, 0], tokens=i)),
            (W.add_lowrank, dict(y=h[:, 0], x=h[:, 0], shrink=h[:1].expand(1, 8, 64), expand=torch.zeros(1, 64, 8).half(), adapters=i))]


def test_host_tensors_are_refused():
    for call, args in calls():
        with pytest.raises(ValueError, match="CUDA"):
            call(**args)


def test_inputs_that_require_a_gradient_are_refused():
    for call, args in calls():
        first = next(iter(args))
        asks = args[first].clone().requires_grad_()
        with pytest.raises(ValueError, match="gradient"):
            call(**{**args, first: asks})
        with torch.no_grad(), pytest.raises(ValueError, match="CUDA"):
            call(**{**args, first: asks})


def test_what_is_no_tensor_is_a_type_error():
    for call, args in calls():
        for name in args:
            for bad in (None, [1, 2], 3.0):
                with pytest.raises(TypeError, match=name):
                    call(**{**args, name: bad})
        first = next(iter(args))
        with pytest.raises(TypeError, match=first):
            call(**{**args, first: None}, stream=0)
    with pytest.raises(TypeError, match="workspace"):
        W.attend_prefix(**calls()[0][1], workspace=7)


def test_a_workspace_is_zeroed_where_it_has_to_be(monkeypatch):
    full = torch.full

    def garbage(size, dtype, device):
        return full((size,), 255, dtype=dtype, device=device)

    monkeypatch.setattr(torch, "empty", garbage)
    ws = W.attend_prefix_workspace(3, 4, 2, 64, "cpu")
    assert ws.shape == (W.wfst_prefix_size(3, 4, 2, 64),)
    assert not bool(ws[:W.WFST_ATTEND_ZEROED].any()) and bool((ws[W.WFST_ATTEND_ZEROED:] == 255).all())
