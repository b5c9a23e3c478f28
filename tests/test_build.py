"""The binding is built where torch can carry it, and again when torch or Python changes."""
import os
from types import SimpleNamespace

import pytest

from wfst_beam_search_gb300 import _build


def pretend(monkeypatch, folder, files):
    for name in files:
        os.makedirs(os.path.dirname(os.path.join(folder, name)), exist_ok=True)
        open(os.path.join(folder, name), "w").close()
    monkeypatch.setattr(_build.importlib.util, "find_spec", lambda name: SimpleNamespace(origin=os.path.join(folder, "__init__.py")))


CUDA = ["lib/libc10_cuda.so", "lib/libtorch_cuda.so", "include/c10/cuda/CUDAStream.h"]


@pytest.mark.parametrize("missing", [None, *CUDA])
def test_a_torch_without_cuda_leaves_the_decoder_alone(monkeypatch, tmp_path, missing):
    pytest.importorskip("torch")
    if _build._torch() is None:
        pytest.skip("no torch with CUDA, or no Python headers")
    folder = str(tmp_path)
    pretend(monkeypatch, folder, ["version.py", "lib/libtorch_cpu.so", *(f for f in CUDA if f != missing)])
    assert _build._torch() == (None if missing else folder)


def test_the_binding_of_another_torch_is_not_up_to_date(monkeypatch, tmp_path):
    _build.build()
    if _build._torch() is None:
        pytest.skip("no torch with CUDA, or no Python headers")
    assert _build.up_to_date()
    with monkeypatch.context() as m:
        pretend(m, str(tmp_path), ["version.py", *CUDA])
        assert not _build.up_to_date()
    with monkeypatch.context() as m:
        m.setattr(_build.sysconfig, "get_config_var", lambda name: "cpython-399-other")
        assert not _build.up_to_date()
    assert _build.up_to_date()
