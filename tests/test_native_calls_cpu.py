"""The binding's native part (_calls.so) where it cannot be built or was built for another torch: the library is
built and called without it."""
import sys
import types
import warnings

import pytest
import torch

import context_zigzag_cp_b200 as cz
from context_zigzag_cp_b200 import _lib, build


@pytest.fixture(scope="module", autouse=True)
def built():
    build.build()


def refused_in_python():
    """The call reaches the checks in Python, which name the device."""
    with pytest.raises(ValueError, match="CUDA device"):
        cz.rope([torch.zeros(1, 1, 2, 64, dtype=torch.bfloat16)], torch.ones(32, dtype=torch.float64))


def test_the_library_is_built_without_a_compiler_for_the_native_part(monkeypatch, tmp_path):
    run = []

    def no_compiler(cmd, target, verbose):
        run.append(target)
        raise FileNotFoundError("g++")

    monkeypatch.setattr(build, "CALLS", str(tmp_path / "_calls.so"))
    monkeypatch.setattr(build, "_run", no_compiler)
    with pytest.warns(UserWarning, match="_calls.so"):
        assert build.build() == build.LIB
    assert run == [build.CALLS]


def test_a_native_part_for_another_torch_is_built_again(monkeypatch, tmp_path):
    assert build.calls_up_to_date()
    with open(build.CALLS, "rb") as f:
        data = f.read()
    mark = build.calls_mark().encode() + b"\0"
    assert data.count(mark) == 1
    (tmp_path / "_calls.so").write_bytes(data.replace(mark, b"built for torch 0.0\0"))
    monkeypatch.setattr(build, "CALLS", str(tmp_path / "_calls.so"))
    assert not build.calls_up_to_date()


@pytest.mark.parametrize("module", [None, "other"])
def test_calls_go_through_python(monkeypatch, module):
    if module:
        module = types.ModuleType("context_zigzag_cp_b200._calls", "built for torch 0.0")
        module.bind = lambda *args: pytest.fail("bound")
    monkeypatch.setattr(_lib, "_calls", None)
    monkeypatch.setitem(sys.modules, "context_zigzag_cp_b200._calls", module)
    monkeypatch.delattr(cz, "_calls", raising=False)
    with pytest.warns(UserWarning, match="through Python"):
        refused_in_python()
    with warnings.catch_warnings():
        warnings.simplefilter("error")     # said once
        refused_in_python()


def test_the_native_part_is_this_torchs(monkeypatch):
    monkeypatch.setattr(_lib, "_calls", None)
    assert _lib.calls().__doc__ == build.calls_mark()
