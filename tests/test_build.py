"""The build step's handling of PyTorch (no GPU needed): the library does not need it, and a binding
built for another one is not used."""
import ctypes
import os

import pytest
import torch

from paged_gqa_attention_gb300 import build as pa_build
from paged_gqa_attention_gb300 import ops


@pytest.fixture
def elsewhere(monkeypatch, tmp_path):
    """The build writes to a folder of the test's, from one small source file."""
    for name, path in (("LIB_PATH", "libpagedattn.so"), ("BINDING_PATH", "_binding.so"),
                       ("BINDING_ABI_PATH", "_binding.abi"), ("BUILD_DIR", "objects")):
        monkeypatch.setattr(pa_build, name, str(tmp_path / path))
    monkeypatch.setattr(pa_build, "SOURCES", ["kv_append.cu"])
    return tmp_path


def test_the_library_is_built_without_pytorch(elsewhere, monkeypatch, capsys):
    monkeypatch.setattr(pa_build, "_torch", lambda: None)
    assert pa_build.build() == str(elsewhere / "libpagedattn.so")
    ctypes.CDLL(str(elsewhere / "libpagedattn.so"))
    assert not os.path.exists(elsewhere / "_binding.so")
    assert "_binding.so is left out" in capsys.readouterr().err
    assert pa_build.library_up_to_date()


def test_the_library_stands_when_the_binding_does_not_compile(elsewhere, monkeypatch):
    broken = elsewhere / "binding.cpp"
    broken.write_text("#error broken\n")
    monkeypatch.setattr(pa_build, "BINDING_SOURCE", str(broken))
    with pytest.raises(RuntimeError, match="compiling .*binding.cpp failed"):
        pa_build.build()
    assert pa_build.library_up_to_date() and not pa_build.binding_up_to_date()


def test_a_binding_of_another_pytorch_is_stale(monkeypatch):
    pa_build.build()
    assert pa_build.library_up_to_date() and pa_build.binding_up_to_date()
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    assert pa_build.library_up_to_date() and not pa_build.binding_up_to_date()


def test_a_binding_without_a_record_of_its_pytorch_is_stale(monkeypatch, tmp_path):
    pa_build.build()
    monkeypatch.setattr(pa_build, "BINDING_ABI_PATH", str(tmp_path / "none"))
    assert not pa_build.binding_up_to_date()


def test_a_binding_of_another_pytorch_is_not_loaded(monkeypatch):
    pa_build.build()
    monkeypatch.setattr(ops, "_binding", None)
    monkeypatch.setattr(torch, "__version__", "0.0.1+other")
    with pytest.raises(RuntimeError, match="_binding.so was built for torch .* this is torch 0.0.1"):
        ops._usual()
    assert ops._binding is None


def test_a_second_build_beside_a_first_leaves_its_record_in_place(elsewhere, monkeypatch):
    """Two processes that build at once: the record of the binding is never away once one is done."""
    small = elsewhere / "binding.cpp"
    small.write_text("extern \"C\" int nothing() { return 0; }\n")
    monkeypatch.setattr(pa_build, "BINDING_SOURCE", str(small))
    pa_build.build()
    assert pa_build.binding_up_to_date()
    removed = []
    monkeypatch.setattr(os, "remove", removed.append)
    pa_build.build(force=True)
    assert pa_build.binding_up_to_date() and not removed
