"""What a build leaves behind when a part of it fails, and when what is there counts as built."""
import os
import stat

import pytest

from transformer_rope_positional_gb300 import build as B


@pytest.fixture
def fakes(tmp_path, monkeypatch):
    """A build into a folder of its own by compilers that only make the output file; returns where."""
    fake = tmp_path / "compiler"
    fake.write_text('#!/bin/sh\nwhile [ $# -gt 0 ]; do [ "$1" = -o ] && echo made > "$2"; shift; done\n')
    fake.chmod(fake.stat().st_mode | stat.S_IXUSR)
    out = tmp_path / "lib"
    for name, value in (("LIB_DIR", str(out)), ("BUILD_DIR", str(tmp_path / "objects")),
                        ("LIB_PATH", str(out / "librope_gb300.so")), ("BINDING_PATH", str(out / "rope_binding.so"))):
        monkeypatch.setattr(B, name, value)
    monkeypatch.setenv("NVCC", str(fake))
    monkeypatch.setenv("CXX", str(fake))
    return out


def test_library_is_linked_where_the_binding_does_not_compile(fakes, monkeypatch):
    """The C library needs nothing of torch: it is there, and the build says that the binding is not."""
    monkeypatch.setenv("CXX", "/bin/false")
    with pytest.raises(RuntimeError, match="binding.cpp"):
        B.build(force=True)
    assert (fakes / "librope_gb300.so").exists()
    assert not (fakes / "rope_binding.so").exists()
    assert not B.up_to_date(B.LIB_PATH)


def test_binding_is_built_again_for_another_torch_or_python(fakes, monkeypatch):
    """It is linked against the torch and the Python that built it, whatever the files' times."""
    B.build(force=True)
    assert (fakes / "rope_binding.so").exists() and B.up_to_date(B.LIB_PATH)
    built_for = B.binding_target()
    monkeypatch.setattr(B, "binding_target", lambda: built_for + "+other")
    assert not B.up_to_date(B.LIB_PATH)
    B.build()
    assert B.up_to_date(B.LIB_PATH)
    monkeypatch.setattr(B, "binding_target", lambda: built_for)
    assert not B.up_to_date(B.LIB_PATH)


def test_binding_of_another_torch_is_not_loaded(monkeypatch):
    import torch

    import transformer_rope_positional_gb300 as R
    from transformer_rope_positional_gb300 import _capi as C

    B.build()
    assert torch.__version__ in B.binding_target()
    monkeypatch.setattr(C, "_binding", None)
    monkeypatch.setattr(B, "binding_target", lambda: "another torch")
    with pytest.raises(RuntimeError, match="transformer_rope_positional_gb300.build"):
        R.rope_frequencies(64)
    monkeypatch.undo()
    assert len(R.rope_frequencies(64)[0]) == 32
