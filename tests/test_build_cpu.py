"""The build's two products: the library comes first and does not depend on the Python binding."""
import os
import types

import pytest

from scaled_fp8_linear_amd import build as b


@pytest.fixture
def stubbed(tmp_path, monkeypatch):
    """A build into a folder of its own whose compiler and linker only make their output files."""
    monkeypatch.setattr(b, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libfp8lin.so"))
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "_binding.so"))

    def run(cmd, **kw):
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(b.subprocess, "run", run)
    return tmp_path


def test_both_products(stubbed):
    assert b.build() == b.LIB
    assert os.path.exists(b.LIB) and os.path.exists(b.BINDING)
    assert not os.path.exists(b.LIB + ".tmp") and not os.path.exists(b.BINDING + ".tmp")


@pytest.mark.parametrize("error", [RuntimeError("g++ failed on binding.cpp"),
                                   FileNotFoundError("g++"), ImportError("no torch")])
def test_the_library_is_built_without_the_binding(stubbed, monkeypatch, error):
    def fail():
        raise error

    monkeypatch.setattr(b, "_compile_binding", fail)
    with open(b.BINDING, "w") as f:
        f.write("of an earlier library")
    with pytest.raises(RuntimeError, match="not .*_binding.so") as e:
        b.build()
    assert str(error) in str(e.value) and e.value.__cause__ is error
    assert os.path.exists(b.LIB) and not os.path.exists(b.BINDING)


def test_a_kernel_that_does_not_compile_ends_the_build(stubbed, monkeypatch):
    def fail(src):
        raise RuntimeError(f"hipcc failed on {src}")

    monkeypatch.setattr(b, "_compile", fail)
    with pytest.raises(RuntimeError, match="hipcc failed"):
        b.build()
    assert not os.path.exists(b.LIB)
