"""What build() makes and when: the library, and the quick calls of the attention operators,
which belong to one Python and one torch."""

import os
import sysconfig
import warnings

import pytest
import torch

import rank_bit_residual_b200.attention as rba
from rank_bit_residual_b200 import build as rbuild


def test_quick_calls_are_built_and_loaded():
    rbuild.build()
    assert rbuild.calls_up_to_date()
    assert hasattr(rba._load_calls(), "prompt")


def test_quick_calls_of_another_torch_or_python_are_not_taken(monkeypatch):
    rbuild.build()
    here = rbuild.calls_path()
    assert torch.__version__ in here and sysconfig.get_config_var("SOABI") in here
    for change in (lambda m: m.setattr(torch, "__version__", "9.9.9"),
                   lambda m: m.setattr(sysconfig, "get_config_var", lambda name: "cpython-399-x86_64-linux-gnu"),
                   lambda m: m.setattr(torch, "compiled_with_cxx11_abi", lambda: False)):
        with monkeypatch.context() as m:
            change(m)
            assert rbuild.calls_path() != here and not rbuild.calls_up_to_date()
            with pytest.raises(ImportError, match="not built"):
                rba._load_calls()
    assert rbuild.calls_up_to_date() and os.path.exists(here)


def test_without_quick_calls_the_long_way_is_taken(monkeypatch, tmp_path):
    """One warning, and the calls go on to the checks of the long way."""
    monkeypatch.setattr(rbuild, "calls_path", lambda: str(tmp_path / "none.so"))
    monkeypatch.setattr(rba, "_calls_lib", None)
    monkeypatch.setattr(rba, "_calls", None)
    t = torch.zeros((2, 4, 64), dtype=torch.bfloat16)
    with pytest.warns(RuntimeWarning, match="quick way"), pytest.raises(ValueError):
        rba.svdq_qk_norm_rope(t, t)                                  # host tensors
    with warnings.catch_warnings():
        warnings.simplefilter("error")
        with pytest.raises(ValueError):
            rba.svdq_attention_prompt(t, t, t)


def test_nothing_to_build_needs_no_compiler(monkeypatch):
    """Where library and quick calls are up to date, build() asks for no toolkit."""
    rbuild.build()

    def none():
        raise RuntimeError("no nvcc here")
    monkeypatch.setattr(rbuild, "nvcc", none)
    assert rbuild.build() == rbuild.LIB


@pytest.fixture
def small_tree(monkeypatch, tmp_path):
    """A tree of one source with a stand-in for nvcc, which makes the file that -o names."""
    src = tmp_path / "csrc"
    src.mkdir()
    (src / "one.cu").write_text("")
    (src / "attention_calls.cpp").write_text("#error no torch headers\n")
    cc = tmp_path / "nvcc"
    cc.write_text("#!/bin/sh\nwhile [ $# -gt 0 ]; do [ \"$1\" = -o ] && : > \"$2\"; shift; done\n")
    cc.chmod(0o755)
    for name, value in (("CSRC", src), ("BUILD", tmp_path / "_build"), ("LIB", tmp_path / "libsvdq.so"),
                        ("CALLS_SRC", src / "attention_calls.cpp"), ("INCLUDE", tmp_path / "include")):
        monkeypatch.setattr(rbuild, name, str(value))
    monkeypatch.setattr(rbuild, "calls_path", lambda: str(tmp_path / "_calls.so"))
    monkeypatch.setenv("NVCC", str(cc))
    return tmp_path


def missing_compiler(out):
    return ["/nowhere/g++", "-o", out]


def missing_torch(out):
    raise ImportError("no torch")


@pytest.mark.parametrize("command", [None, missing_compiler, missing_torch])
def test_the_library_is_built_whatever_becomes_of_the_quick_calls(small_tree, monkeypatch, command):
    if command is not None:
        monkeypatch.setattr(rbuild, "calls_command", command)
    for _ in range(2):                       # the second time only the quick calls are missing
        with pytest.warns(RuntimeWarning, match="quick calls"):
            assert rbuild.build() == rbuild.LIB
        assert os.path.exists(rbuild.LIB) and not os.path.exists(rbuild.calls_path())


def test_a_failure_of_the_library_raises(small_tree, monkeypatch):
    monkeypatch.setattr(rbuild, "calls_command", lambda out: ["touch", out])
    (small_tree / "nvcc").write_text("#!/bin/sh\necho wrong; exit 1\n")
    with pytest.raises(RuntimeError, match="wrong"):
        rbuild.build()
    assert not os.path.exists(rbuild.LIB)
