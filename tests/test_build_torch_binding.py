"""The torch binding is rebuilt, and refused, when it was made for another torch or Python."""

import subprocess
import sys

import pytest

import grouped_query_attention_attn_b200 as gqa
from grouped_query_attention_attn_b200 import _binding, build

MODULE = "grouped_query_attention_attn_b200._torch_binding"


@pytest.fixture
def compiles(gqa_lib, monkeypatch):
    """The commands that the build would run; none is run, all fail."""
    cmds = []

    def run(cmd, **kw):
        cmds.append(cmd)
        return subprocess.CompletedProcess(cmd, 1, "", "a stand-in")

    monkeypatch.setattr(build.subprocess, "run", run)
    return cmds


def test_up_to_date(compiles):
    build.build_library()
    assert compiles == []


@pytest.mark.parametrize("here", ["torch 2.0.0, CXX11 ABI 0, Python .cpython-310-x86_64-linux-gnu.so", "torch 2.1"])
def test_another_torch_means_a_rebuild(compiles, monkeypatch, here):
    assert build.torch_binding_fits()
    monkeypatch.setattr(build, "torch_binding_target", lambda: here)
    with pytest.raises(RuntimeError, match="a stand-in"):
        build.build_library()
    assert len(compiles) == 1 and compiles[0][0] == "g++" and f'-DGQA_BUILT_FOR="<{here}>"' in compiles[0]


def test_another_torch_is_refused(gqa_lib, monkeypatch):
    monkeypatch.setattr(_binding, "_torch", None)
    monkeypatch.setattr(build, "torch_binding_target", lambda: "torch 9.9.9")
    with pytest.raises(RuntimeError, match="not built for torch 9.9.9"):
        _binding.torch_binding()
    monkeypatch.setattr(build, "TORCH_BINDING", build.TORCH_BINDING + ".missing")
    with pytest.raises(RuntimeError, match="is not built"):
        _binding.torch_binding()


def test_it_says_what_it_was_built_for(gqa_lib):
    assert _binding.torch_binding().built_for == f"<{build.torch_binding_target()}>"


def test_the_reason_of_a_failed_import_is_given(gqa_lib, monkeypatch):
    monkeypatch.setattr(_binding, "_torch", None)
    monkeypatch.delattr(gqa, "_torch_binding", raising=False)
    monkeypatch.setitem(sys.modules, MODULE, None)
    with pytest.raises(RuntimeError, match="does not load .*halted"):
        _binding.torch_binding()


@pytest.mark.parametrize("missing", ["torch", "g++"])
def test_the_library_is_built_without(compiles, monkeypatch, capsys, missing):
    monkeypatch.setattr(build, "TORCH_BINDING", build.TORCH_BINDING + ".missing")
    if missing == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)
        monkeypatch.setattr(build.importlib.util, "find_spec", lambda name: None)
    else:
        monkeypatch.setattr(build.shutil, "which", lambda name: None)
        monkeypatch.setattr(build.subprocess, "run", no_such_file)
    assert build.build_library() == build.LIB
    assert f"no {missing}" in capsys.readouterr().err and compiles == []


def no_such_file(cmd, **kw):
    raise FileNotFoundError(cmd[0])
