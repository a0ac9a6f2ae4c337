"""The build of the library and of its PyTorch binding (no GPU, no compiler)."""
import os
import subprocess

import pytest

from mla_decode_attention_12_b200 import build


@pytest.fixture
def empty(tmp_path, monkeypatch):
    """A package folder without built files, and compilers that write their output file; the commands run."""
    monkeypatch.setattr(build, "LIB", str(tmp_path / "_mla_decode.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_mla_torch.so"))
    monkeypatch.setattr(build, "BINDING_STAMP", str(tmp_path / "_mla_torch.so.built_with"))
    ran = []

    def run(cmd, verbose):
        ran.append(cmd)
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("built")

    monkeypatch.setattr(build, "_run", run)
    return ran


def test_the_library_is_linked_where_the_binding_does_not_compile(empty, monkeypatch):
    def fails(*args):
        raise subprocess.CalledProcessError(1, "g++")

    monkeypatch.setattr(build, "_compile_binding", fails)
    with pytest.raises(subprocess.CalledProcessError):
        build.build(out=build.LIB)
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)


def test_a_binding_of_another_torch_is_built_again(empty):
    import torch

    build.build(out=build.LIB)
    assert os.path.exists(build.LIB) and os.path.exists(build.BINDING)
    n = len(empty)
    build.build(out=build.LIB)
    assert len(empty) == n  # up to date
    with open(build.BINDING_STAMP) as f:
        mine = f.read()
    assert torch.__version__ in mine
    with open(build.BINDING_STAMP, "w") as f:
        f.write(mine.replace(torch.__version__, "1.0.0"))
    build.build(out=build.LIB)
    assert len(empty) == n + 2  # the binding alone: compiled and linked
    assert build.binding_up_to_date()
    os.remove(build.BINDING_STAMP)
    assert not build.binding_up_to_date()


def test_the_binding_is_compiled_for_torchs_abi(empty):
    import torch

    build.build(out=build.LIB)
    compiled = [c for c in empty if build.BINDING_SOURCE in c]
    assert len(compiled) == 1 and f"-D_GLIBCXX_USE_CXX11_ABI={int(torch.compiled_with_cxx11_abi())}" in compiled[0]


def test_other_builds_leave_the_binding_alone(empty, tmp_path):
    build.build(extra=["-DMLA_TIMELINE"], out=str(tmp_path / "other.so"))
    assert not os.path.exists(build.BINDING) and not any(build.BINDING_SOURCE in c for c in empty)
