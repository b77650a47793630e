"""The compiled argument handling beside the library: who needs it, and how it is built (CPU)."""
import importlib
import os
import subprocess

import pytest
import torch

from long_context_sparse_lsa_b200 import binding as lsa
from long_context_sparse_lsa_b200 import build

t = torch.zeros


def _prompt_call():
    bf = torch.bfloat16
    pr = lsa.Prompts(t(2, dtype=torch.int32), t(1, dtype=torch.int64), t(1, dtype=torch.int32), 3, 10, 10)
    q, kv = t(3, 8, 128, dtype=bf), t(10, 2, 128, dtype=bf)
    lsa.lsa_attend_prompt(q, kv, kv, pr, torch.empty_like(q), stream=0)


@pytest.mark.parametrize("how", ["missing", "of another torch"])
def test_only_the_calls_that_go_through_it_need_it(how, monkeypatch, tmp_path):
    monkeypatch.setattr(lsa, "_lib", None)
    monkeypatch.setattr(lsa, "_marshal", None)
    if how == "missing":
        monkeypatch.setattr(lsa, "_MARSHAL_PATH", str(tmp_path / "_marshal.so"))
    else:
        def fails(*_):
            raise ImportError("undefined symbol")
        monkeypatch.setattr(importlib, "import_module", fails)
    assert lsa.lsa_version() == 100
    b = lsa.Batch(t(1, dtype=torch.int64), t(1, dtype=torch.int32), t(3, dtype=torch.int32), t(3, dtype=torch.int32), 10, 10)
    assert lsa.lsa_attend_fp4_workspace_size(b, 8, 2, 128, 3136, 1) > 0
    with pytest.raises(RuntimeError, match="build it with"):
        _prompt_call()
    monkeypatch.undo()
    with pytest.raises(ValueError, match="CUDA device"):  # (host tensors)
        _prompt_call()


@pytest.fixture
def compilers(monkeypatch, tmp_path):
    """build() with compilers that write what they are asked for, into a directory of its own."""
    calls, broken = [], set()

    def run(cmd, **_):
        calls.append(cmd)
        if any(os.path.basename(x) in broken for x in cmd):
            return subprocess.CompletedProcess(cmd, 1, "", "no such header")
        with open(cmd[cmd.index("-o") + 1], "w") as f:
            f.write("\0".join(cmd) + "\0")
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(build.subprocess, "run", run)
    monkeypatch.setattr(build, "_nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    for name, file in (("LIBRARY", "liblsa.so"), ("MARSHAL", "_marshal.so"), ("BUILD_DIR", "_build")):
        monkeypatch.setattr(build, name, str(tmp_path / file))
    return calls, broken


def test_the_library_stands_where_the_module_does_not_build(compilers):
    calls, broken = compilers
    broken.add("marshal.cpp")
    with pytest.raises(RuntimeError, match="marshal.cpp"):
        build.build(force=True)
    assert os.path.exists(build.LIBRARY) and not os.path.exists(build.MARSHAL)
    assert {c[0] for c in calls} == {"/usr/local/cuda/bin/nvcc"}  # no compiler but nvcc (and its own host compiler)


def test_a_module_of_another_build_is_not_used(monkeypatch):
    monkeypatch.setattr(lsa, "_marshal", None)
    assert lsa._marshalling().built_for == build.built_for()
    monkeypatch.setattr(lsa, "_marshal", None)
    monkeypatch.setattr(torch, "__version__", "1.0.0")
    with pytest.raises(RuntimeError, match="torch 1.0.0"):
        _prompt_call()


def test_a_module_of_another_build_is_not_up_to_date(compilers, monkeypatch):
    build.build(force=True)
    with open(build.MARSHAL, "w") as f:
        f.write(f"...{build.built_for()}\0...")
    assert build.up_to_date()
    monkeypatch.setattr(torch, "__version__", torch.__version__ + "0")
    assert not build.up_to_date()
    build.build()
    with open(os.path.join(build.BUILD_DIR, "built_for.h")) as f:
        assert f'"{build.built_for()}"' in f.read()
