"""What the build makes when a tool or torch is missing, and when torch changes: compilers replaced by a stand-in
that creates the file after -o."""
import os
import subprocess
import types

import pytest
import torch

from diagonal_state_space_gb300 import build


@pytest.fixture
def tools(monkeypatch, tmp_path):
    """runs: the programs that were run, with their outputs' names; broken: programs that fail."""
    t = types.SimpleNamespace(runs=[], broken=set())
    src = tmp_path / "one.cu"
    src.write_text("")
    monkeypatch.setattr(build, "OBJ", str(tmp_path / "obj"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libs5.so"))
    monkeypatch.setattr(build, "MARSHAL", str(tmp_path / "_marshal.so"))
    monkeypatch.setattr(build, "sources", lambda: [str(src)])
    monkeypatch.setattr(build, "_nvcc", lambda: "/cuda/bin/nvcc")
    monkeypatch.delenv("CXX", raising=False)

    def run(cmd, **kw):
        tool, out = os.path.basename(cmd[0]), cmd[cmd.index("-o") + 1]
        t.runs.append((tool, os.path.basename(out)))
        if tool in t.broken:
            return subprocess.CompletedProcess(cmd, 1, "", "no " + tool)
        open(out, "w").close()
        return subprocess.CompletedProcess(cmd, 0, "", "")

    monkeypatch.setattr(subprocess, "run", run)
    return t


def test_the_library_is_linked_without_a_host_compiler(tools):
    tools.broken.add("g++")
    with pytest.raises(RuntimeError, match="g..."):
        build.build()
    assert os.path.exists(build.LIB)


def test_without_torch_the_library_is_all_there_is_to_build(tools, monkeypatch):
    monkeypatch.setattr(build, "_has_torch", lambda: False)
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert not any(tool == "g++" for tool, _ in tools.runs) and not os.path.exists(build.MARSHAL)


def test_a_torch_without_cuda_gets_no_binding(monkeypatch):
    assert build._has_torch() == (torch.version.cuda is not None)
    monkeypatch.setattr(torch.version, "cuda", None)
    assert not build._has_torch()
    monkeypatch.setitem(__import__("sys").modules, "torch", None)
    assert not build._has_torch()


def links(tools):
    return [out for tool, out in tools.runs if tool == "g++" and out.startswith("_marshal.so")]


@pytest.mark.parametrize("what", ["torch", "python", "abi"])
def test_the_binding_is_linked_again_when_what_it_was_made_for_comes_back(tools, monkeypatch, what):
    def become(which):
        if what == "torch":
            monkeypatch.setattr(torch, "__version__", which)
        elif what == "python":
            monkeypatch.setattr(build.sysconfig, "get_config_var", lambda name: which)
        else:
            monkeypatch.setattr(torch._C, "_GLIBCXX_USE_CXX11_ABI", which == "a")

    for n, which in enumerate("aba", 1):
        become(which)
        build.build()
        assert len(links(tools)) == n
        build.build()
        assert len(links(tools)) == n        # nothing has changed
