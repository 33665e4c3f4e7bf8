"""What build() compiles and when, with the compilers replaced by a record of their calls."""
import os
import types

import pytest

from paged_kv_attention_07_gb300 import build as B


@pytest.fixture
def tools(monkeypatch, tmp_path):
    """A build directory of its own; the compilers' calls, each of which makes its output."""
    calls = []

    def run(cmd, **_):
        out = cmd[cmd.index("-o") + 1]
        calls.append((os.path.basename(cmd[0]), os.path.basename(out).split(".")[0]))
        open(out, "w").close()
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(B, "OUT_DIR", str(tmp_path))
    monkeypatch.setattr(B, "LIB", str(tmp_path / "libpka.so"))
    monkeypatch.setattr(B, "TORCH_CALLS", str(tmp_path / "_pka_torch.so"))
    monkeypatch.setattr(B.subprocess, "run", run)
    return calls


def test_builds_the_library_without_torch(tools, monkeypatch):
    find_spec = B.importlib.util.find_spec
    monkeypatch.setattr(B.importlib.util, "find_spec", lambda name: None if name == "torch" else find_spec(name))
    assert B.build() == B.LIB and os.path.exists(B.LIB)
    assert len(tools) == len(B.sources()) + 1 and all(tool == "nvcc" for tool, _ in tools)
    tools.clear()
    assert B.build() == B.LIB and not tools  # and once only


def test_builds_what_is_out_of_date(tools):
    pytest.importorskip("torch")
    B.build()
    assert ("nvcc", "libpka") in tools and ("g++", "_pka_torch") in tools
    tools.clear()
    B.build()
    assert not tools
    os.remove(B.TORCH_CALLS)  # the module alone
    B.build()
    assert [tool for tool, _ in tools] == ["g++", "g++"]
    tools.clear()
    B.build(force=True)
    assert len(tools) == len(B.sources()) + 3
