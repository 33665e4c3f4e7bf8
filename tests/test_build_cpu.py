"""What build() compiles and when, with the compilers replaced by a record of their calls."""
import os
import types

import pytest

from paged_kv_attention_07_gb300 import build as B
from paged_kv_attention_07_gb300 import pka


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
    monkeypatch.setattr(B.subprocess, "run", run)
    return calls


@pytest.mark.parametrize("installed", [False, True])
def test_builds_the_library_without_torch(tools, monkeypatch, tmp_path, installed):
    """None at all, or one without CUDA."""
    find_spec = B.importlib.util.find_spec
    other = types.SimpleNamespace(origin=str(tmp_path / "torch" / "__init__.py")) if installed else None
    monkeypatch.setattr(B.importlib.util, "find_spec", lambda name: other if name == "torch" else find_spec(name))
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
    [module] = [f for f in os.listdir(B.OUT_DIR) if f.startswith("_pka_torch") and f.endswith(".so")]
    os.remove(os.path.join(B.OUT_DIR, module))  # the module alone
    B.build()
    assert [tool for tool, _ in tools] == ["g++", "g++"]
    tools.clear()
    B.build(force=True)
    assert len(tools) == len(B.sources()) + 3


@pytest.mark.parametrize("change", ["torch", "python"])
def test_another_torch_or_python_gets_a_module_of_its_own(tools, monkeypatch, change):
    torch = pytest.importorskip("torch")
    B.build()
    here = B.torch_calls_path(torch.__version__)
    assert os.path.exists(here)  # where the calls look for it
    if change == "torch":
        monkeypatch.setattr(B, "_torch_version", lambda _: "9.9.9")
    else:
        soabi = B.sysconfig.get_config_var
        monkeypatch.setattr(B.sysconfig, "get_config_var", lambda n: "cpython-399" if n == "SOABI" else soabi(n))
    there = B.torch_calls_path("9.9.9" if change == "torch" else torch.__version__)
    assert there != here and not os.path.exists(there)
    tools.clear()
    B.build()
    assert os.path.exists(there) and [tool for tool, _ in tools] == ["g++", "g++"]  # the library is what it was


def test_calls_do_not_load_a_module_of_another_torch(monkeypatch):
    torch = pytest.importorskip("torch")
    monkeypatch.setattr(pka, "_torch_calls", None)
    monkeypatch.setattr(pka, "load", lambda: None)
    monkeypatch.setattr(torch, "__version__", "9.9.9")
    with pytest.raises(RuntimeError, match="9.9.9.*not found"):
        pka._calls()
