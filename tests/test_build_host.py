"""The build without a GPU: what each part needs and what makes it stale, with the
compilers replaced by a record of their commands."""
import importlib.util
import os
import subprocess
import sys
import types

import pytest
import torch

import exact_tiled_attention_gb300 as gb
from exact_tiled_attention_gb300 import _build, paged

SOURCE = os.path.abspath(_build.__file__)


@pytest.fixture
def fake(tmp_path, monkeypatch):
    """A copy of the module that builds into an empty folder; `fake.ran` holds the
    commands, each of which writes its output unless its tool is in `fake.broken`."""
    spec = importlib.util.spec_from_file_location("build_under_test", SOURCE)
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    m.PKG, m.BUILD, m.LIB = str(tmp_path), str(tmp_path / "objects"), str(tmp_path / "libgbattn.so")
    m.ran, m.broken = [], set()

    def run(cmd, **kw):
        tool = os.path.basename(cmd[0])
        m.ran.append((tool, cmd[cmd.index("-o") + 1]))
        bad = tool in m.broken
        if not bad:
            open(cmd[cmd.index("-o") + 1], "w").close()
        return types.SimpleNamespace(returncode=int(bad), stdout="", stderr="")

    monkeypatch.setattr(m, "nvcc", lambda: "/cuda/bin/nvcc")
    monkeypatch.setattr(m, "subprocess", types.SimpleNamespace(run=run))
    monkeypatch.setenv("CXX", "/usr/bin/g++")
    return m


def _tools(m):
    ran, m.ran[:] = [t for t, _ in m.ran], []
    return ran


def test_library_and_binding(fake):
    fake.build()
    tools = _tools(fake)
    assert tools.count("nvcc") == len(fake.SOURCES) + 1 and tools.count("g++") == 2
    assert os.path.exists(fake.LIB) and os.path.exists(fake.ext_path())
    fake.build()
    assert _tools(fake) == []


def test_library_alone_without_pytorch(fake, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch raises ImportError
    fake.build()
    assert "g++" not in _tools(fake) and os.path.exists(fake.LIB)
    assert "PyTorch" in capsys.readouterr().err
    fake.build()
    assert _tools(fake) == []


def test_a_failing_binding_leaves_the_library(fake):
    fake.broken = {"g++"}
    with pytest.raises(RuntimeError, match="g\\+\\+"):
        fake.build()
    assert os.path.exists(fake.LIB) and not os.path.exists(fake.ext_path())
    fake.broken = set()
    _tools(fake)
    fake.build()
    assert _tools(fake) == ["g++", "g++"]  # the library is up to date


def test_another_pytorch_gets_a_binding_of_its_own(fake, monkeypatch):
    fake.build()
    first = fake.ext_path()
    _tools(fake)
    monkeypatch.setattr(torch, "__version__", "0.0.1")
    assert fake.ext_path() != first
    fake.build()
    assert _tools(fake) == ["g++", "g++"] and os.path.exists(first) and os.path.exists(fake.ext_path())


def test_a_binding_for_another_pytorch_is_not_loaded(monkeypatch):
    _build.build()
    monkeypatch.setattr(paged, "_native", None)
    with monkeypatch.context() as m:
        m.setattr(torch, "__version__", "0.0.1")
        with pytest.raises(RuntimeError, match="is missing"):
            gb.attn_cache_gather(None, None, None, None, 1)
    with pytest.raises((TypeError, ValueError)):  # loaded, and refused by its checks
        gb.attn_cache_gather(None, None, None, None, 1)


def test_the_script_needs_no_pytorch():
    """What `python _build.py` imports before it compiles."""
    code = ("import sys, runpy; sys.modules['torch'] = None; sys.argv = ['_build.py']\n"
            f"m = runpy.run_path({SOURCE!r}); print(len(m['SOURCES']))")
    r = subprocess.run([sys.executable, "-c", code], capture_output=True, text=True)
    assert r.returncode == 0 and int(r.stdout) == len(_build.SOURCES), r.stderr
