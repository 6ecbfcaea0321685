"""What the build does when parts of it are missing or fail, with fakes for the
compilers (CPU)."""
import importlib.util
import os
import subprocess
import types

import pytest

from exact_attention_75_gb300 import build as b


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A build directory of its own; compilers that note what they made."""
    made = []

    def touch(path, text=""):
        made.append(os.path.basename(path))
        with open(path, "w") as f:
            f.write(text)
        return ""

    def link(cmd, **kw):
        touch(cmd[cmd.index("-o") + 1])
        return types.SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(b, "BUILD", str(tmp_path))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libattn.so"))
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(b, "_compile", lambda src, obj, verbose: touch(obj))
    monkeypatch.setattr(b, "_compile_binding", lambda src, out: touch(out))
    monkeypatch.setattr(b, "nvcc", lambda: "nvcc")
    monkeypatch.setattr(subprocess, "run", link)
    return made


def test_library_is_built_without_torch(tree, monkeypatch, capsys):
    """The C library needs nvcc alone; the Python entry is left out, and said to be."""
    find = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec",
                        lambda name, *a: None if name == "torch" else find(name, *a))
    assert b.build() == b.LIB and os.path.exists(b.LIB)
    assert not os.path.exists(b.BINDING) and "torch" in capsys.readouterr().err


def test_library_is_built_when_the_python_entry_fails(tree, monkeypatch):
    def fail(src, out):
        raise RuntimeError("compiling binding.cpp failed")
    monkeypatch.setattr(b, "_compile_binding", fail)
    with pytest.raises(RuntimeError, match="binding.cpp"):
        b.build()
    assert os.path.exists(b.LIB) and not os.path.exists(b.BINDING)


def test_python_entry_follows_the_installed_torch(tree, monkeypatch, tmp_path):
    """Compiled once for a torch, and again for another one."""
    torch = tmp_path / "site" / "torch"
    torch.mkdir(parents=True)
    (torch / "version.py").write_text("__version__ = '1'\n")
    spec = types.SimpleNamespace(origin=str(torch / "__init__.py"))
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: spec)
    b.build()
    assert tree.count("_binding.so") == 1
    b.build()
    assert tree.count("_binding.so") == 1 and tree.count("libattn.so.tmp") == 1
    (torch / "version.py").write_text("__version__ = '2'\n")
    b.build()
    assert tree.count("_binding.so") == 2 and tree.count("libattn.so.tmp") == 1
    b.build()
    assert tree.count("_binding.so") == 2
