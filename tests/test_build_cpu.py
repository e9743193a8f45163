"""What the build script does where the torch extension cannot be built, and when torch changes (the compilers'
place is taken by a recorder)."""
import importlib.util
import os
import sys
import types

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def build(tmp_path, monkeypatch):
    """The build script with its outputs in a folder of the test's, and (commands, failing): what it ran, and words
    of a command that is to fail."""
    path = os.path.join(ROOT, "persistent_sm_decode_megakernel_gb300", "_build.py")
    spec = importlib.util.spec_from_file_location("_build_under_test", path)
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    monkeypatch.setattr(mod, "OBJ", str(tmp_path / "objs"))
    monkeypatch.setattr(mod, "LIB", str(tmp_path / "libmk.so"))
    monkeypatch.setattr(mod, "EXT", str(tmp_path / "_mk_torch.so"))
    commands, failing = [], []

    def run(cmd, **kw):
        commands.append(cmd)
        bad = any(w in cmd for w in failing)
        if "-o" in cmd and not bad:
            with open(cmd[cmd.index("-o") + 1], "w"):
                pass
        return types.SimpleNamespace(returncode=int(bad), stdout="", stderr="cannot find it" if bad else "")

    monkeypatch.setattr(mod.subprocess, "run", run)
    return mod, commands, failing


def _torch(folder, monkeypatch, cuda, version="2.0"):
    """A torch that is no more than the build script looks at."""
    root = folder / f"torch-{cuda}-{version}"
    (root / "torch" / "lib").mkdir(parents=True)
    (root / "torch" / "__init__.py").write_text(
        f"__version__ = {version!r}\nclass _C:\n    _GLIBCXX_USE_CXX11_ABI = True\n")
    (root / "torch" / "version.py").write_text(f"__version__ = {version!r}\n")
    if cuda:
        (root / "torch" / "lib" / "libc10_cuda.so").write_text("")
    monkeypatch.delitem(sys.modules, "torch", raising=False)
    monkeypatch.syspath_prepend(str(root))


def _compiles_extension(commands):
    return any("mk_torch.cpp" in " ".join(c) for c in commands)


def test_a_torch_without_cuda_leaves_the_library_usable(build, tmp_path, monkeypatch, capsys):
    mod, commands, failing = build
    _torch(tmp_path, monkeypatch, cuda=False)
    failing.append("-lc10_cuda")
    assert mod.build() == mod.LIB and os.path.exists(mod.LIB) and not os.path.exists(mod.EXT)
    assert "paged" in capsys.readouterr().err     # and says what is missing
    commands.clear()
    mod.build()
    assert not commands                           # nothing to do: not built again every time


def test_no_torch_at_all_leaves_the_library_usable(build, tmp_path, monkeypatch, capsys):
    mod, commands, failing = build
    real = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else real(name, *a))
    monkeypatch.setitem(sys.modules, "torch", None)
    mod.build()
    assert os.path.exists(mod.LIB) and not os.path.exists(mod.EXT) and not _compiles_extension(commands)


@pytest.mark.parametrize("word", ["-lc10_cuda", "-w"])
def test_an_extension_that_fails_is_an_error_after_the_library(build, tmp_path, monkeypatch, word):
    """With a CUDA torch a failure to compile or to link is loud, and libmk.so is there all the same."""
    mod, commands, failing = build
    _torch(tmp_path, monkeypatch, cuda=True)
    failing.append(word)
    with pytest.raises(RuntimeError, match="extension|mk_torch"):
        mod.build()
    assert os.path.exists(mod.LIB)
    failing.clear()
    commands.clear()
    mod.build()                                   # and only what is missing is made then
    assert os.path.exists(mod.EXT) and not any(c[0] != "g++" for c in commands)


def test_the_extension_is_rebuilt_when_torch_changes(build, tmp_path, monkeypatch):
    mod, commands, failing = build
    _torch(tmp_path, monkeypatch, cuda=True)
    mod.build()
    assert os.path.exists(mod.EXT)
    commands.clear()
    mod.build()
    assert not commands
    _torch(tmp_path, monkeypatch, cuda=True, version="2.1")
    mod.build()
    assert _compiles_extension(commands) and not any(c[0] != "g++" for c in commands)
