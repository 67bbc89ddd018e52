"""The build: the plain C library needs no torch, and a failure of the CPython
binding leaves it linked."""
import ctypes
import os
import sys

import pytest

from paged_kv_cache_193_gb300 import build

SOURCE = 'extern "C" int pa_tiny(void) { return 7; }\n'


@pytest.fixture
def tree(monkeypatch, tmp_path):
    """A library of one small source, built into a folder of its own."""
    src = tmp_path / "tiny.cu"
    src.write_text(SOURCE)
    out = tmp_path / "out"
    monkeypatch.setattr(build, "_sources", lambda: [str(src)])
    monkeypatch.setattr(build, "OUT_DIR", str(out))
    monkeypatch.setattr(build, "LIB", str(out / "libpa.so"))
    monkeypatch.setattr(build, "BINDING", str(out / "_pa_binding.so"))
    return out


def linked(path):
    return ctypes.CDLL(str(path)).pa_tiny() == 7


def test_the_library_is_built_without_torch(tree, monkeypatch, capfd):
    monkeypatch.setitem(sys.modules, "torch", None)  # not importable
    lib = build.build()
    assert lib == str(tree / "libpa.so") and linked(lib)
    assert not (tree / "_pa_binding.so").exists()
    assert "torch" in capfd.readouterr().err  # said, not silent
    # and again, with nothing to compile
    before = os.path.getmtime(lib)
    assert build.build() == lib and os.path.getmtime(lib) == before


def test_the_library_is_built_beside_a_torch_without_cuda(tree, monkeypatch, tmp_path):
    torch = type(sys)("torch")
    torch.__file__ = str(tmp_path / "torch" / "__init__.py")
    torch.__version__ = "0+cpu"
    (tmp_path / "torch" / "lib").mkdir(parents=True)
    monkeypatch.setitem(sys.modules, "torch", torch)
    assert linked(build.build()) and not (tree / "_pa_binding.so").exists()
    with pytest.raises(ImportError, match="CUDA"):
        build.build_binding(force=True)


def test_a_binding_that_does_not_compile_is_raised_after_the_link(tree, monkeypatch, tmp_path):
    broken = tmp_path / "binding.cpp"
    broken.write_text("#error broken\n")
    monkeypatch.setattr(build, "BINDING_SRC", str(broken))
    with pytest.raises(RuntimeError, match="binding"):
        build.build()
    assert linked(tree / "libpa.so")


def test_a_binding_of_another_torch_is_built_again(tree, monkeypatch):
    """Its C++ interface is that of the torch, and the Python, that it was built with, whatever the files' times."""
    built = []

    def compiled(cmd, **kw):
        if build.BINDING_SRC in cmd:
            built.append(cmd)
            open(cmd[cmd.index("-o") + 1], "wb").close()
            return build.subprocess.CompletedProcess(cmd, 0, "", "")
        return run(cmd, **kw)

    run = build.subprocess.run
    monkeypatch.setattr(build.subprocess, "run", compiled)
    import torch
    build.build_binding()
    build.build_binding()
    assert len(built) == 1
    monkeypatch.setattr(torch, "__version__", "9.9.9+cu999")
    build.build_binding()
    build.build_binding()
    assert len(built) == 2
    os.remove(build.BINDING + ".for")  # one that does not say
    build.build_binding()
    assert len(built) == 3


def test_a_binding_of_another_torch_is_not_loaded(monkeypatch, tmp_path):
    import torch

    from paged_kv_cache_193_gb300 import _lib
    path = tmp_path / "_pa_binding.so"
    path.write_bytes(b"not a module: reading it would fail differently")
    (tmp_path / "_pa_binding.so.for").write_text(build.binding_for(torch).replace(torch.__version__, "1.0"))
    monkeypatch.setattr(_lib, "_binding", None)
    monkeypatch.setattr(_lib, "BINDING_PATH", str(path))
    with pytest.raises(ImportError, match="torch 1.0.*build"):
        _lib.binding()
