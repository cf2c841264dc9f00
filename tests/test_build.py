"""What the build step makes, with stand-ins for the compilers: the C library
does not depend on the Python binding, and each is rebuilt when what it is made
from has changed."""
import os
import sys

import pytest

import sigmoid_attention_b200 as sa
from sigmoid_attention_b200 import build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """Paths of a build in an empty folder, and compilers that note each call
    and create what they are asked for (g++ fails while `broken` exists)."""
    log, broken = tmp_path / "log", tmp_path / "broken"
    script = f"""#!{sys.executable}
import os, sys
name = os.path.basename(sys.argv[0])
open({str(log)!r}, "a").write(name + "\\n")
if name == "g++" and os.path.exists({str(broken)!r}):
    sys.exit("no headers")
open(sys.argv[sys.argv.index("-o") + 1], "w").close()
"""
    for name in ("nvcc", "g++"):
        (tmp_path / name).write_text(script)
        (tmp_path / name).chmod(0o755)
    monkeypatch.setenv("PATH", f"{tmp_path}{os.pathsep}{os.environ['PATH']}")
    monkeypatch.setattr(build, "_nvcc", lambda: str(tmp_path / "nvcc"))
    for name, file in (("BUILD", "objects"), ("LIB", "libsigattn.so"), ("BINDING", "_binding.so")):
        monkeypatch.setattr(build, name, str(tmp_path / file))

    def calls():
        names = log.read_text().split() if log.exists() else []
        log.unlink(missing_ok=True)
        return names.count("nvcc"), names.count("g++")

    return tmp_path, broken, calls


def test_library_without_a_binding(tree):
    folder, broken, calls = tree
    broken.touch()
    with pytest.raises(RuntimeError, match="binding"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)
    calls()
    broken.unlink()
    assert build.build() == build.LIB and os.path.exists(build.BINDING)
    assert calls() == (0, 2)  # the library was there
    build.build()
    assert calls() == (0, 0)
    build.build(force=True)
    assert calls() == (len(build.SOURCES) + 1, 2)


def test_binding_follows_python_and_torch(tree, monkeypatch):
    folder, broken, calls = tree
    build.build()
    calls()
    monkeypatch.setattr(build.torch, "__version__", "0.0")
    build.build()
    assert calls() == (0, 2)
    build.build()
    assert calls() == (0, 0)


def test_message_of_a_binding_that_does_not_load(monkeypatch):
    monkeypatch.setattr(sa, "_calls", None)
    monkeypatch.delattr(sa, "_binding", raising=False)
    monkeypatch.setitem(sys.modules, "sigmoid_attention_b200._binding", None)
    with pytest.raises(RuntimeError, match="another Python or torch"):
        sa._paged()
