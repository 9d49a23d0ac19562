"""What the build compiles, with the compilers replaced by a recorder (no GPU)."""
import os
import sys

import pytest

from tiled_memory_efficient_gb300 import build


class Recorder:
    """Stands in for subprocess: notes the sources and leaves empty outputs, but for `fails`."""
    STDOUT = None

    def __init__(self):
        self.ran, self.fails = [], set()

    def check_call(self, cmd, **_):
        src = [os.path.basename(a) for a in cmd if a.endswith((".cu", ".cpp"))]
        self.ran += src or ["link"]
        if not self.fails.intersection(src):
            open(cmd[cmd.index("-o") + 1], "w").close()
        return cmd[cmd.index("-o") + 1]

    def Popen(self, cmd, **_):
        out = self.check_call(cmd)

        class Done:
            wait = staticmethod(lambda: 0 if os.path.exists(out) else 1)
        return Done


@pytest.fixture
def compilers(monkeypatch, tmp_path):
    monkeypatch.setattr(build, "BUILD", str(tmp_path))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "libattn.so"))
    monkeypatch.setattr(build, "BIND", str(tmp_path / "_bind.so"))
    rec = Recorder()
    monkeypatch.setattr(build, "subprocess", rec)
    return rec


def test_the_library_needs_no_torch(compilers, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)      # as where it is not installed
    assert build.build() == build.LIB and os.path.exists(build.LIB)
    assert sorted(compilers.ran) == sorted(build.SOURCES + ["link"])
    compilers.ran.clear()
    build.build()
    assert compilers.ran == []                           # up to date


def test_both_are_built_and_kept(compilers):
    build.build()
    assert sorted(compilers.ran) == sorted(build.SOURCES + ["link", "bind.cpp"])
    assert os.path.exists(build.LIB) and os.path.exists(build.BIND)
    compilers.ran.clear()
    build.build()
    assert compilers.ran == []
    os.remove(build.BIND)
    build.build()
    assert compilers.ran == ["bind.cpp"]                 # the library is up to date
    compilers.ran.clear()
    build.build(force=True)
    assert sorted(compilers.ran) == sorted(build.SOURCES + ["link", "bind.cpp"])


def test_a_binding_that_does_not_compile_leaves_the_library(compilers):
    compilers.fails.add("bind.cpp")
    with pytest.raises(RuntimeError, match="bind.cpp"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.BIND)


def test_a_kernel_that_does_not_compile_is_named(compilers):
    compilers.fails.add("kvp.cu")
    with pytest.raises(RuntimeError, match="kvp.cu"):
        build.build()
    assert not os.path.exists(build.LIB)
