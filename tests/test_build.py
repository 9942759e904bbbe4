"""What the build needs: hipcc for the library, and torch only for the Python binding."""
import os
import shutil
import sys

import pytest

from dual_scale_w4a4_amd import build


@pytest.fixture
def commands(monkeypatch, tmp_path):
    """build() with its paths in a folder of the test's, and its commands recorded, not run."""
    ran = []

    def run(cmd, verbose):
        ran.append(cmd)
        out = cmd[cmd.index("-o") + 1]
        assert out.startswith(str(tmp_path)), out
        open(out, "w").close()

    monkeypatch.setattr(build, "_run", run)
    monkeypatch.setattr(build, "LIB_PATH", str(tmp_path / "libdq.so"))
    monkeypatch.setattr(build, "BIND_PATH", str(tmp_path / "_bind.so"))
    monkeypatch.setattr(build, "HERE", str(tmp_path))
    return ran


def test_the_library_is_built_without_torch(commands, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)  # what an import of it meets is an ImportError
    open(build.BIND_PATH, "w").close()
    assert build.build() == build.LIB_PATH and os.path.exists(build.LIB_PATH)
    assert not os.path.exists(build.BIND_PATH)  # one built for an older library does not stay
    assert all(os.path.basename(c[0]) == "hipcc" for c in commands)


def test_the_binding_is_built_with_torch(commands):
    assert build.build() == build.LIB_PATH
    assert os.path.exists(build.LIB_PATH) and os.path.exists(build.BIND_PATH)


def test_the_binding_needs_no_compiler_but_hipccs(commands, monkeypatch):
    monkeypatch.delenv("CXX", raising=False)
    monkeypatch.setattr(shutil, "which", lambda name: None if name == "g++" else name)
    build.build()
    bind = [c for c in commands if c[-1].startswith("-Wl,-rpath")]
    assert len(bind) == 1 and os.path.exists(bind[0][0]), bind[0][0]
