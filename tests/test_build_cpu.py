"""What the build needs: the library nvcc alone, the Python module PyTorch and both headers too."""
import os
import subprocess
import sys

import pytest

from causal_sliding_window_rope_b200 import build as cs_build


@pytest.fixture
def compiler(monkeypatch, tmp_path):
    """Files of nobody's, and compilers that only write their output."""
    made = []

    def check_call(cmd, **kw):
        made.append(os.path.basename(cmd[cmd.index("-o") + 1]).split(".")[0])
        open(cmd[cmd.index("-o") + 1], "wb").close()
    monkeypatch.setattr(cs_build, "LIB", str(tmp_path / "libcswattn.so"))
    monkeypatch.setattr(cs_build, "LIB_BINDING", str(tmp_path / "_paged_binding.so"))
    monkeypatch.setattr(subprocess, "check_call", check_call)
    return made


def test_the_library_builds_without_pytorch(compiler, monkeypatch, capsys):
    monkeypatch.setitem(sys.modules, "torch", None)  # import torch raises, as where it is not installed
    assert cs_build.build() == cs_build.LIB
    assert compiler == ["libcswattn"] and os.path.exists(cs_build.LIB)
    assert "PyTorch" in capsys.readouterr().err  # said, not passed over


def test_the_library_builds_without_pythons_headers(compiler, monkeypatch, tmp_path):
    import sysconfig
    monkeypatch.setattr(sysconfig, "get_paths", lambda *a, **k: {"include": str(tmp_path)})
    cs_build.build()
    assert compiler == ["libcswattn"]


def test_both_are_built(compiler):
    cs_build.build()
    assert sorted(compiler) == ["_paged_binding", "libcswattn"]
    compiler.clear()
    with pytest.raises(subprocess.CalledProcessError):  # a compiler that fails is an error
        with pytest.MonkeyPatch.context() as m:
            def fail(cmd, **kw):
                raise subprocess.CalledProcessError(1, cmd)
            m.setattr(subprocess, "check_call", fail)
            cs_build.build_binding(force=True)
