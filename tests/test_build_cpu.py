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


def test_another_pytorch_makes_the_module_stale(monkeypatch):
    """The module is compiled for one PyTorch and one Python, and says which."""
    cs_build.build_binding()
    assert not cs_build.stale(cs_build.LIB_BINDING)
    with pytest.MonkeyPatch.context() as m:
        m.setattr(cs_build, "torch_version", lambda: "1.2.3+other", raising=False)
        assert cs_build.stale(cs_build.LIB_BINDING)
    with pytest.MonkeyPatch.context() as m:
        m.setattr(sys, "version_info", (3, 99, 0, "final", 0))
        assert cs_build.stale(cs_build.LIB_BINDING)


def test_a_module_for_another_pytorch_is_refused(monkeypatch):
    import torch

    import causal_sliding_window_rope_b200 as cs
    cs_build.build()
    monkeypatch.setattr(cs, "_paged", None)
    cs._paged_calls()
    monkeypatch.setattr(cs, "_paged", None)
    monkeypatch.setattr(torch, "__version__", "1.2.3+other")
    with pytest.raises(RuntimeError, match="1.2.3"):
        cs._paged_calls()
