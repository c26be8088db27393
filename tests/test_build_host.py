"""What build.py makes, and when it makes it again, with the compilers replaced by a function that writes their outputs."""
import os
import subprocess
import sys
import types

import pytest

pytest.importorskip("torch")

from decoder_only_transformer_gpt_gb300 import build  # noqa: E402


@pytest.fixture
def tools(monkeypatch, tmp_path):
    """Commands run so far; those that contain a word of `fail` fail."""
    t = types.SimpleNamespace(commands=[], fail=())

    def run(cmd, **_):
        t.commands.append(cmd)
        bad = any(w in " ".join(cmd) for w in t.fail)
        if not bad:
            with open(cmd[cmd.index("-o") + 1], "w") as f:
                f.write("x")
        return subprocess.CompletedProcess(cmd, int(bad), "", "failed" if bad else "")
    monkeypatch.setattr(build.subprocess, "run", run)
    monkeypatch.setattr(build, "nvcc", lambda: "/usr/local/cuda/bin/nvcc")
    for name in ("BUILD", "LIB", "CALLS", "CALLS_FOR"):
        if hasattr(build, name):
            monkeypatch.setattr(build, name, str(tmp_path / os.path.basename(getattr(build, name))))
    return t


def test_everything_and_then_nothing(tools):
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and os.path.exists(build.CALLS) and build.up_to_date()
    n = len(tools.commands)
    build.build()
    assert len(tools.commands) == n


def test_the_library_needs_no_torch(tools, monkeypatch, capfd):
    with monkeypatch.context() as m:
        m.setitem(sys.modules, "torch", None)        # `import torch` raises, and there is none to be found
        assert build.build() == build.LIB
        assert os.path.exists(build.LIB) and not os.path.exists(build.CALLS) and build.up_to_date()
        assert "_calls" in capfd.readouterr().err
    assert not build.up_to_date()                    # with a torch the module is wanted


@pytest.mark.parametrize("word", ["py_calls.cpp", "-ltorch_python"])
def test_a_module_that_fails_leaves_the_library(tools, word):
    tools.fail = (word,)
    with pytest.raises(RuntimeError, match="_calls"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.CALLS) and not build.up_to_date()


def test_another_torch_or_python_makes_the_module_anew(tools, monkeypatch):
    build.build()
    for what, value in (("metadata.version", "9.9"), ("soabi", "cpython-399")):
        with monkeypatch.context() as m:
            if what == "soabi":
                m.setattr(build.sysconfig, "get_config_var", lambda _: value)
            else:
                m.setattr(build.importlib.metadata, "version", lambda _: value)
            assert not build.up_to_date()
            tools.commands.clear()
            build.build()
            assert len(tools.commands) == 2 and not any("nvcc" in c[0] for c in tools.commands)   # the module alone
            assert build.up_to_date()
        assert not build.up_to_date()
        build.build()
