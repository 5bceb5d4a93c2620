"""Building the marshalling extension: a user of libdg.so alone needs neither g++ nor torch's headers (no GPU needed)."""
import importlib.metadata
import os
import shutil
import subprocess
import sys
import sysconfig

import pytest

from moe_grouped_gemm_weight_b200 import build as dgbuild


@pytest.fixture
def runs(monkeypatch, tmp_path):
    """Commands that build() runs, none of them in earnest; the extension lies in an empty directory."""
    done = []

    def run(cmd, check):
        done.append(cmd)
        out = cmd[cmd.index("-o") + 1]
        open(out, "w").close()
        return subprocess.CompletedProcess(cmd, 0)

    monkeypatch.setattr(dgbuild.subprocess, "run", run)
    monkeypatch.setattr(dgbuild, "up_to_date", lambda: True)
    monkeypatch.setattr(dgbuild, "CALL_LIB", str(tmp_path / "_dgcall.so"))
    return done


def test_the_library_builds_without_a_cxx_compiler(runs, monkeypatch, capsys):
    which = shutil.which
    monkeypatch.setattr(shutil, "which", lambda name, *a, **k: None if name == "g++" else which(name, *a, **k))
    assert dgbuild.build() == dgbuild.LIB
    assert runs == [] and "g++" in capsys.readouterr().err


def test_the_library_builds_without_torch():
    code = """
import sys, shutil, subprocess
sys.modules["torch"] = None
from moe_grouped_gemm_weight_b200 import build
build.CALL_LIB = "/nonexistent/_dgcall.so"
build.up_to_date = lambda: True
assert build.build() == build.LIB
"""
    out = subprocess.run([sys.executable, "-c", code], cwd=os.path.dirname(dgbuild.HERE), capture_output=True, text=True)
    assert out.returncode == 0 and "torch" in out.stderr, out.stderr


def test_an_extension_that_does_not_compile_is_an_error(runs, monkeypatch):
    def run(cmd, check):
        raise subprocess.CalledProcessError(1, cmd)

    monkeypatch.setattr(dgbuild.subprocess, "run", run)
    with pytest.raises(subprocess.CalledProcessError):
        dgbuild.build()


def test_a_current_extension_is_left_alone(runs):
    dgbuild.build()
    assert len(runs) == 1 and "g++" in runs[0][0]
    dgbuild.build()
    assert len(runs) == 1


def test_an_extension_of_another_torch_or_python_is_built_again(runs, monkeypatch):
    dgbuild.build()
    assert len(runs) == 1
    monkeypatch.setattr(importlib.metadata, "version", lambda name: "0.0.0+other")
    dgbuild.build()
    assert len(runs) == 2
    dgbuild.build()
    assert len(runs) == 2
    monkeypatch.setattr(sysconfig, "get_config_var", lambda name: "cpython-399")
    dgbuild.build()
    assert len(runs) == 3


def test_an_extension_that_does_not_load_is_not_called_missing(monkeypatch):
    import moe_grouped_gemm_weight_b200 as dg
    dgbuild.build()
    assert os.path.exists(dgbuild.CALL_LIB)
    monkeypatch.setattr(dg, "_calls", None)
    monkeypatch.setitem(sys.modules, dg.__name__ + "._dgcall", None)
    monkeypatch.delattr(dg, "_dgcall", raising=False)
    with pytest.raises(RuntimeError, match="_dgcall.so.*does not load") as ei:
        dg._marshal()
    assert "missing" not in str(ei.value) and isinstance(ei.value.__cause__, ImportError)
