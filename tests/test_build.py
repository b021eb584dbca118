"""The build module: its two spellings, and what it builds when (no GPU; nothing is compiled here)."""
import os
import subprocess
import sys

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.mark.parametrize("code", [
    "import task_graph_interpreter_gb300 as p; f = p.build; import task_graph_interpreter_gb300.build as b; g = b.build",
    "import task_graph_interpreter_gb300.build as b; g = b.build; from task_graph_interpreter_gb300 import build as f",
    "from task_graph_interpreter_gb300.build import build as g; from task_graph_interpreter_gb300 import build as f",
    "from task_graph_interpreter_gb300 import build as f; import task_graph_interpreter_gb300 as p; g = p.build.build"])
def test_the_package_has_its_build_under_both_spellings(code):
    """As a function of the package and as the module with the function, whichever is imported first."""
    code += "; assert f() == g() == f(force=False, verbose=False) and f().endswith('libmk.so')"
    r = subprocess.run([sys.executable, "-c", code], cwd=ROOT, capture_output=True, text=True)
    assert r.returncode == 0, r.stderr


def test_the_build_runs_as_a_program_without_a_warning():
    r = subprocess.run([sys.executable, "-m", "task_graph_interpreter_gb300.build"], cwd=ROOT, capture_output=True,
                       text=True)
    assert r.returncode == 0 and r.stdout.strip().endswith("libmk.so") and "Warning" not in r.stderr, r.stderr


def test_the_package_has_no_other_attributes():
    import task_graph_interpreter_gb300 as p
    with pytest.raises(AttributeError):
        p.no_such_name


def test_the_calls_module_belongs_to_one_python_and_one_torch(monkeypatch):
    """A module that was compiled against another PyTorch is neither taken for up to date nor loaded."""
    import torch

    from task_graph_interpreter_gb300 import _lib
    from task_graph_interpreter_gb300 import build as b
    b.build()
    assert not b._stale() and os.path.exists(b.calls_path())
    assert b.calls_path().endswith(b.sysconfig.get_config_var("EXT_SUFFIX")) and torch.__version__[:4] in b.calls_path()
    monkeypatch.setattr(torch, "__version__", "1.0.0+other")
    assert b._stale() and not os.path.exists(b.calls_path())
    monkeypatch.setattr(_lib, "_calls", None)
    with pytest.raises(ImportError, match="PyTorch"):
        _lib.calls()
