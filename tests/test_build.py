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
    assert os.path.exists(b.calls_path())
    assert b.calls_path().endswith(b.sysconfig.get_config_var("EXT_SUFFIX")) and torch.__version__[:4] in b.calls_path()
    monkeypatch.setattr(torch, "__version__", "1.0.0+other")
    assert not os.path.exists(b.calls_path())
    compiled = []
    monkeypatch.setattr(b, "_compile_calls", lambda: compiled.append(b.calls_path()))
    b.build()
    assert compiled == [b.calls_path()]
    monkeypatch.setattr(_lib, "_calls", None)
    with pytest.raises(ImportError, match="PyTorch"):
        _lib.calls()


@pytest.fixture
def fake(monkeypatch, tmp_path):
    """The build module with nothing built and nothing that really compiles; the steps it takes, in a list."""
    import importlib
    b = importlib.import_module("task_graph_interpreter_gb300.build")
    steps = []
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libmk.so"))
    monkeypatch.setattr(b, "BUILD", str(tmp_path / "build"))
    monkeypatch.setattr(b, "calls_path", lambda: str(tmp_path / "calls.so"))
    monkeypatch.setattr(b, "_compile", lambda src, verbose: os.path.basename(src))

    def link(objs):
        assert objs == [os.path.basename(s) for s in b.SOURCES]
        steps.append("link")
        open(b.LIB, "w").close()

    def calls():
        steps.append("calls")
        open(b.calls_path(), "w").close()
    monkeypatch.setattr(b, "_link", link)
    monkeypatch.setattr(b, "_compile_calls", calls)
    return b, steps


def test_each_library_is_built_when_it_is_out_of_date(fake):
    b, steps = fake
    b.build()
    assert sorted(steps) == ["calls", "link"]
    b.build()
    assert len(steps) == 2
    os.unlink(b.calls_path())
    b.build()
    os.unlink(b.LIB)
    b.build()
    assert steps[2:] == ["calls", "link"]
    os.utime(b.calls_path(), (0, 0))
    b.build()
    assert steps[4:] == ["calls"]
    b.build(force=True)
    assert len(steps) == 7


def test_the_library_is_linked_although_the_calls_do_not_compile(fake, monkeypatch):
    b, steps = fake

    def fails():
        raise RuntimeError("no C++ compiler found")
    monkeypatch.setattr(b, "_compile_calls", fails)
    with pytest.raises(RuntimeError, match="compiler"):
        b.build()
    assert steps == ["link"] and os.path.exists(b.LIB)


def test_the_library_is_built_without_torch(fake, monkeypatch):
    b, steps = fake

    def missing():
        raise ImportError("No module named 'torch'")
    monkeypatch.setattr(b, "calls_path", missing)
    assert b.build() == b.LIB and b.build() == b.LIB
    assert steps == ["link"]
    b.build(force=True)
    assert steps == ["link", "link"]


LOG = """ptxas info    : Compiling entry function '_ZN2mk_12chunk_kernelILi64EEEvNS' for 'sm_103a'
ptxas info    : Function properties for _ZN2mk_12chunk_kernelILi64EEEvNS
    128 bytes stack frame, 0 bytes spill stores, 0 bytes spill loads
ptxas info    : Used %d registers, used 1 barriers, 128 bytes cumulative stack size
ptxas info    : Compiling entry function '_ZN2mk_12chunk_kernelILi128EEEvNS' for 'sm_103a'
ptxas info    : Used %d registers, used 1 barriers
ptxas info    : Compiling entry function '_ZN2mk_other' for 'sm_103a'
ptxas info    : Used 40 registers, used 1 barriers
"""


def test_the_chunk_kernel_has_to_be_compiled_to_the_registers_of_its_launch():
    import importlib
    b = importlib.import_module("task_graph_interpreter_gb300.build")
    with open(os.path.join(b.OPS, "paged_chunk.cu")) as f:
        source = f.read()
    b.check_launch_registers(source, LOG % (168, 168))
    for log in (LOG % (166, 168), LOG % (168, 128), LOG.split("ptxas info    : Compiling entry function '_ZN2mk_other")[1], ""):
        with pytest.raises(RuntimeError, match="168 registers"):
            b.check_launch_registers(source, log)
