"""When the build makes the compiled calls again, with the compilers replaced
by a record of what they were asked."""
import importlib.util
import os
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


@pytest.fixture
def made(tmp_path, monkeypatch):
    """The build script over an empty output folder and a torch of our own;
    made() runs it and returns the outputs it made."""
    spec = importlib.util.spec_from_file_location(
        "_build_of_the_calls", os.path.join(ROOT, "sequence_slot_kv_gb300", "build.py"))
    b = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(b)
    out, torch = tmp_path / "out", tmp_path / "torch"
    out.mkdir()
    headers = torch / "include" / "torch" / "csrc" / "autograd"
    headers.mkdir(parents=True)
    (headers / "python_variable.h").write_text("")
    (torch / "version.py").write_text("__version__ = '1'\n")
    (torch / "__init__.py").write_text("")
    inc = tmp_path / "python"
    inc.mkdir()
    (inc / "Python.h").write_text("")
    monkeypatch.setattr(b, "OBJDIR", str(out / "obj"))
    monkeypatch.setattr(b, "LIB", str(out / "lib.so"))
    monkeypatch.setattr(b, "CALL", str(out / "call.so"))
    real = importlib.util.find_spec
    monkeypatch.setattr(b.importlib.util, "find_spec", lambda name, *a: (
        importlib.util.spec_from_file_location("torch", torch / "__init__.py",
                                               submodule_search_locations=[str(torch)])
        if name == "torch" else real(name, *a)))
    monkeypatch.setattr(b.sysconfig, "get_paths", lambda: {"include": str(inc)})
    asked = []

    class Compiler:
        returncode = 0

        def __init__(self, cmd, **kw):
            asked.append(os.path.basename(cmd[cmd.index("-o") + 1]))
            open(cmd[cmd.index("-o") + 1], "w").close()

        def communicate(self):
            return "", None

    monkeypatch.setattr(b.subprocess, "Popen", Compiler)
    monkeypatch.setattr(b.subprocess, "run", lambda cmd, check=True: Compiler(cmd))

    def run(**kw):
        asked.clear()
        b.build(**kw)
        return list(asked)

    run.call, run.torch, run.headers, run.python = out / "call.so", torch, headers, inc
    assert subprocess.Popen is Compiler
    return run


def test_nothing_is_made_twice(made):
    assert "call.o" in made() and made.call.exists()
    assert made() == []


def test_another_torch(made):
    made()
    (made.torch / "version.py").write_text("__version__ = '2'\n")
    assert made() == ["call.o", "call.so"]
    assert made() == []


def test_another_python(made, monkeypatch):
    made()
    monkeypatch.setattr("sys.version", "another one")
    assert made() == ["call.o", "call.so"]
    assert made() == []


@pytest.mark.parametrize("gone", ["python", "headers"])
def test_without_headers_no_old_module_stays(made, gone):
    made()
    for f in getattr(made, gone).iterdir():
        f.unlink()
    assert made() == []
    assert not made.call.exists()


def test_force(made):
    made()
    assert {"call.o", "call.so", "lib.so"} < set(made(force=True))
