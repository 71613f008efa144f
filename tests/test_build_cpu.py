"""Which compiled files the binding takes: only ones made from the sources that
are there, against the torch and the interpreter that run; with stand-ins for
the compilers."""
import os
import subprocess
import threading
import time

import pytest
import torch

import w8a8_post_quantization_channel_b200 as sq
from w8a8_post_quantization_channel_b200 import build


class Compilers:
    """Stands in for subprocess.run: fails, or copies the true binary; counts calls."""

    def __init__(self, result=None):
        self.result, self.calls, self.inside, self.most = result, 0, 0, 0

    def __call__(self, cmd, **kw):
        self.calls += 1
        self.inside += 1
        self.most = max(self.most, self.inside)
        time.sleep(0.05)
        self.inside -= 1
        if self.result is None:
            return subprocess.CompletedProcess(cmd, 1, "", "no compiler here")
        with open(cmd[cmd.index("-o") + 1], "wb") as f:
            f.write(self.result)
        return subprocess.CompletedProcess(cmd, 0, "", "")


@pytest.fixture
def binding(tmp_path, monkeypatch):
    """A copy of the binding's binary and source; the compilers fail."""
    sq._marshal()  # built where it was not
    with open(build.BINDING, "rb") as f:
        binary = f.read()
    (tmp_path / "_binding.so").write_bytes(binary)
    with open(build.BINDING_SRC) as f:
        (tmp_path / "sq_binding.cpp").write_text(f.read())
    os.utime(tmp_path / "sq_binding.cpp", (2, 2))  # older than the binary
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "_binding.so"))
    monkeypatch.setattr(build, "BINDING_SRC", str(tmp_path / "sq_binding.cpp"))
    run = Compilers()
    monkeypatch.setattr(build.subprocess, "run", run)
    return tmp_path, run, binary


def test_the_binary_that_fits_is_taken_whatever_the_file_times(binding):
    path, run, _ = binding
    os.utime(path / "_binding.so", (1, 1))
    assert build.build_binding() == str(path / "_binding.so") and run.calls == 0


def test_another_source_is_not_taken(binding):
    path, run, _ = binding
    with open(path / "sq_binding.cpp", "a") as f:
        f.write("// changed\n")
    os.utime(path / "sq_binding.cpp", (2, 2))
    with pytest.raises(RuntimeError):
        build.build_binding()
    assert run.calls == 1


@pytest.mark.parametrize("what", ["version", "abi", "interpreter"])
def test_a_binary_for_another_torch_or_interpreter_is_not_taken(binding, monkeypatch, what):
    import sysconfig
    _, run, _ = binding
    if what == "version":
        monkeypatch.setattr(torch, "__version__", "0.0.1")
    elif what == "abi":
        abi = torch.compiled_with_cxx11_abi()
        monkeypatch.setattr(torch, "compiled_with_cxx11_abi", lambda: not abi)
    else:
        real = sysconfig.get_config_var
        monkeypatch.setattr(sysconfig, "get_config_var", lambda n: "cpython-30" if n == "SOABI" else real(n))
    with pytest.raises(RuntimeError):
        build.build_binding()
    assert run.calls == 1


def test_no_fallback_to_a_binding_that_does_not_fit(binding, monkeypatch):
    path, _, _ = binding
    with open(path / "sq_binding.cpp", "a") as f:
        f.write("// changed\n")
    os.utime(path / "sq_binding.cpp")
    monkeypatch.setattr(sq, "_native", None)
    with pytest.raises(RuntimeError):
        sq._marshal()
    assert sq._native is None


def test_builds_take_turns(binding):
    path, _, binary = binding
    run = Compilers(binary)
    build.subprocess.run = run  # (put back with the fixture's)
    threads = [threading.Thread(target=build.build_binding, args=(True,)) for _ in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert run.calls == 4 and run.most == 1
    assert sorted(p.name for p in path.iterdir()) == ["_binding.so", "sq_binding.cpp"]
    with open(path / "_binding.so", "rb") as f:
        assert f.read() == binary


def test_the_library_is_held_to_its_sources_too(tmp_path, monkeypatch):
    sq.lib()
    monkeypatch.setattr(build.subprocess, "run", Compilers())
    os.utime(build.LIB, (1, 1))
    try:
        assert build.build() == build.LIB  # the file's time does not count
    finally:
        os.utime(build.LIB)
    more = tmp_path / "more.h"
    more.write_text("// one more source\n")
    sources = build._sources()
    monkeypatch.setattr(build, "_sources", lambda: sources + [str(more)])
    with pytest.raises(RuntimeError):
        build.build()
    monkeypatch.setattr(sq, "_lib", None)
    with pytest.raises(RuntimeError):
        sq.lib()


def test_a_tree_without_sources_uses_what_it_has(binding, monkeypatch):
    path, run, _ = binding
    (path / "sq_binding.cpp").unlink()
    monkeypatch.setattr(build, "_sources", lambda: [])
    assert build.build_binding() == str(path / "_binding.so")
    assert build.build() == build.LIB and run.calls == 0
