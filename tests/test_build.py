"""What build.build() compiles, and when: a small source in a folder of its own, with stand-ins for the binding's
compiler."""
import os
import time

import pytest
import torch


@pytest.fixture
def build(monkeypatch, tmp_path):
    from paged_kv_prefill_gb300 import build as b

    monkeypatch.setattr(b, "SOURCES", ["append.cu"])
    monkeypatch.setattr(b, "BUILD", str(tmp_path / "_build"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libb2pa.so"))
    monkeypatch.setattr(b, "NATIVE", str(tmp_path / "_native.so"))
    made = []

    def commands(tmp):
        made.append(tmp)
        return [["true"], ["cp", "/dev/null", tmp]]

    monkeypatch.setattr(b, "_native_commands", commands)
    b.made = made
    yield b
    del b.made


def test_the_library_does_not_need_the_binding(build, monkeypatch):
    """Without a compiler that takes native.cpp, or torch's headers, the C library is built all the same."""
    monkeypatch.setattr(build, "_native_commands", lambda tmp: [["false"], ["false"]])
    with pytest.raises(RuntimeError, match="native.cpp"):
        build.build()
    assert os.path.getsize(build.LIB) > 0 and not os.path.exists(build.NATIVE)

    def no_torch(tmp):
        raise ImportError("no torch here")

    monkeypatch.setattr(build, "_native_commands", no_torch)
    os.remove(build.LIB)
    with pytest.raises((RuntimeError, ImportError), match="no torch here"):
        build.build()
    assert os.path.getsize(build.LIB) > 0


def test_the_binding_follows_torch_and_python(build, monkeypatch):
    assert build.build() == build.LIB and len(build.made) == 1
    before = os.path.getmtime(build.LIB)
    build.build()
    assert len(build.made) == 1  # nothing has changed
    monkeypatch.setattr(torch, "__version__", "0.1")
    build.build()
    build.build()
    assert len(build.made) == 2
    monkeypatch.setattr(build.sys, "version", "9.9 (another)")
    build.build()
    build.build()
    assert len(build.made) == 3
    assert os.path.getmtime(build.LIB) == before  # the library is not concerned
    time.sleep(0.01)
    build.build(force=True)
    assert len(build.made) == 4 and os.path.getmtime(build.LIB) > before
