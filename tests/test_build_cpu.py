"""The build without torch, and with a binding that does not compile: the library is still made."""
import os

import pytest

from precision_tensor_core_gb300 import build as b


@pytest.fixture
def fake(tmp_path, monkeypatch):
    """The build with its compilers replaced by something that writes the named files."""
    made = []

    def compiled(src):
        made.append(src)
        obj = tmp_path / (src + ".o")
        obj.write_text("")
        return str(obj), ""

    def run(cmd, **kw):
        class Done:
            returncode, stdout, stderr = 0, "", ""
        out = cmd[cmd.index("-o") + 1]
        made.append(os.path.basename(out).split(".tmp")[0])
        open(out, "w").close()
        return Done()

    monkeypatch.setattr(b, "BUILD", str(tmp_path / "build"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libptc.so"))
    monkeypatch.setattr(b, "NATIVE", str(tmp_path / "_native.so"))
    monkeypatch.setattr(b, "_compile", compiled)
    monkeypatch.setattr(b.subprocess, "run", run)
    return made


def test_without_torch_the_library_is_built_alone(fake, monkeypatch):
    import importlib.util
    real = importlib.util.find_spec
    monkeypatch.setattr(importlib.util, "find_spec", lambda n, *a: None if n == "torch" else real(n, *a))
    assert b.build() == b.LIB and os.path.exists(b.LIB) and not os.path.exists(b.NATIVE)
    assert "_native.so" not in fake and "libptc.so" in fake
    n = len(fake)
    b.build()  # up to date
    assert len(fake) == n


def test_with_torch_both_are_built(fake):
    b.build()
    assert os.path.exists(b.LIB) and os.path.exists(b.NATIVE)
    os.remove(b.NATIVE)
    n = len(fake)
    b.build()
    assert len(fake) > n and os.path.exists(b.NATIVE)


def test_a_binding_that_does_not_compile_is_reported_after_the_library(fake, monkeypatch):
    def broken(*a):
        raise RuntimeError("g++ failed for binding.cpp")

    monkeypatch.setattr(b, "_compile_binding", broken)
    with pytest.raises(RuntimeError, match="binding.cpp"):
        b.build()
    assert os.path.exists(b.LIB)
