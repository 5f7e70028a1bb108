"""The library is built with hipcc alone: a host compiler that is missing, or a binding that
does not compile, costs the binding and nothing else.  Built in a folder of its own from
one source."""
import os
import shutil

import pytest

from w6a6_w6a8_integer_amd import build as b

pytestmark = pytest.mark.skipif(shutil.which(b.HIPCC) is None, reason="hipcc is not there")


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    monkeypatch.setattr(b, "SOURCES", ["pack_quant.hip"])
    monkeypatch.setattr(b, "BUILD_DIR", str(tmp_path / "objects"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libflexq.so"))
    monkeypatch.setattr(b, "BINDING", str(tmp_path / "_serve.so"))
    (tmp_path / "_serve.so").write_bytes(b"of an older library")
    return tmp_path


def test_no_host_compiler(elsewhere, monkeypatch, capfd):
    monkeypatch.setenv("CXX", str(elsewhere / "no-such-compiler"))
    assert b.build() == str(elsewhere / "libflexq.so")
    assert os.path.getsize(elsewhere / "libflexq.so") > 0
    assert not os.path.exists(elsewhere / "_serve.so")
    assert "_serve.so is not built" in capfd.readouterr().err


def test_binding_that_does_not_compile(elsewhere, monkeypatch):
    monkeypatch.setenv("CXX", shutil.which("false"))
    with pytest.raises(RuntimeError, match="serve_binding"):
        b.build()
    assert os.path.getsize(elsewhere / "libflexq.so") > 0
    assert not os.path.exists(elsewhere / "_serve.so")
