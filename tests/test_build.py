"""What build() makes, keeps and makes again, on stand-ins for the two compilers."""

import os
import sys

import pytest

from tiled_fp16_gemm_gb300 import build as b


def writes(path, text):
    return [sys.executable, "-c", f"open({path!r}, 'wb').write({text!r}.encode())"]


@pytest.fixture
def made(monkeypatch, tmp_path):
    """build.py on outputs of its own; returns the list of what was compiled."""
    ran = []
    monkeypatch.setattr(b, "LIB", str(tmp_path / "libtgemm.so"))
    monkeypatch.setattr(b, "CALLS", str(tmp_path / "_calls.so"))

    def nvcc(out, extra=None):
        ran.append("lib")
        return writes(out, "lib")

    def calls(out):
        ran.append("calls")
        return writes(out, "x" + b._mark(b._torch()) + "\0y")

    monkeypatch.setattr(b, "nvcc_command", nvcc)
    monkeypatch.setattr(b, "calls_command", calls)
    monkeypatch.setattr(b, "_torch", lambda: ("/nowhere", "2.9.1+cu130"))
    return ran


def test_both_are_built_once(made):
    assert not b.up_to_date()
    assert b.build() == b.LIB and sorted(made) == ["calls", "lib"]
    assert b.up_to_date()
    b.build()
    assert len(made) == 2
    b.build(force=True)
    assert len(made) == 4


def test_the_c_library_alone_without_pytorch(made, monkeypatch):
    monkeypatch.setattr(b, "_torch", lambda: None)
    b.build()
    assert made == ["lib"] and os.path.exists(b.LIB) and not os.path.exists(b.CALLS)
    assert b.up_to_date()


@pytest.mark.parametrize("command", [["false"], ["/nowhere/g++"]])
def test_the_c_library_is_kept_where_the_other_fails(made, monkeypatch, command):
    monkeypatch.setattr(b, "calls_command", lambda out: command)
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        b.build()
    assert os.path.exists(b.LIB) and not b.up_to_date()


def test_a_failing_nvcc_is_reported(made, monkeypatch):
    monkeypatch.setattr(b, "nvcc_command", lambda out, extra=None: ["false"])
    with pytest.raises(RuntimeError, match="nvcc failed"):
        b.build()
    assert not os.path.exists(b.LIB)


def test_another_pytorch(made, monkeypatch):
    b.build()
    monkeypatch.setattr(b, "_torch", lambda: ("/nowhere", "2.9.1+cu13"))
    assert not b.up_to_date()
    b.build()
    assert sorted(made) == ["calls", "calls", "lib"] and b.up_to_date()


def test_a_changed_source(made, monkeypatch, tmp_path):
    b.build()
    source = tmp_path / "new.cu"
    source.write_text("")
    later = os.path.getmtime(b.LIB) + 10
    os.utime(source, (later, later))
    monkeypatch.setattr(b, "sources", lambda: [str(source)])
    assert not b.up_to_date()


def test_the_pytorch_here():
    torch = pytest.importorskip("torch")
    if torch.version.cuda is None:
        assert b._torch() is None
        return
    where, version = b._torch()
    assert os.path.samefile(where, os.path.dirname(torch.__file__)) and version == torch.__version__
