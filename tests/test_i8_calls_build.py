"""The marshalling module of the 8-bit calls belongs to one interpreter."""
import importlib.machinery
import importlib.util
import os
import sysconfig

import pytest

TAGGED = "_i8_calls" + importlib.machinery.EXTENSION_SUFFIXES[0]


@pytest.fixture
def build(monkeypatch, tmp_path):
    """The build's module with its output in a directory of its own."""
    from dense_gemm_09_gb300 import _build
    monkeypatch.setattr(_build, "PKG", str(tmp_path))
    monkeypatch.setattr(_build, "CALLS", str(tmp_path / os.path.basename(_build.CALLS)))
    return _build


def test_the_name_carries_the_interpreters_tag(build, tmp_path):
    assert TAGGED != "_i8_calls.so" and sysconfig.get_config_var("SOABI") in TAGGED
    assert os.path.basename(build.build_calls()) == TAGGED
    assert [f.name for f in tmp_path.iterdir()] == [TAGGED]


def test_a_file_without_a_tag_is_removed(build, tmp_path):
    (tmp_path / "_i8_calls.so").write_bytes(b"of some interpreter")
    build.build_calls()
    assert [f.name for f in tmp_path.iterdir()] == [TAGGED]


def test_no_headers(build, tmp_path, monkeypatch, capfd):
    monkeypatch.setattr(sysconfig, "get_paths", lambda: {"include": str(tmp_path / "nowhere")})
    assert build.build_calls(force=True) is None
    assert "Python.h" in capfd.readouterr().err
    assert not (tmp_path / TAGGED).exists()


def test_a_file_without_a_tag_is_not_loaded(monkeypatch):
    import dense_gemm_09_gb300 as dg
    path = os.path.join(os.path.dirname(dg.__file__), "_i8_calls.so")
    spec = importlib.machinery.ModuleSpec("dense_gemm_09_gb300._i8_calls", None, origin=path)
    monkeypatch.setattr(dg, "_calls_module", None)
    monkeypatch.setattr(importlib.util, "find_spec", lambda *a: spec)
    with pytest.raises(RuntimeError, match="another interpreter"):
        dg.quantize_i8(None, None, None)
