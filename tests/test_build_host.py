"""The build's own steps: what a failed compilation of the binding's native part leaves behind."""
import os

from paged_decode_attention_reshape_gb300 import _build


def test_no_older_binding_part_is_left(tmp_path, monkeypatch):
    """Where csrc/pa_marshal.cpp does not compile, the one of an earlier source is not loaded either."""
    for name in ("MARSHAL", "NO_MARSHAL"):
        monkeypatch.setattr(_build, name, str(tmp_path / name))
    monkeypatch.setenv("CXX", "false")
    (tmp_path / "MARSHAL").write_text("of an earlier source")
    _build._build_marshal()
    assert os.path.exists(_build.NO_MARSHAL) and not os.path.exists(_build.MARSHAL)


def test_a_compiler_that_is_not_there(tmp_path, monkeypatch):
    for name in ("MARSHAL", "NO_MARSHAL"):
        monkeypatch.setattr(_build, name, str(tmp_path / name))
    monkeypatch.setenv("CXX", str(tmp_path / "none"))
    _build._build_marshal()
    assert os.path.exists(_build.NO_MARSHAL)
