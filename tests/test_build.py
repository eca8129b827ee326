"""The library and the compiled binding are built apart: where the binding does not compile against
the installed torch, the library (the INT8 layer, through ctypes) is built all the same, and what
needs the binding says that it is missing."""
import os

import pytest

from int8_weight_quantized_gb300 import build, transformer


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A small library of one source and a binding that cannot be compiled."""
    (tmp_path / "one.cu").write_text('extern "C" int one() { return 1; }\n')
    (tmp_path / "binding.cpp").write_text("#error no such torch\n")
    monkeypatch.setattr(build, "CSRC", str(tmp_path))
    monkeypatch.setattr(build, "SOURCES", ["one.cu"])
    monkeypatch.setattr(build, "HEADERS", [])
    monkeypatch.setattr(build, "OBJ_DIR", str(tmp_path / "_build"))
    monkeypatch.setattr(build, "LIB_DIR", str(tmp_path / "lib"))
    monkeypatch.setattr(build, "LIB", str(tmp_path / "lib" / "libone.so"))
    monkeypatch.setattr(build, "BINDING", str(tmp_path / "lib" / "_binding.so"))
    return tmp_path


def test_the_library_is_built_without_the_binding(tree, capsys):
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and not os.path.exists(build.BINDING)
    assert "no such torch" in capsys.readouterr().err
    made = os.path.getmtime(build.LIB)
    assert build.build() == build.LIB
    assert os.path.getmtime(build.LIB) == made  # only the binding is tried again


def test_a_binding_of_other_sources_does_not_stay(tree):
    os.makedirs(build.LIB_DIR)
    with open(build.BINDING, "w") as f:
        f.write("old")
    os.utime(build.BINDING, (1, 1))
    build.build()
    assert not os.path.exists(build.BINDING)


def test_a_build_that_needs_the_binding_fails(tree):
    with pytest.raises(RuntimeError, match="no such torch"):
        build.build(require_binding=True)
    assert os.path.exists(build.LIB)


def test_operators_say_that_the_binding_is_missing(tree, monkeypatch):
    monkeypatch.setattr(transformer, "_b", None)
    monkeypatch.setattr(transformer.ck, "load_library", lambda path=None: None)
    with pytest.raises(RuntimeError, match="is not built"):
        transformer.ck_attention(None, None, None, None)
