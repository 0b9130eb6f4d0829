"""What is built again when, in a folder of small sources (CPU)."""
import os

import pytest

from trellis_quantized_moe_exl3_gb300 import _lib, build


@pytest.fixture
def tree(tmp_path, monkeypatch):
    src, out = tmp_path / "csrc", tmp_path / "_build"
    src.mkdir()
    (src / "a.cu").write_text('extern "C" int exl3_a() { return 3; }\n')
    (src / "binding.cpp").write_text('extern "C" int exl3_a();\nextern "C" int b() { return exl3_a(); }\n')
    monkeypatch.setattr(build, "CSRC", str(src))
    monkeypatch.setattr(build, "OUT_DIR", str(out))
    monkeypatch.setattr(build, "LIB_PATH", str(out / "libexl3_gb300.so"))
    monkeypatch.setattr(build, "NATIVE_PATH", str(out / "_native.so"))
    return src


def times():
    return [os.stat(p).st_mtime_ns for p in (build.LIB_PATH, build.NATIVE_PATH)]


def test_the_binding_is_rebuilt_for_another_torch_or_python(tree, monkeypatch):
    assert build.built_stamp() is None
    build.build()
    assert build.built_stamp() == build.native_stamp()
    first = times()
    build.build()
    assert times() == first
    real = build.native_stamp()
    monkeypatch.setattr(build, "native_stamp", lambda: "torch 99.0")
    build.build()
    second = times()
    assert second[0] == first[0] and second[1] > first[1] and build.built_stamp() == "torch 99.0"
    assert real != "torch 99.0"


def test_a_binding_of_another_torch_is_not_loaded(tree, monkeypatch):
    build.build()
    monkeypatch.setattr(_lib, "_native", None)
    monkeypatch.setattr(_lib, "NATIVE_PATH", build.NATIVE_PATH)
    monkeypatch.setattr(_lib, "native_stamp", lambda: "torch 99.0")
    monkeypatch.setattr(_lib, "lib", lambda: None)
    with pytest.raises(ImportError, match="torch 99.0.*build it again"):
        _lib.native()


def test_the_library_is_built_where_the_binding_fails(tree):
    (tree / "binding.cpp").write_text("#include <no_such_header.h>\n")
    with pytest.raises(RuntimeError, match=r"^g\+\+ failed"):
        build.build()
    assert os.path.exists(build.LIB_PATH) and not os.path.exists(build.NATIVE_PATH)
    (tree / "binding.cpp").write_text("int x;\n")
    build.build()
    assert os.path.exists(build.NATIVE_PATH) and build.built_stamp() == build.native_stamp()
    (tree / "a.cu").write_text("no\n")
    with pytest.raises(RuntimeError, match="^nvcc failed"):
        build.build()
