"""The build: libmla.so needs nvcc alone, the binding's compiled module also torch, whose version it
follows. On a small source in a folder of its own."""
import importlib.metadata
import os
import sys

import pytest


@pytest.fixture
def build(tmp_path, monkeypatch):
    from mla_latent_kv_44_b200 import build as b

    csrc = tmp_path / "csrc"
    csrc.mkdir()
    (csrc / "one.cu").write_text('extern "C" int one() { return 1; }\n')
    (csrc / "fast_call.cpp").write_text('extern "C" int two() { return 2; }\n')
    for name, value in (("CSRC", csrc), ("INCLUDE", csrc), ("BUILD", tmp_path / "_build"),
                        ("LIB", tmp_path / "lib.so"), ("TEST_LIB", tmp_path / "lib_test.so"),
                        ("FAST_SOURCE", csrc / "fast_call.cpp"), ("FAST_LIB", tmp_path / "fast.so")):
        monkeypatch.setattr(b, name, str(value))
    return b


def test_the_library_builds_where_torch_is_missing(build, monkeypatch, capfd):
    monkeypatch.setitem(sys.modules, "torch", None)
    monkeypatch.setitem(sys.modules, "torch.utils", None)
    assert build.build() == build.LIB
    assert os.path.exists(build.LIB) and os.path.exists(build.TEST_LIB)
    assert not os.path.exists(build.FAST_LIB)
    assert "torch" in capfd.readouterr().err


def test_the_library_is_linked_where_the_module_does_not_compile(build):
    with open(build.FAST_SOURCE, "w") as f:
        f.write("#error no\n")
    with pytest.raises(RuntimeError, match="fast_call"):
        build.build()
    assert os.path.exists(build.LIB) and not os.path.exists(build.FAST_LIB)


def test_the_module_is_rebuilt_for_another_torch(build, monkeypatch):
    build.build()
    first = os.stat(build.FAST_LIB).st_mtime_ns
    build.build()
    assert os.stat(build.FAST_LIB).st_mtime_ns == first  # nothing to do
    version = importlib.metadata.version
    monkeypatch.setattr(importlib.metadata, "version",
                        lambda name: "0.0" if name == "torch" else version(name))
    build.build()
    assert os.stat(build.FAST_LIB).st_mtime_ns > first
