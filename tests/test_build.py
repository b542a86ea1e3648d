"""The build: the C library and the module that reads the tensors of small calls."""

import os

import pytest


@pytest.fixture
def small(tmp_path, monkeypatch):
    """The build module on a tree of two small sources."""
    from affine_bit_matmul_gb300 import build as b

    (tmp_path / "a.cu").write_text('extern "C" int answer() { return 42; }\n')
    (tmp_path / "c.cpp").write_text("#include <Python.h>\n"
                                    'static PyModuleDef m = {PyModuleDef_HEAD_INIT, "_calls", 0, -1, 0, 0, 0, 0, 0};\n'
                                    "PyMODINIT_FUNC PyInit__calls(void) { return PyModule_Create(&m); }\n")
    monkeypatch.setattr(b, "BUILD", str(tmp_path / "build"))
    monkeypatch.setattr(b, "LIB", str(tmp_path / "lib.so"))
    monkeypatch.setattr(b, "CALLS", str(tmp_path / "_calls.so"))
    monkeypatch.setattr(b, "sources", lambda: [str(tmp_path / "a.cu")])
    monkeypatch.setattr(b, "calls_source", lambda: str(tmp_path / "c.cpp"))
    return b


def test_the_library_is_built_where_the_module_cannot_be(small):
    with open(small.calls_source(), "w") as f:
        f.write("#error no torch here\n")
    with pytest.raises(RuntimeError, match="no torch here"):
        small.build(force=True)
    assert os.path.exists(small.LIB) and not os.path.exists(small.CALLS)
