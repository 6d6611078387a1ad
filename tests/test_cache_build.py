"""The library's build does not depend on the module that hands torch tensors to the cache operators; no GPU."""
from __future__ import annotations

import os
import shutil

import pytest

from tensor_command_execution_gb300 import _build


@pytest.fixture
def small(tmp_path, monkeypatch):
    """A build of one source file and a module that does not compile."""
    csrc = tmp_path / "csrc"
    csrc.mkdir()
    for name in ("gen_interp.py", "interp_asm.cuh"):
        shutil.copy2(os.path.join(_build.CSRC, name), csrc / name)
    (csrc / "a.cpp").write_text('extern "C" int a() { return 1; }\n')
    (csrc / _build.TORCH_SOURCE).write_text("#error the headers are not here\n")
    for name, value in dict(CSRC=str(csrc), OUT_DIR=str(tmp_path / "lib"), OBJ_DIR=str(tmp_path / "obj"), CU_SOURCES=[], CPP_SOURCES=["a.cpp"],
                            HEADERS=["gen_interp.py", "interp_asm.cuh"], LIB_PATH=str(tmp_path / "lib" / "libcmdexec.so"),
                            TORCH_PATH=str(tmp_path / "lib" / "_cache_torch.so"), TORCH=True).items():
        monkeypatch.setattr(_build, name, value)
    return csrc


def test_the_library_is_built_where_the_module_cannot_be(small):
    os.makedirs(_build.OUT_DIR)
    with open(_build.TORCH_PATH, "w") as f:
        f.write("an older build")
    assert _build.build() == _build.LIB_PATH and os.path.exists(_build.LIB_PATH)
    assert not os.path.exists(_build.TORCH_PATH)  # (not taken for the present one)
    before = os.path.getmtime(_build.LIB_PATH)
    _build.build()
    assert os.path.getmtime(_build.LIB_PATH) == before  # (nor tried again with every start)
    with pytest.raises(RuntimeError, match="module for torch tensors could not be built(.|\n)*the headers are not here"):
        _build.module_path()
    assert os.path.getmtime(_build.LIB_PATH) == before


def test_the_module_is_built_when_it_can_be(small):
    pytest.importorskip("torch")
    _build.build()
    source = small / _build.TORCH_SOURCE
    source.write_text('extern "C" int b() { return 2; }\n')
    os.utime(source, (0, 0))  # (the library stays as it is)
    assert _build.module_path() == _build.TORCH_PATH and os.path.exists(_build.TORCH_PATH)


def test_a_missing_torch_is_an_error_of_the_module_alone(small, monkeypatch):
    monkeypatch.setattr(_build, "TORCH", False)
    assert _build.build() == _build.LIB_PATH
    with pytest.raises(RuntimeError, match="torch is not installed"):
        _build.module_path()
