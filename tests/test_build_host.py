"""What build() makes, and when: the library by itself where the extension cannot be built,
and the extension anew for another torch."""
import os

import pytest
import torch

from w4a16_int4_weight_sigmoid_gb300 import build as B
from w4a16_int4_weight_sigmoid_gb300 import chord


@pytest.fixture(autouse=True)
def _built():
    B.build()
    yield
    assert B.up_to_date()


def test_the_library_does_not_need_the_extension(monkeypatch, tmp_path):
    """Without a C++ compiler for it the extension is missing, with a warning; the library is
    built, nothing else is compiled, and calls that need the extension say what is missing."""
    ext = tmp_path / "_chord.so"
    ext.write_bytes(b"of other headers")
    os.utime(ext, (1, 1))
    before = os.path.getmtime(B.LIB_PATH)
    monkeypatch.setattr(B, "EXT_PATH", str(ext))
    monkeypatch.setattr(B, "CXX", str(tmp_path / "no-compiler"))
    with pytest.warns(RuntimeWarning, match="extension is not"):
        assert B.build() == B.LIB_PATH
    assert os.path.getmtime(B.LIB_PATH) == before and not ext.exists()
    monkeypatch.setattr(chord, "EXT_PATH", str(ext))
    monkeypatch.setattr(chord, "_ext_module", None)
    chord.lib()
    with pytest.raises(RuntimeError, match="missing"):
        chord.chord_mxfp4_dequantize(None, None, None)


def test_the_extension_is_of_the_torch_that_loads_it(monkeypatch):
    assert B.up_to_date()
    monkeypatch.setattr(torch, "__version__", torch.__version__ + ".other")
    assert not B.up_to_date()
