"""The build: the library needs nvcc alone; the Python binding's marshalling
module is optional, and one compiled for another PyTorch is not loaded."""
import os
import shutil

import pytest

from logits_processing_token_gb300 import _build
from logits_processing_token_gb300 import tg as T


@pytest.fixture(scope="module", autouse=True)
def _lib():
    _build.build()


def test_library_builds_without_the_binding(monkeypatch, capfd, tmp_path):
    monkeypatch.setattr(_build, "BINDING", str(tmp_path / "tg_binding.so"))

    def fails():
        raise RuntimeError("no headers")

    monkeypatch.setattr(_build, "build_binding", fails)
    assert _build.build() == _build.LIB and os.path.exists(_build.LIB)
    assert "no headers" in capfd.readouterr().err
    monkeypatch.setattr(_build, "_binding_for", lambda: None)  # no PyTorch at all
    assert _build.build() == _build.LIB
    assert capfd.readouterr().err == ""
    monkeypatch.setattr(T, "_binding", None)
    with pytest.warns(UserWarning, match="not built"):
        assert T._load_binding() is None


def test_binding_of_another_pytorch_is_stale(monkeypatch, tmp_path):
    assert _build.binding_current()
    other = str(tmp_path / "tg_binding.so")
    shutil.copy(_build.BINDING, other)
    monkeypatch.setattr(_build, "BINDING", other)
    assert not _build.binding_current()  # of unknown origin
    for text, current in ((_build._binding_for(), True), ("cpython-312-x86_64-linux-gnu, torch 1.0.0", False)):
        with open(other + ".for", "w") as f:
            f.write(text)
        assert _build.binding_current() == current
    monkeypatch.setattr(T, "_binding", None)
    with pytest.warns(UserWarning, match="not built"):
        assert T._load_binding() is None
    built = []
    monkeypatch.setattr(_build, "build_binding", lambda: built.append(1))
    _build.build()
    assert built == [1]
