"""What a build needs: libmk.so nvcc alone, the Python module the torch that is installed."""
import os

import pytest

from moe_decode_megakernel_persistent_gb300 import _build


@pytest.fixture
def elsewhere(tmp_path, monkeypatch):
    """Builds of one small source into a folder of their own."""
    monkeypatch.setattr(_build, "LIB", str(tmp_path / "libmk.so"))
    monkeypatch.setattr(_build, "MODULE", str(tmp_path / "_torch.so"))
    monkeypatch.setattr(_build, "BUILD", str(tmp_path / "build"))
    monkeypatch.setattr(_build, "SOURCES", [("mk_pack.cu", "mk_pack", [])])
    return tmp_path


def test_the_library_is_there_where_the_module_does_not_compile(elsewhere, monkeypatch):
    monkeypatch.setenv("CXX", "/bin/false")
    with pytest.raises(RuntimeError, match="Python module"):
        _build.build()
    assert os.listdir(elsewhere) and os.path.exists(_build.LIB) and not os.path.exists(_build.MODULE)
    assert not _build.up_to_date()
    made = os.path.getmtime(_build.LIB)
    with pytest.raises(RuntimeError, match="Python module"):   # said again, and the library is not built again
        _build.build()
    assert os.path.getmtime(_build.LIB) == made


def test_without_torch_there_is_the_library_alone(elsewhere, monkeypatch):
    monkeypatch.setattr(_build, "_built_for", lambda: None)
    assert _build.build() == _build.LIB and os.path.exists(_build.LIB) and not os.path.exists(_build.MODULE)
    assert _build.up_to_date()


def test_another_torch_makes_the_module_stale(elsewhere, monkeypatch):
    os.makedirs(_build.BUILD)
    for f in (_build.LIB, _build.MODULE):
        open(f, "w").close()
    assert not _build.up_to_date()                             # nothing says what it was built for
    with open(_build._stamp(), "w") as f:
        f.write(_build._built_for())
    assert _build.up_to_date()
    monkeypatch.setattr(_build, "_built_for", lambda: "cpython-312 torch 0.0")
    assert not _build.up_to_date()
