"""The build of the compiled module beside the library's."""
import os

import pytest

from bit_quantized_all_gb300 import build as b


@pytest.fixture
def away(monkeypatch, tmp_path):
    """The built files in a folder of their own; the library there is up to date."""
    b.build()
    monkeypatch.setattr(b, "OBJ_DIR", str(tmp_path))
    for name in ("FAST_PATH", "FAST_FAILED"):
        monkeypatch.setattr(b, name, str(tmp_path / os.path.basename(getattr(b, name, name))), raising=False)
    monkeypatch.setattr(b, "_build_locked", lambda *args: pytest.fail("the library was built again"))
    return tmp_path


def test_what_cannot_be_built_stops_nothing_else(monkeypatch, away):
    tries = []

    def no_headers():
        tries.append(1)
        raise RuntimeError("Python.h: no such file")

    monkeypatch.setattr(b, "_build_fast", no_headers)
    old = away / os.path.basename(b.FAST_PATH)
    old.write_text("of other sources")
    os.utime(old, (1, 1))
    with pytest.warns(RuntimeWarning, match="Python.h"):
        assert b.build() == b.LIB_PATH
    assert not old.exists()
    assert b.build() == b.LIB_PATH and len(tries) == 1  # not tried again at every call


def test_the_module_alone(away):
    assert b.build() == b.LIB_PATH
    assert os.path.exists(b.FAST_PATH) and not b._fast_stale()
