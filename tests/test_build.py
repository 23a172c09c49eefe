"""Which built files the build takes for current (no GPU, nothing is compiled)."""
import os
import shutil

import pytest

from paged_kv_cache_306_gb300 import build as pa_build

pytest.importorskip("torch")


@pytest.fixture
def tree(tmp_path, monkeypatch):
    """A copy of the sources with an empty output folder."""
    for name in ("CSRC", "INCLUDE"):
        d = tmp_path / name.lower()
        shutil.copytree(getattr(pa_build, name), d)
        monkeypatch.setattr(pa_build, name, str(d))
    out = tmp_path / "out"
    out.mkdir()
    monkeypatch.setattr(pa_build, "OUT_DIR", str(out))
    monkeypatch.setattr(pa_build, "LIB", str(out / "libpa.so"))
    return tmp_path


@pytest.mark.parametrize("source", ["include/pa.h", "csrc/fp4_calls.cpp"])
def test_an_extension_of_another_source_is_not_taken(tree, source):
    """Two environments share the output folder: when one has built the library from a changed header, the other's
    extension, compiled from the old one, must not be what it loads."""
    old = pa_build.calls_path()
    open(old, "w").close()
    assert pa_build.calls_path() == old
    with open(tree / source, "a") as f:
        f.write("\n// changed\n")
    open(pa_build.LIB, "w").close()                     # the other environment's build, newer than everything
    later = max(os.path.getmtime(tree / source), os.path.getmtime(old)) + 10
    os.utime(pa_build.LIB, (later, later))
    assert pa_build.calls_path() != old and not os.path.exists(pa_build.calls_path())
    assert pa_build._stale()
