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


@pytest.fixture
def built(tree, monkeypatch):
    """A current library, and a record of what is compiled instead of compiling it."""
    open(pa_build.LIB, "w").close()
    asked = []
    monkeypatch.setattr(pa_build, "_build_lib", lambda *a: asked.append("library"))

    def calls(out):
        asked.append("calls")
        open(out, "w").close()
    monkeypatch.setattr(pa_build, "_build_calls", calls)
    return asked


def test_a_missing_extension_is_built_by_itself(built):
    pa_build.build()
    assert built == ["calls"] and os.path.exists(pa_build.calls_path())
    pa_build.build()
    assert built == ["calls"]
    pa_build.build(force=True)
    assert sorted(built) == ["calls", "calls", "library"]


def test_an_extension_that_cannot_be_built_is_reported_and_retried_on_request(built, monkeypatch, capsys):
    works = pa_build._build_calls
    monkeypatch.setattr(pa_build, "_build_calls", lambda out: built.append("calls") or "first line\nno such header")
    for n in range(2):                                  # tried once, said every time
        pa_build.build()
        assert built == ["calls"] and "no such header" in capsys.readouterr().out
    monkeypatch.setattr(pa_build, "_build_calls", works)
    pa_build.build(retry=True)
    assert built == ["calls"] * 2 and os.path.exists(pa_build.calls_path()) and not capsys.readouterr().out
    assert not os.path.exists(pa_build.calls_path() + ".failed")


def test_a_current_library_needs_no_compiler(tree, monkeypatch, capsys):
    open(pa_build.LIB, "w").close()

    def none():
        raise RuntimeError("nvcc not found")
    monkeypatch.setattr(pa_build, "_nvcc", none)
    assert pa_build.build() == pa_build.LIB
    assert "nvcc not found" in capsys.readouterr().out


def test_what_older_sources_left_goes(built, tree):
    old = pa_build.calls_path()
    open(old, "w").close()
    with open(tree / "include" / "pa.h", "a") as f:
        f.write("\n")
    os.utime(tree / "include" / "pa.h", (0, 0))
    pa_build.build()
    assert os.path.exists(pa_build.calls_path()) and not os.path.exists(old)


def test_without_torch_there_is_no_extension_to_report(built, tree, monkeypatch, capsys):
    monkeypatch.setattr(pa_build, "calls_path", lambda: None)
    monkeypatch.chdir(tree)
    (tree / ".failed").write_text("another program's file")
    pa_build.build()
    assert built == [] and not capsys.readouterr().out
