"""The build's two products: libpkv.so, which needs no torch, and
_torch_calls.so, made against the installed torch."""
import ctypes
import os

import pytest

from paged_kv_cache_tables_gb300 import build as B


@pytest.fixture
def place(tmp_path, monkeypatch):
    """The build with its products in a folder of their own, libpkv.so of the host's part alone (seconds to compile)."""
    for name, value in (("BUILD", "_build"), ("LIB", "libpkv.so"), ("CALLS", "_torch_calls.so")):
        monkeypatch.setattr(B, name, str(tmp_path / value))
    monkeypatch.setattr(B, "SOURCES", ["host_sched.cpp"])
    return tmp_path


def missing():
    raise RuntimeError("torch not found")


def test_the_library_is_built_without_torch(place, monkeypatch):
    monkeypatch.setattr(B, "_torch_dir", missing)
    assert B.build() == str(place / "libpkv.so")
    assert ctypes.CDLL(str(place / "libpkv.so")).pkv_pool_create is not None
    assert not (place / "_torch_calls.so").exists()
    before = os.stat(place / "libpkv.so").st_mtime_ns
    B.build()   # nothing changed: nothing is made again
    assert os.stat(place / "libpkv.so").st_mtime_ns == before


def test_the_library_is_built_where_the_calls_do_not_compile(place, monkeypatch):
    """A torch that the calls do not compile against: an error, after the library is in its place."""
    (place / "torch" / "include").mkdir(parents=True)
    monkeypatch.setattr(B, "_torch_dir", lambda: str(place / "torch"))
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        B.build()
    assert (place / "libpkv.so").exists() and not (place / "_torch_calls.so").exists()


def test_the_calls_are_built_again_for_another_torch(place, monkeypatch):
    made = []
    (place / "_build").mkdir()
    monkeypatch.setattr(B, "_compile", lambda src, verbose: made.append(src) or str(place / src))
    monkeypatch.setattr(B, "_link", lambda objs: made.append("lib") or (place / "libpkv.so").write_text("x"))
    monkeypatch.setattr(B, "_compile_calls", lambda: made.append("calls") or str(place / "calls.o"))
    monkeypatch.setattr(B, "_link_calls", lambda obj: (place / "_torch_calls.so").write_text("x"))
    torch = ["/a/torch 2.9"]
    monkeypatch.setattr(B, "_torch_built_for", lambda: torch[0])
    B.build()
    assert sorted(made) == ["calls", "host_sched.cpp", "lib"]
    del made[:]
    B.build()
    assert made == []
    torch[0] = "/a/torch 2.11"
    B.build()
    assert made == ["calls"]
