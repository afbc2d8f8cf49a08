"""What the build makes when, with a compiler that only touches its output."""
import os

import pytest

from sparse_gemm_irregular_gm_gb300 import build


@pytest.fixture
def place(tmp_path, monkeypatch):
    nvcc = tmp_path / "nvcc"
    nvcc.write_text('#!/bin/sh\necho "$@" >> ' + str(tmp_path / "calls") +
                    '\nwhile [ $# -gt 0 ]; do [ "$1" = -o ] && touch "$2"; shift; done\n')
    nvcc.chmod(0o755)
    monkeypatch.setenv("NVCC", str(nvcc))
    for name, at in (("LIB", "lib.so"), ("MARSHAL", "marshal.so"), ("BUILD", "objects"), ("MARSHAL_FOR", "objects/marshal.for")):
        monkeypatch.setattr(build, name, str(tmp_path / at), raising=False)
    return tmp_path


def compiles(place):
    calls = place / "calls"
    return len(calls.read_text().splitlines()) if calls.exists() else 0


def made(monkeypatch, place):
    """A stand-in for the extension's compilation; the list of its calls."""
    calls = []

    def marshal():
        calls.append(1)
        os.makedirs(place / "objects", exist_ok=True)
        (place / "marshal.so").touch()
        (place / "objects" / "marshal.for").write_text(build.made_for())

    monkeypatch.setattr(build, "build_marshal", marshal)
    return calls


def test_the_library_is_there_where_the_extension_fails(place, monkeypatch):
    def fails():
        raise RuntimeError("g++ failed")

    monkeypatch.setattr(build, "build_marshal", fails)
    with pytest.raises(RuntimeError, match="g\\+\\+ failed"):
        build.build()
    assert (place / "lib.so").exists()


def test_without_torch_the_library_alone_is_built(place, monkeypatch):
    calls = made(monkeypatch, place)
    find = build.importlib.util.find_spec
    monkeypatch.setattr(build.importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    assert build.build() == str(place / "lib.so")
    assert (place / "lib.so").exists() and not calls


def test_another_torch_rebuilds_the_extension_alone(place, monkeypatch):
    calls = made(monkeypatch, place)
    build.build()
    n = compiles(place)
    assert n == len(build.SOURCES) + 1 and len(calls) == 1
    build.build()
    assert compiles(place) == n and len(calls) == 1
    version = build.importlib.metadata.version
    monkeypatch.setattr(build.importlib.metadata, "version", lambda name: "0.0" if name == "torch" else version(name))
    build.build()
    assert compiles(place) == n and len(calls) == 2


def test_each_is_rebuilt_when_its_sources_are_newer(place, monkeypatch):
    calls = made(monkeypatch, place)
    build.build()
    n = compiles(place)
    os.utime(place / "lib.so", (1, 1))
    build.build()
    assert compiles(place) == 2 * n and len(calls) == 1
    os.utime(place / "marshal.so", (1, 1))
    build.build()
    assert compiles(place) == 2 * n and len(calls) == 2
    build.build(force=True)
    assert compiles(place) == 3 * n and len(calls) == 3
