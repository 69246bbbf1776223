"""The build without torch or a host compiler for it (compilers replaced by scripts, in a folder of its own)."""
import importlib.metadata
import importlib.util
import os

import pytest

from barrier_free_message_gb300 import _build, sfar

FAKE = '''#!/bin/sh
echo "$@" >> "$0.log"
while [ $# -gt 0 ]; do [ "$1" = -o ] && echo built > "$2"; shift; done
'''


@pytest.fixture
def place(tmp_path, monkeypatch):
    out = tmp_path / "out"
    for name, value in (("OUT_DIR", out), ("LIB", out / "libsfar.so"), ("TENSORS", out / "sfar_tensors.so"), ("SOURCES", ["k_misc.cu", "k_ll.cu"])):
        monkeypatch.setattr(_build, name, value if isinstance(value, list) else str(value))
    for name in ("nvcc", "cxx"):
        (tmp_path / name).write_text(FAKE)
        (tmp_path / name).chmod(0o755)
        monkeypatch.setenv(name.upper(), str(tmp_path / name))
    return tmp_path


def runs(place, name):
    log = place / (name + ".log")
    return len(log.read_text().splitlines()) if log.exists() else 0


def without_torch(monkeypatch):
    find, version = importlib.util.find_spec, importlib.metadata.version

    def no_version(name):
        if name == "torch":
            raise importlib.metadata.PackageNotFoundError(name)
        return version(name)

    monkeypatch.setattr(importlib.util, "find_spec", lambda name, *a: None if name == "torch" else find(name, *a))
    monkeypatch.setattr(importlib.metadata, "version", no_version)


def test_the_library_builds_without_torch(place, monkeypatch):
    with monkeypatch.context() as m:
        without_torch(m)
        with pytest.warns(RuntimeWarning, match="torch is not installed"):
            assert _build.build() == _build.LIB
        assert os.path.exists(_build.LIB) and not os.path.exists(_build.TENSORS)
        assert runs(place, "nvcc") == 3 and runs(place, "cxx") == 0
        m.setattr(sfar, "_native", None)
        m.setattr(sfar, "lib", lambda: None)
        with pytest.raises(RuntimeError, match="torch is not installed"):
            sfar._tensors()
    _build.build()                                               # torch is there now: the module alone is built
    assert _build.tensors_error() == "" and runs(place, "nvcc") == 3 and runs(place, "cxx") == 1
    monkeypatch.setattr(_build, "nvcc", lambda: pytest.fail("nothing is to be built"))
    _build.build()
    assert runs(place, "nvcc") == 3 and runs(place, "cxx") == 1


@pytest.mark.parametrize("cxx", ["/bin/false", "/nowhere/c++"])
def test_the_library_builds_without_a_host_compiler_for_torch(place, monkeypatch, cxx):
    _build.build()
    monkeypatch.setenv("CXX", cxx)
    with pytest.warns(RuntimeWarning, match=cxx):
        _build.build(force=True)
    assert os.path.exists(_build.LIB) and cxx in _build.tensors_error()          # none of other sources stays
    with pytest.warns(RuntimeWarning):
        _build.build()                                           # tried again, the library kept
    assert runs(place, "nvcc") == 6


def test_a_library_that_does_not_compile_is_an_error(place, monkeypatch):
    monkeypatch.setenv("NVCC", "/bin/false")
    with pytest.raises(RuntimeError, match="nvcc failed"):
        _build.build()
