"""Building the Python extension of the attention calls: the C library needs
neither torch's headers nor a host compiler of its own, so a machine without
them builds the library and is told what is left out; an extension that does
not compile is an error."""
import os
import subprocess
import sys

import pytest

from ring_collectives_amd import build as rb


def _stale(monkeypatch, tmp_path):
    old = tmp_path / "_binding.so"
    old.write_bytes(b"built against an older library")
    monkeypatch.setattr(rb, "BINDING", str(old))
    return old


@pytest.mark.parametrize("lacks", ["torch", "g++", "headers"])
def test_without_what_it_needs_the_extension_is_left_out(lacks, monkeypatch, tmp_path, capsys):
    old = _stale(monkeypatch, tmp_path)
    if lacks == "torch":
        monkeypatch.setitem(sys.modules, "torch", None)          # as if it were not installed
    elif lacks == "g++":
        monkeypatch.setenv("PATH", str(tmp_path))
    else:
        import sysconfig
        paths = dict(sysconfig.get_paths(), include=str(tmp_path))
        monkeypatch.setattr(sysconfig, "get_paths", lambda *a, **k: paths)
    rb._build_binding(False)
    assert not old.exists()                                      # never one that belongs to another library
    assert "_binding.so" in capsys.readouterr().out


def test_an_extension_that_does_not_compile_is_an_error(monkeypatch, tmp_path):
    _stale(monkeypatch, tmp_path)
    (tmp_path / "binding.cpp").write_text("#error no\n")
    monkeypatch.setattr(rb, "CSRC", str(tmp_path))
    with pytest.raises(subprocess.CalledProcessError):
        rb._build_binding(False)
    assert not [f for f in os.listdir(tmp_path) if ".tmp" in f]
