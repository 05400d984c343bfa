"""The library is rebuilt when any file it is made of is newer."""

import glob
import os
import re

import pytest

from attention_forward_09_gb300 import _build

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_every_included_header_is_an_input():
    have = {os.path.realpath(p) for p in _build.inputs()}
    for src in [p for p in have if p.endswith((".cu", ".cpp", ".h", ".cuh"))]:
        for name in re.findall(r'^#include "([^"]+)"', open(src).read(), flags=re.M):
            assert os.path.realpath(os.path.join(os.path.dirname(src), name)) in have, (src, name)
    assert {os.path.realpath(p) for p in glob.glob(os.path.join(ROOT, "include", "*.h"))} <= have


@pytest.mark.parametrize("name", sorted(os.path.basename(p) for p in glob.glob(os.path.join(ROOT, "include", "*.h"))))
def test_a_newer_header_means_a_new_library(name, tmp_path, monkeypatch):
    """A library newer than all its inputs is taken as it is; one older than a header goes to the compiler."""
    lib = tmp_path / "lib.so"
    lib.write_bytes(b"")
    newest = max(os.path.getmtime(p) for p in _build.inputs())
    at = {os.path.join(ROOT, "include", name): newest + 10}
    real = os.path.getmtime
    monkeypatch.setattr(_build, "LIB", str(lib))
    monkeypatch.setattr(_build.os.path, "getmtime", lambda p: at.get(os.path.realpath(str(p)), real(p)))

    def compiler():
        raise FileNotFoundError("asked for")

    monkeypatch.setattr(_build, "nvcc", compiler)
    os.utime(lib, (newest + 20, newest + 20))
    assert _build.build() == str(lib)
    os.utime(lib, (newest + 5, newest + 5))
    with pytest.raises(FileNotFoundError, match="asked for"):
        _build.build()
