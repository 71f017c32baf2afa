"""When the library is built again (CPU only)."""

import os
import re

import pytest

from hybrid_linear_attention_prefill_gb300 import build as B


def included():
    """The files of this tree that the sources include, and those include."""
    found, left = set(), list(B.sources())
    while left:
        path = left.pop()
        for name in re.findall(r'^#include "(.+)"', open(path).read(), re.M):
            there = os.path.normpath(os.path.join(os.path.dirname(path), name))
            if there not in found:
                found.add(there)
                left.append(there)
    return sorted(found)


def test_every_included_file_is_looked_at():
    assert set(included()) <= {os.path.normpath(p) for p in B._deps()}


@pytest.mark.parametrize("path", included(), ids=os.path.basename)
def test_a_newer_header_builds_again(monkeypatch, tmp_path, path):
    lib = tmp_path / "libgdn.so"
    lib.write_bytes(b"")
    monkeypatch.setattr(B, "LIB", str(lib))
    newest = max(os.path.getmtime(p) for p in B._deps() + included())
    os.utime(lib, (newest + 1, newest + 1))
    assert not B.needs_build()
    there = os.path.getmtime
    monkeypatch.setattr(B.os.path, "getmtime", lambda p: newest + 2 if os.path.normpath(p) == path else there(p))
    assert B.needs_build()
