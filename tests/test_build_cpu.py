"""The in-tree build: each library is compiled when it is first needed, from its own sources."""
import os
from types import SimpleNamespace

import pytest

from sparse_moe_routed_gb300 import _block, _lib
from sparse_moe_routed_gb300 import build as B


@pytest.fixture
def compiled(tmp_path, monkeypatch):
    """The .cu files handed to the compiler, with the libraries in an empty folder and a compiler that touches its
    output."""
    seen = []

    def run(cmd, **kw):
        out = cmd[cmd.index("-o") + 1]
        os.makedirs(os.path.dirname(out), exist_ok=True)
        open(out, "w").close()
        if "-c" in cmd:
            seen.append(os.path.relpath(cmd[cmd.index("-c") + 1], B.HERE))
        return SimpleNamespace(returncode=0, stdout="", stderr="")

    monkeypatch.setattr(B.subprocess, "run", run)
    monkeypatch.setattr(B, "LIB", str(tmp_path / "libmoe.so"))
    monkeypatch.setattr(B, "LIB_BLOCK", str(tmp_path / "libmoe_block.so"))
    monkeypatch.setattr(B, "BUILD_DIR", str(tmp_path / "objs"))

    class Library:
        def __init__(self, path):
            self.path = path

        def __getattr__(self, name):
            return SimpleNamespace()

    monkeypatch.setattr(_lib.C, "CDLL", Library)
    monkeypatch.setattr(_lib, "_lib", None)
    monkeypatch.setattr(_block, "_blk", None)
    return seen


def folders(seen):
    return {os.path.dirname(s) for s in seen}


def test_libmoe_alone_compiles_no_source_of_the_other_library(compiled):
    assert _lib.load().path == B.LIB
    assert folders(compiled) == {"csrc"} and not os.path.exists(B.LIB_BLOCK)
    n = len(compiled)
    assert _block.load().path == B.LIB_BLOCK
    assert folders(compiled[n:]) == {"csrc_block"}


def test_build_makes_both_and_only_what_is_out_of_date(compiled):
    assert B.build() == B.LIB
    assert folders(compiled) == {"csrc", "csrc_block"} and os.path.exists(B.LIB_BLOCK)
    assert B.up_to_date()
    compiled.clear()
    B.build()
    assert compiled == []
    os.utime(B.LIB_BLOCK, (0, 0))  # older than its sources
    assert not B.up_to_date()
    B.build()
    assert folders(compiled) == {"csrc_block"} and B.up_to_date()
    compiled.clear()
    B.build(force=True)
    assert folders(compiled) == {"csrc", "csrc_block"}
