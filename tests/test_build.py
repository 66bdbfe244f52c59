"""Building without a compiler for the CPython module: the C library, and the
steps with it, need none of that."""
import os
import stat

import pytest

from bit_blockwise_adamw_gb300 import _binding as B
from bit_blockwise_adamw_gb300 import build


@pytest.fixture
def no_host_compiler(tmp_path, monkeypatch):
    """A build folder of its own, a stand-in for nvcc that makes its output, a
    host compiler that fails."""
    fake = tmp_path / "nvcc"
    fake.write_text('#!/bin/sh\nwhile [ "$1" != -o ]; do shift; done\ntouch "$2"\n')
    fake.chmod(fake.stat().st_mode | stat.S_IXUSR)
    out = tmp_path / "out"
    monkeypatch.setattr(build, "OUT_DIR", str(out))
    monkeypatch.setattr(build, "LIB", str(out / "libq8adamw.so"))
    monkeypatch.setattr(build, "nvcc", lambda: str(fake))
    monkeypatch.setenv("CXX", "false")
    monkeypatch.setattr(B, "_lists", None)
    return out


def test_the_library_is_built_without_the_lists_module(no_host_compiler):
    with pytest.warns(RuntimeWarning, match="q8_lists"):
        assert build.build() == build.LIB
    assert os.path.exists(build.LIB)
    with pytest.warns(RuntimeWarning, match="q8_lists"):         # said again by a build that has nothing else to do
        build.build()
    with pytest.raises(RuntimeError, match="not built"):
        B.pack_grads([])


def test_a_module_of_older_sources_does_not_stay(no_host_compiler):
    no_host_compiler.mkdir()
    old = build.lists_module()
    with open(old, "w"):
        os.utime(old, (0, 0))
    with pytest.warns(RuntimeWarning, match="q8_lists"):
        build.build()
    assert not os.path.exists(old)


def test_no_host_compiler_at_all(no_host_compiler, monkeypatch):
    monkeypatch.setenv("CXX", "/nowhere/g++")
    with pytest.warns(RuntimeWarning, match="q8_lists"):
        build.build()
    assert os.path.exists(build.LIB)
