"""The build: the C library does not hang on what only the Python binding needs."""
from __future__ import annotations

import os
import sysconfig

import pytest

from paged_fp8_speculative_gb300 import api, build

NVCC = """#!/bin/sh
# takes down what it is asked for, and makes it
echo "$@" >> "$(dirname "$0")/calls"
while [ $# -gt 1 ]; do [ "$1" = -o ] && echo made > "$2"; shift; done
"""


@pytest.fixture
def place(tmp_path, monkeypatch):
    """A package folder of its own, the real sources, and an nvcc that only makes its output files."""
    nvcc = tmp_path / "bin" / "nvcc"
    nvcc.parent.mkdir()
    nvcc.write_text(NVCC)
    nvcc.chmod(0o755)
    pkg = tmp_path / "pkg"
    pkg.mkdir()
    monkeypatch.setattr(build, "nvcc", lambda: str(nvcc))
    for name, path in (("PKG", pkg), ("BUILD", pkg / "_build"), ("LIB", pkg / "libmtpattn.so"),
                       ("BINDING", pkg / os.path.basename(build.BINDING))):
        monkeypatch.setattr(build, name, str(path))
    return pkg


def no_torch():
    raise RuntimeError("PyTorch not found")


@pytest.mark.parametrize("torch_dir", [no_torch, lambda: "/nonexistent"], ids=["none", "headers"])
def test_the_library_is_linked_where_the_binding_cannot_be_built(place, monkeypatch, torch_dir):
    monkeypatch.setattr(build, "_torch_dir", torch_dir)
    with pytest.raises(RuntimeError, match="libmtpattn.so is built, the Python binding is not"):
        build.build(lib_path=build.LIB)
    assert (place / "libmtpattn.so").read_text() == "made\n"
    assert not os.path.exists(build.BINDING)
    calls = (place.parent / "bin" / "nvcc").with_name("calls").read_text().splitlines()
    assert calls[-1].count("-shared") == 1 and all(" -c " in c for c in calls[:-1])


def test_the_binding_is_this_interpreters():
    assert os.path.basename(build.BINDING) == "_binding" + sysconfig.get_config_var("EXT_SUFFIX")
    assert os.path.samefile(api.binding().__file__, build.BINDING)
