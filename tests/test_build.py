"""The build's order and flags, with the compilers replaced by a recorder."""
import os
import sys

import pytest

from rank_gemm_svdq_amd import build as BLD


@pytest.fixture
def recorded(tmp_path, monkeypatch):
    lib = tmp_path / "lib"
    for name, value in (("LIBDIR", lib), ("LIB", lib / "libsvdq.so"), ("EXT", lib / "_block.so"), ("BUILD", tmp_path / "obj")):
        monkeypatch.setattr(BLD, name, str(value))
    done = []

    def run(cmd):
        done.append(cmd)
        if run.fails and any(run.fails in c for c in cmd):
            raise RuntimeError("build step failed")
        open(cmd[cmd.index("-o") + 1], "w").close()
        return ""

    run.fails = None
    monkeypatch.setattr(BLD, "_run", run)
    return run, done


def test_all_units_and_the_module(recorded):
    _, done = recorded
    assert BLD.build() == BLD.LIB
    assert os.path.exists(BLD.LIB) and os.path.exists(BLD.EXT)
    assert sum("-c" in c for c in done) == len(BLD.UNITS)


def test_the_library_does_not_need_the_module(recorded):
    """A machine on which the module's headers are missing still gets the C library."""
    run, _ = recorded
    run.fails = "py_block.cpp"
    with pytest.raises(RuntimeError):
        BLD.build()
    assert os.path.exists(BLD.LIB) and not os.path.exists(BLD.EXT)


def test_without_torch_there_is_no_module_to_build(recorded, monkeypatch):
    monkeypatch.setitem(sys.modules, "torch", None)
    assert BLD.build() == BLD.LIB
    assert os.path.exists(BLD.LIB) and not os.path.exists(BLD.EXT)


def test_the_module_is_compiled_with_its_warnings_on(recorded):
    """Torch's headers are system headers, so that what is said is said of the module."""
    _, done = recorded
    BLD.build()
    cmd = next(c for c in done if any("py_block.cpp" in a for a in c))
    assert "-Wall" in cmd and "-Wextra" in cmd and "-w" not in cmd and not any(a.startswith("-I") for a in cmd)
