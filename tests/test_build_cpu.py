"""The build knows by content what a library was made from (a stand-in for nvcc: it puts its inputs together)."""
import os
import stat

import pytest

from top_sparse_attention_02_b200 import build as real

FAKE = """#!/bin/sh
echo "$@" >> "$CALLS"
while [ $# -gt 0 ]; do
  case "$1" in
    -o) out="$2"; shift ;;
    *.cu|*.o) in="$in $1" ;;
  esac
  shift
done
cat $in > "$out"
"""


@pytest.fixture
def build(tmp_path, monkeypatch):
    """The build module over two small sources and a header, with the stand-in compiler."""
    csrc, inc = tmp_path / "csrc", tmp_path / "include"
    csrc.mkdir(), inc.mkdir()
    (csrc / "a.cu").write_text("a1"), (csrc / "b.cu").write_text("b1"), (inc / "h.h").write_text("h1")
    nvcc = tmp_path / "nvcc"
    nvcc.write_text(FAKE)
    nvcc.chmod(nvcc.stat().st_mode | stat.S_IXUSR)
    monkeypatch.setenv("NVCC", str(nvcc))
    monkeypatch.setenv("CALLS", str(tmp_path / "calls"))
    for name, value in dict(CSRC=csrc, INCLUDE=inc, LIB=tmp_path / "l.so", BUILD_DIR=tmp_path / "o", DEBUG_LIB=tmp_path / "d.so",
                            DEBUG_BUILD_DIR=tmp_path / "od").items():
        monkeypatch.setattr(real, name, str(value))
    real.compiled = lambda: (tmp_path / "calls").read_text().count(" -c ") if (tmp_path / "calls").exists() else 0
    yield real
    del real.compiled


@pytest.mark.parametrize("debug", [False, True])
@pytest.mark.parametrize("edit,again", [("csrc/a.cu", 1), ("csrc/b.cu", 1), ("include/h.h", 2)])
def test_an_edit_is_seen_whatever_its_time(build, tmp_path, debug, edit, again):
    lib = build.ensure(debug=debug)
    assert build.current(debug) and build.compiled() == 2
    assert build.ensure(debug=debug) == lib and build.build(debug=debug) == lib and build.compiled() == 2
    (tmp_path / edit).write_text("edited")
    os.utime(tmp_path / edit, (1, 1))  # as a copy that keeps times may leave it
    assert not build.current(debug)
    build.ensure(debug=debug)
    assert build.current(debug) and build.compiled() == 2 + again
    if edit != "include/h.h":
        assert "edited" in open(lib).read()


def test_the_two_libraries_are_told_apart(build, tmp_path):
    build.ensure()
    build.ensure(debug=True)
    assert build.compiled() == 4
    os.replace(build.LIB, build.DEBUG_LIB)
    assert not build.current(debug=True) and not build.current()


def test_a_library_of_other_sources_is_an_error_without_a_compiler(build, tmp_path, monkeypatch):
    build.ensure(debug=True)

    def none():
        raise RuntimeError("nvcc not found")

    monkeypatch.setattr(build, "_nvcc", none)
    assert build.ensure(debug=True) == build.DEBUG_LIB  # nothing to do
    (tmp_path / "csrc" / "a.cu").write_text("a2")
    with pytest.raises(RuntimeError, match="was not built from these sources"):
        build.ensure(debug=True)
    os.remove(build.DEBUG_LIB)
    with pytest.raises(RuntimeError, match="missing"):
        build.ensure(debug=True)


def test_a_failed_compilation_is_not_taken_for_done(build, tmp_path, monkeypatch):
    build.ensure()
    good = open(os.environ["NVCC"]).read()
    (tmp_path / "csrc" / "a.cu").write_text("a2")
    open(os.environ["NVCC"], "w").write("#!/bin/sh\nexit 1\n")
    with pytest.raises(RuntimeError, match="nvcc failed"):
        build.ensure()
    assert not build.current()
    open(os.environ["NVCC"], "w").write(good)
    build.ensure()
    assert build.current() and "a2" in open(build.LIB).read()


def test_bounded_wait_tests_bring_their_library_up_to_date(pytestconfig, monkeypatch):
    """conftest.py does so before a test that takes it."""
    asked = []
    monkeypatch.setattr(real, "ensure", lambda debug=False: asked.append(debug))

    class Item:
        fixturenames = ["dbg", "cuda_dev"]

    class Other:
        fixturenames = ["cuda_dev"]

    import conftest

    conftest.pytest_runtest_setup(Other)
    assert asked == []
    conftest.pytest_runtest_setup(Item)
    assert asked == [True]
    here = os.path.dirname(os.path.abspath(__file__))
    for name in os.listdir(here):  # whoever loads it takes the fixture of that name
        src = open(os.path.join(here, name)).read() if name.startswith("test_") and name.endswith("_gpu.py") else ""
        if "libtsa_debug.so" in src and "CDLL" in src:
            assert "def dbg(" in src, name
