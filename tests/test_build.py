"""The in-tree build with a stand-in for nvcc (CPU only): several at once, a failed
one, and what makes the library stale."""
import os
import stat
import threading

import pytest

from paged_kv_cache_109_gb300 import _build

# "compiles" by writing its source's name, links by joining its inputs; fails on demand
FAKE = """#!/bin/sh
out=; inputs=
while [ $# -gt 0 ]; do
  case "$1" in
    -o) out=$2; shift;;
    *.cu|*.o) inputs="$inputs $1";;
  esac
  shift
done
for i in $inputs; do
  case "$i" in
    *"$FAIL_ON") [ -n "$FAIL_ON" ] && { echo broken >&2; exit 1; };;
  esac
done
sleep 0.2
for i in $inputs; do
  case "$i" in
    *.cu) basename "$i" >> "$out.part";;
    *) cat "$i" >> "$out.part" || exit 1;;
  esac
done
mv "$out.part" "$out"
"""


@pytest.fixture
def package(tmp_path, monkeypatch):
    nvcc = tmp_path / "bin" / "nvcc"
    nvcc.parent.mkdir()
    nvcc.write_text(FAKE)
    nvcc.chmod(nvcc.stat().st_mode | stat.S_IXUSR)
    pkg = tmp_path / "pkg"
    pkg.mkdir()
    monkeypatch.setenv("NVCC", str(nvcc))
    monkeypatch.setenv("FAIL_ON", "")
    monkeypatch.setattr(_build, "PKG", str(pkg))
    monkeypatch.setattr(_build, "LIB", str(pkg / "libpa.so"))
    return pkg


def test_builds_at_once_do_not_meet(package):
    wrong = []

    def work(delay):
        try:
            threading.Event().wait(delay)
            _build.build(force=True)
        except Exception as e:                          # a thread's error must reach the test
            wrong.append(repr(e))
    threads = [threading.Thread(target=work, args=(0.1 * i,)) for i in range(4)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not wrong
    assert (package / "libpa.so").read_text().split() == ["pa.cu", "serving.cu"]
    assert os.listdir(package) == ["libpa.so"]


def test_a_failed_build_leaves_nothing_behind(package, monkeypatch):
    (package / "libpa.so").write_text("before")
    monkeypatch.setenv("FAIL_ON", "serving.cu")
    with pytest.raises(RuntimeError, match="broken"):
        _build.build(force=True)
    assert os.listdir(package) == ["libpa.so"] and (package / "libpa.so").read_text() == "before"


def test_every_file_that_is_compiled_makes_the_library_stale(tmp_path):
    lib = tmp_path / "libpa.so"
    lib.write_text("")
    named = {os.path.basename(f) for f in _build.sources()}
    here = {f for f in os.listdir(_build.CSRC) if f.endswith((".cu", ".cuh", ".h"))}
    assert here | {"pa.h"} == named and "debug_checks.h" in named
    newest = max(os.path.getmtime(f) for f in _build.sources())
    for age, stale in ((1, False), (-1, True)):
        os.utime(lib, (newest + age, newest + age))
        assert _build.stale(str(lib)) == stale
