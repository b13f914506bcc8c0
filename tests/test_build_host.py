"""build.py's handling of compiler runs that fail, with a stand-in for the compiler (no GPU)."""
import os
import subprocess

import pytest

from backward_lstm_fwd_b200 import build as lbuild

# writes its -o file; fails on sources that say so, after it began to write
COMPILER = """#!/bin/sh
out= src= link=
while [ $# -gt 0 ]; do
  case "$1" in
    -o) out="$2"; shift;;
    -shared) link=1;;
    *.cu) src="$1";;
  esac
  shift
done
echo object > "$out"
if [ -n "$src" ] && grep -q broken "$src"; then exit 1; fi
if [ -n "$link" ] && [ -e "$(dirname "$0")/no_link" ]; then exit 1; fi
exit 0
"""


@pytest.fixture()
def tree(tmp_path, monkeypatch):
    tmp_path = tmp_path / f"in.tmp{os.getpid()}"  # (a folder's own name says nothing)
    tmp_path.mkdir()
    csrc = tmp_path / "csrc"
    csrc.mkdir()
    for n in ("a", "b", "c"):
        (csrc / f"{n}.cu").write_text("fine")
    nvcc = tmp_path / "nvcc"
    nvcc.write_text(COMPILER)
    nvcc.chmod(0o755)
    monkeypatch.setattr(lbuild, "PKG", str(tmp_path))
    monkeypatch.setattr(lbuild, "CSRC", str(csrc))
    monkeypatch.setattr(lbuild, "LIB_PATH", str(tmp_path / "lib.so"))
    monkeypatch.setattr(lbuild, "_nvcc", lambda: str(nvcc))
    return tmp_path


def left(tree):
    return sorted(p.name for d in (tree, tree / "_build") if d.exists() for p in d.iterdir() if ".tmp" in p.name)


def test_a_failed_compile_leaves_nothing(tree):
    (tree / "csrc" / "b.cu").write_text("broken")
    with pytest.raises(RuntimeError, match="b.cu"):
        lbuild.build()
    assert not left(tree) and not (tree / "lib.so").exists()
    (tree / "csrc" / "b.cu").write_text("fine")
    assert lbuild.build() == str(tree / "lib.so") and (tree / "lib.so").exists()
    assert not left(tree)


def test_a_failed_link_leaves_nothing(tree):
    (tree / "no_link").write_text("")
    with pytest.raises(subprocess.CalledProcessError):
        lbuild.build()
    assert not left(tree) and not (tree / "lib.so").exists()


def test_leftovers_of_a_killed_build_go(tree):
    gone = subprocess.Popen(["true"])
    gone.wait()
    (tree / "_build").mkdir()
    (tree / "_build" / f"a.o.tmp{gone.pid}.o").write_text("")
    (tree / f"lib.so.tmp{gone.pid}").write_text("")
    other = tree / "_build" / f"b.o.tmp{os.getpid()}.o"  # (of a process that lives: another build's)
    other.write_text("")
    lbuild.build()
    assert left(tree) == []  # this process is that other one, and used the name itself
    alive = tree / "_build" / f"b.o.tmp{os.getppid()}.o"
    alive.write_text("")
    lbuild.build(force=True)
    assert left(tree) == [alive.name]
