"""Which objects the build makes again, with a stand-in for the compiler (no GPU, no nvcc needed)."""
import os
import shutil
import subprocess
import sys

import pytest

from weight_state_recurrence_b200 import build

STUB = """#!/bin/sh
# writes its arguments to the file behind -o and to a log
for a in "$@"; do [ "$last" = -o ] && out="$a"; last="$a"; done
echo "$@" > "$out"
echo "$last" >> "$STUB_LOG"
"""


@pytest.fixture
def tree(tmp_path):
    """A small library with this build.py, built once an hour ago; returns a call that builds it and
    names what was compiled or linked."""
    pkg, inc, bin_ = tmp_path / "pkg", tmp_path / "include", tmp_path / "bin"
    for d in (pkg / "csrc", inc, bin_):
        d.mkdir(parents=True)
    shutil.copy(build.__file__, pkg / "build.py")
    (inc / "linattn.h").write_text("")
    (pkg / "csrc" / "shared.cuh").write_text('#include "../../include/linattn.h"\n')
    for name in ("one", "two"):
        (pkg / "csrc" / f"{name}.cu").write_text('#include "shared.cuh"\n' if name == "one" else "")
    (bin_ / "nvcc").write_text(STUB)
    (bin_ / "nvcc").chmod(0o755)
    log = tmp_path / "log"

    def run():
        log.write_text("")
        env = dict(os.environ, PATH=f"{bin_}:{os.environ['PATH']}", STUB_LOG=str(log))
        subprocess.check_call([sys.executable, str(pkg / "build.py")], env=env, stdout=subprocess.DEVNULL)
        return sorted({os.path.basename(x) for x in log.read_text().split()})

    run.pkg = pkg
    then = 1_000_000_000
    for p in tmp_path.rglob("*"):
        os.utime(p, (then, then))
    assert run() == ["one.cu", "two.cu", "two.o"]   # the last argument of each call
    for i, p in enumerate([pkg / "_build" / "one.o", pkg / "_build" / "two.o", pkg / "liblinattn.so"]):
        os.utime(p, (then + 10 + i, then + 10 + i))
    return run


def test_nothing_is_made_again_without_a_change(tree):
    assert tree() == []


def test_a_changed_header_remakes_what_reads_it(tree):
    os.utime(tree.pkg / "csrc" / "shared.cuh")
    assert tree() == ["one.cu", "two.o"]


def test_a_changed_flag_remakes_every_object(tree):
    recipe = tree.pkg / "build.py"
    text = recipe.read_text()
    assert '"-O3"' in text
    recipe.write_text(text.replace('"-O3"', '"-O2"'))
    assert tree() == ["one.cu", "two.cu", "two.o"]
    assert "-O2" in (tree.pkg / "_build" / "two.o").read_text()
    assert tree() == []
