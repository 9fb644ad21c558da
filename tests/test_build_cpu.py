"""The build script's own files: nothing beside the sources, and nothing that another build of the same
library, running at the same time, could take away. With a compiler of a few lines of shell."""

import os
import threading

import pytest

from sparse_delta_rule_amd import build

# Writes what it is given: an object holds its source, a library its objects, each after a while.
COMPILER = """#!/bin/sh
out= ; inputs= ; compile=
while [ $# -gt 0 ]; do
  case "$1" in
    -o) out=$2; shift ;;
    -I|-Xclang) shift ;;
    -c) compile=1 ;;
    -*) ;;
    *) inputs="$inputs $1" ;;
  esac
  shift
done
cat $inputs > "$out" || exit 1
sleep 0.2
for i in $inputs; do grep -q broken "$i" && { echo "error: $i" >&2; exit 1; }; done
[ -z "$compile" ] && for i in $inputs; do [ -f "$i" ] || { echo "lost: $i" >&2; exit 1; }; done
exit 0
"""


@pytest.fixture
def project(tmp_path, monkeypatch):
    compiler = tmp_path / "compiler"
    compiler.write_text(COMPILER)
    compiler.chmod(0o755)
    monkeypatch.setenv("HIPCC", str(compiler))
    (tmp_path / "csrc").mkdir()
    for name in "abc":
        (tmp_path / "csrc" / f"{name}.hip").write_text(f"source {name}\n")
    return tmp_path, [str(tmp_path / "csrc" / f"{name}.hip") for name in "abc"]


def files(path):
    return sorted(os.path.relpath(os.path.join(d, f), path) for d, _, fs in os.walk(path) for f in fs)


def test_a_build_leaves_its_library_alone(project):
    path, sources = project
    before = files(path)
    assert build._hipcc(str(path / "lib.so"), sources, False) == str(path / "lib.so")
    assert (path / "lib.so").read_text() == "source a\nsource b\nsource c\n"
    assert files(path) == sorted(before + ["lib.so"])


def test_builds_at_once(project):
    path, sources = project
    failed = []

    def one(n):
        try:
            build._hipcc(str(path / "lib.so"), sources, False)
        except Exception as e:  # noqa: BLE001
            failed.append(e)

    threads = [threading.Thread(target=one, args=(n,)) for n in range(3)]
    for i, t in enumerate(threads):
        t.start()
        if i == 0:
            threading.Event().wait(0.1)  # the others begin while the first compiles
    for t in threads:
        t.join()
    assert failed == []
    assert (path / "lib.so").read_text() == "source a\nsource b\nsource c\n"


@pytest.mark.parametrize("where", ["csrc/b.hip", "link"])
def test_a_failed_build_leaves_nothing_and_the_old_library(project, where, monkeypatch):
    path, sources = project
    (path / "lib.so").write_text("old")
    if where == "link":
        run = build._run_hipcc

        def fail_at_the_link(args, out, verbose):
            run(args, out, verbose)
            if "-shared" in args:
                raise RuntimeError("hipcc failed")

        monkeypatch.setattr(build, "_run_hipcc", fail_at_the_link)
    else:
        (path / where).write_text("broken\n")
    before = files(path)
    with pytest.raises(RuntimeError, match="hipcc failed"):
        build._hipcc(str(path / "lib.so"), sources, False)
    assert files(path) == before and (path / "lib.so").read_text() == "old"
